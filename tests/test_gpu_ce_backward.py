"""The cross entropy's backward pass: how exact its gradients are over the whole range of probabilities, and rows
without loss, against 64 bits.

Tolerances: a rounding to bf16 is off by at most 2^-8 of the value, dz as the sum of two bf16 numbers by 2^-16
(half a step of what the first one left, which is at most 2^-8 of the value), an fp32 step is 2 u = 2^-23.
"""
import pytest
import torch

from sparse_linear_layers_bitlinear_b200 import sbl
from tests.test_gpu_train_ops import BF, U, ce_backward, ce_forward, ce_inputs, logit_bound, randn

pytestmark = pytest.mark.gpu


def pulled_inputs(t, v, d, seed, pull):
    """Rows whose h leans towards its target's row of w by `pull`: a trained network's probabilities."""
    h, w, y = ce_inputs(t, v, d, seed)
    at = y.clamp_min(0)
    return (h.float() + pull * w[at].float()).to(BF), w, y


def exact_backward(h, w, y, lse, dloss):
    """dh, dw in 64 bits, and for each the largest error that the kernel's arithmetic before the outputs' rounding may
    have: every step's own bound on the sum of the magnitudes that it enters."""
    (t, d), v = h.shape, w.shape[0]
    hd, wd = h.double(), w.double()
    z = hd @ wd.T
    live = (y >= 0) & (y < v)
    p = torch.where(live[:, None], (z - lse.double()[:, None]).exp(), 0.0)
    dz = p.clone()
    dz[torch.arange(t, device="cuda")[live], y[live]] -= 1
    g = torch.where(live, dloss.double().expand(t), 0.0)[:, None]
    # the exponential: the logit's error, the rounding of z - lse and the product with log2 e (4 u of the
    # magnitudes), 2^-20 for exp2; the subtraction and the factor dloss 2 u; then the two numbers
    off = p * g.abs() * (logit_bound(h, w) + 4 * U * (z.abs() + lse.double().abs()[:, None]) + 2.0 ** -20) * 1.01
    dz *= g
    off += (2.0 ** -16 + 4 * U) * (dz.abs() + off)
    out = []
    for a, o, b, n in ((dz, off, wd, v), (dz.T, off.T, hd, t)):
        # the sums over both numbers: 2 n / 16 + 64 (pieces and slices among them) of a step each
        out.append((a @ b, o @ b.abs() + (n / 8 + 64) * 2 * U * ((a.abs() + o) @ b.abs())))
    return out


@pytest.mark.parametrize("one", [False, True], ids=["each", "one"])
@pytest.mark.parametrize("pull", [0.0, 5.5, 7.4, 10.0])
@pytest.mark.parametrize("t,v,d", [(512, 4099, 512), (63, 4099, 512), (700, 2048, 136), (4100, 9001, 64), (200, 32768, 256)])
def test_gradients_are_as_exact_as_their_rounding(t, v, d, pull, one):
    """What is left of the arithmetic before the outputs' one rounding to bf16 stays far below it, whatever the
    probabilities: element by element, and over all of a gradient."""
    h, w, y = pulled_inputs(t, v, d, t + v, pull * 512 / d)
    loss, lse = ce_forward(h, w, y)
    dloss = randn(1 if one else t, seed=9, std=0.3, mean=1.0)
    dh, dw = ce_backward(h, w, y, lse, dloss)
    for got, (want, tol) in zip((dh, dw), exact_backward(h, w, y, lse, dloss)):
        err = (got.double() - want).abs()
        assert (err <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
        # all of it: the rounding of the exact values and the bound on the rest.  The rounding errors of the
        # values that were rounded instead are of the same size: 10^4 and more of them, their mean square 2 % at most off
        rounding = (want.to(BF).double() - want).norm()
        assert err.norm() <= 1.02 * rounding + tol.norm(), (err.norm() / rounding).item()


def test_one_gradient_for_no_rows():
    """The mean loss over no rows: its gradient is not finite, and no row has a loss to take it."""
    for t, v, d in ((40, 90, 64), (40, 2500, 64), (3000, 2100, 64)):
        h, w, y = ce_inputs(t, v, d, 3)
        y[:] = -100
        loss, lse = ce_forward(h, w, y)
        for value in (float("inf"), float("nan")):
            dh, dw = ce_backward(h, w, y, lse, torch.tensor([value], device="cuda"))
            assert not dh.any() and not dw.any()


def test_many_tokens_keep_their_pieces_wide():
    """dh's sums pass through memory once a piece of the vocabulary: at least 2048 entries each, however many tokens."""
    t, v, d = 40000, 4500, 64
    h, w, y = ce_inputs(t, v, d, 4)
    loss, lse = ce_forward(h, w, y)
    dloss = randn(t, seed=9, std=0.3, mean=1.0)
    launched = sbl.launch_count()
    dh, dw = ce_backward(h, w, y, lse, dloss)
    assert sbl.launch_count() - launched <= 5  # three pieces: dz of the first, products of each, and a sum at most
    for got, (want, tol) in zip((dh, dw), exact_backward(h, w, y, lse, dloss)):
        assert ((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
