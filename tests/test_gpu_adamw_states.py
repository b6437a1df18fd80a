"""AdamW: the 8-bit states against a plain fp32 form bit for bit, and the root that the update divides by."""
import warnings

import pytest
import torch

from sparse_linear_layers_bitlinear_b200 import sbl
from tests.test_gpu_train_ops import BF, F32, U, randn, same_bits

pytestmark = pytest.mark.gpu
BLOCK = sbl.SBL_ADAMW_BLOCK


def plain_codes(x, top, positive):
    """Codes of fp32 magnitudes as documented: 448 times the reciprocal of the largest, nearest; no zero of a positive."""
    q = x * (448.0 * top.reciprocal()).repeat_interleave(BLOCK)
    if positive:
        q = torch.where(q > 0, q.clamp_min(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("spread", [1.0, 6.0])
def test_8_bit_states_equal_a_plain_form(spread):
    """First moments and both scales bit for bit.  A second moment's code may be that of the root's neighbour in
    fp32, which is another one only next to a border of two codes."""
    n, b1, b2 = 1 << 20, 0.9, 0.95
    w = randn(n, seed=1, std=0.02, dtype=BF)
    # gradients over many magnitudes: with the wide spread roots of fewer bits than the smallest code are among them
    grad = randn(n, seed=2) * (randn(n, seed=3) * spread).exp()
    t = sbl.AdamWTensor.allocate(w, grad, bits=8)
    plan = sbl.AdamWTensors([t])
    for step in (1, 2, 3):
        m0 = t.m.float() * t.m_scale.repeat_interleave(BLOCK)
        v0 = t.v.float() * t.v_scale.repeat_interleave(BLOCK)
        grad.mul_(0.7)
        f = [torch.tensor(x, dtype=F32, device="cuda") for x in (b1, 1 - b1, b2, 1 - b2)]
        m = f[0] * m0 + f[1] * grad
        v = f[2] * (v0 * v0) + f[3] * grad * grad
        root = v.sqrt()
        mtop, rtop = m.abs().view(-1, BLOCK).amax(1), root.view(-1, BLOCK).amax(1)
        sbl.adamw_step(plan, step, lr=1e-3, beta1=b1, beta2=b2)
        unit = torch.tensor(1 / 448, dtype=F32, device="cuda")
        assert same_bits(t.m_scale, mtop * unit) and same_bits(t.v_scale, rtop * unit)
        assert torch.equal(t.m.view(torch.uint8), plain_codes(m, mtop, False))
        got = t.v.view(torch.uint8)
        near = [plain_codes(r, rtop, True) for r in (root, torch.nextafter(root, root * 2), torch.nextafter(root, root * 0))]
        assert ((got == near[0]) | (got == near[1]) | (got == near[2])).all()
        # a neighbour in one root of two million, and one code of some 2^19 next to a border
        assert (got != near[0]).sum().item() <= 1


def test_the_update_s_root():
    """beta1 = beta2 = eps = 0 and w = 0: the update is g / sqrt(g^2), 1 but for the roundings: g^2 half of u (of its
    root), the root itself one step (2 u), the quotient two steps (4 u)."""
    n = 1 << 20
    grad = randn(n, seed=4) * (randn(n, seed=5) * 4).exp()
    t = sbl.AdamWTensor.allocate(torch.zeros(n, dtype=BF, device="cuda"), grad, bits=8)
    sbl.adamw_step(sbl.AdamWTensors([t]), 1, lr=1.0, beta1=0.0, beta2=0.0, eps=0.0)
    live = grad.abs() > 2.0 ** -49  # squares that are normal numbers far inside
    assert live.sum() > n // 2
    assert ((t.master.double() + grad.sign().double())[live].abs() <= 6.5 * U).all()


def test_gradients_allocated_anew_each_step():
    """set_grads: the next step reads the new gradients, of another type too; a refused set changes nothing."""
    sizes = (1000, 0, 257, 4096)

    def tensors():
        out = []
        for i, n in enumerate(sizes):
            w = randn(n, seed=i, std=0.02, dtype=BF)
            out.append(sbl.AdamWTensor.allocate(w, torch.zeros(n, dtype=BF, device="cuda"), bits=8 if i == 3 else 32))
        return out

    a, b = tensors(), tensors()
    plan = sbl.AdamWTensors(a)
    for step, dtype in ((1, BF), (2, F32), (3, BF)):
        grads = [randn(n, seed=10 * step + i, std=1e-3, dtype=dtype) for i, n in enumerate(sizes)]
        plan.set_grads(grads)
        with pytest.raises(sbl.SblError, match="3 gradients for 4 tensors"):
            plan.set_grads(grads[:3])
        with pytest.raises(sbl.SblError, match="missing"):
            plan.set_grads(grads[:3] + [None])
        with pytest.raises(sbl.SblError, match="has 4095 elements"):
            plan.set_grads([g.clone() for g in grads[:3]] + [grads[3][:4095]])
        with pytest.raises(sbl.SblError, match="float16"):
            plan.set_grads([g.clone() for g in grads[:3]] + [grads[3].half()])
        with pytest.raises(sbl.SblError, match="aligned"):
            plan.set_grads(grads[:3] + [torch.zeros(4097, dtype=dtype, device="cuda")[1:]])
        with pytest.raises(sbl.SblError, match="on cpu"):
            plan.set_grads(grads[:3] + [grads[3].cpu()])
        for t, g in zip(b, grads):
            t.grad = g
        sbl.adamw_step(plan, step, lr=1e-3)
        sbl.adamw_step(sbl.AdamWTensors(b), step, lr=1e-3)
        for t, u in zip(a, b):
            assert same_bits(t.w, u.w) and same_bits(t.master, u.master)
            assert torch.equal(t.m.view(torch.uint8), u.m.view(torch.uint8))


def test_arrays_in_two_places_are_refused():
    w, u, grad = (randn(512, seed=i, dtype=BF) for i in range(3))
    z = torch.zeros(512, device="cuda")
    with pytest.raises(sbl.SblError, match="two places"):
        sbl.AdamWTensors([sbl.AdamWTensor(w, grad, z, z)])
    a, b = sbl.AdamWTensor.allocate(w, grad), sbl.AdamWTensor.allocate(u, grad, bits=8)
    sbl.AdamWTensors([a, b])  # the gradient is only read
    with pytest.raises(sbl.SblError, match="two places"):
        sbl.AdamWTensors([a, sbl.AdamWTensor(u, grad, a.m, z)])
    with pytest.raises(sbl.SblError, match="two places"):
        sbl.AdamWTensors([a, sbl.AdamWTensor(w, grad, z, z.clone())])
    with pytest.raises(sbl.SblError, match="two places"):
        sbl.AdamWTensors([a, sbl.AdamWTensor(u, w, z, z.clone())])
    with pytest.raises(sbl.SblError, match="is updated"):
        sbl.AdamWTensors([a]).set_grads([a.m])
    b.m_scale = b.v_scale
    with pytest.raises(sbl.SblError, match="two places"):
        sbl.AdamWTensors([b])


def test_8_bit_states_say_where_they_cannot_follow():
    """The documented reach of nearest rounding, and the warning beyond it."""
    n = BLOCK

    def codes(beta2, ratio):
        """The second moments' codes before and after a step whose gradients are `ratio` times each one's root; the
        block's largest stays."""
        v = torch.linspace(8, 112, n, device="cuda").to(torch.float8_e4m3fn)
        v[0] = 448.0
        scale = torch.ones(1, device="cuda")
        grad = v.float() * ratio
        grad[0] = 448.0
        t = sbl.AdamWTensor(torch.zeros(n, dtype=BF, device="cuda"), grad, torch.zeros_like(v), v.clone(), scale.clone(), scale.clone())
        sbl.adamw_step(sbl.AdamWTensors([t]), 100, lr=1e-3, beta2=beta2)
        assert abs(t.v_scale.item() - 1) < 1e-6
        return v.float()[1:], t.v.float()[1:]

    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for ratio, moves in ((0.0, False), (1.4, False), (2.0, True)):
            before, after = codes(0.95, ratio)
            assert torch.equal(before, after) != moves
            assert not moves or (after > before).all()
    with pytest.warns(UserWarning, match="hardly move"):
        for ratio, moves in ((0.0, False), (8.0, False), (12.0, True)):
            before, after = codes(0.999, ratio)
            assert torch.equal(before, after) != moves
