"""Norm, AdamW and linear cross entropy on the GPU against plain 64-bit forms.

Tolerances: u = 2^-24 is half a step of fp32, a rounding to bf16 is off by at
most 2^-8 of the value (half a step), one to e4m3 by 2^-4 (or half of its smallest
step, 2^-10, at the bottom).  Each bound below counts the roundings of the
formula it stands beside, on the sum of the magnitudes that enter it.
"""
import math

import pytest
import torch

from sparse_linear_layers_bitlinear_b200 import sbl, synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16
F32 = torch.float32
EPS = 1e-5


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed, std=1.0, mean=0.0, dtype=F32):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * std + mean).to(dtype)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def same_bits(a, b):
    view = {2: torch.int16, 4: torch.int32, 1: torch.int8}[a.element_size()]
    return a.dtype == b.dtype and torch.equal(a.view(view), b.view(view))


# ---------------------------------------------------------------------------
# Norm, forward
# ---------------------------------------------------------------------------
def norm_all(x, res=None, w=None, eps=EPS, st=None, stream=None):
    """Every output of one call."""
    t, k = x.shape
    dt = x.dtype if res is None else res.dtype
    out = {"h_out": torch.empty(t, k, dtype=dt, device="cuda"), "xn_out": torch.empty(t, k, dtype=BF, device="cuda"),
           "xhat_out": torch.empty(t, k, dtype=BF, device="cuda"), "xq_out": torch.empty(t, k, dtype=torch.int8, device="cuda"),
           "xscale_out": torch.empty(t, device="cuda"), "rstd_out": torch.empty(t, device="cuda")}
    sbl.rmsnorm_forward(x, t, k, eps, residual=res, weight=w, status=st, stream=stream, **out)
    return out


def check_norm(out, x, res, w, eps=EPS):
    t, k = x.shape
    if res is None:
        assert same_bits(out["h_out"], x)
    else:
        assert same_bits(out["h_out"], (x.float() + res.float()).to(res.dtype))  # one fp32 sum, one rounding
    h = out["h_out"].float()
    exact = (h.double().square().mean(1) + eps).rsqrt()
    assert ((out["rstd_out"].double() - exact).abs() <= U * (1 + 1e-6) * exact).all()
    xn = h * out["rstd_out"][:, None]
    if w is not None:
        xn = xn * w.float()
    assert same_bits(out["xn_out"], xn.to(BF))
    # the codes: those of the act-quant of xn (its own kernel takes k % 64 == 0), and their values
    xf = out["xn_out"].double()
    top = xf.abs().amax(1).clamp_min(float(torch.tensor(1e-5)))
    assert torch.equal(out["xscale_out"].double(), top)
    assert torch.equal(out["xq_out"].double(), (127 * xf / top[:, None]).round())
    assert same_bits(out["xhat_out"], (out["xq_out"].double() * top[:, None] / 127).to(BF))
    if k % 64 == 0:
        xq, xs = torch.empty_like(out["xq_out"]), torch.empty(t, device="cuda")
        sbl.quantize_activations(out["xn_out"], t, k, xq, xs, status())
        assert torch.equal(xq, out["xq_out"]) and torch.equal(xs, out["xscale_out"])


NORM_TYPES = [(BF, None), (F32, None), (BF, BF), (F32, BF), (BF, F32), (F32, F32)]


@pytest.mark.parametrize("k", [8, 64, 264, 512, 768, 1024, 1032, 2048, 2056, 2560, 4096, 4104, 6912, 8200, 12288,
                               16384])
@pytest.mark.parametrize("xt,rt", NORM_TYPES)
def test_norm_row_lengths_and_types(k, xt, rt):
    for t, wt in ((1, None), (5, BF), (37, F32)):
        x = randn(t, k, seed=k, dtype=xt)
        res = None if rt is None else randn(t, k, seed=k + 1, std=2.0, dtype=rt)
        w = None if wt is None else randn(k, seed=3, std=0.2, mean=1.0, dtype=wt)
        check_norm(norm_all(x, res, w), x, res, w)


@pytest.mark.parametrize("k", [8, 64, 264, 768, 1024, 1032, 2048, 2560, 4096, 4104, 5128, 6912, 8200, 12288, 16384])
@pytest.mark.parametrize("xt,rt", NORM_TYPES)
def test_norm_rows_walked_by_resident_blocks(k, xt, rt):
    """More than two rows an SM: blocks walk rows (other warps a row, other vectors a lane), one row or several a block."""
    t = 1801 if k <= 1032 else 701
    x = randn(t, k, seed=k, dtype=xt)
    res = None if rt is None else randn(t, k, seed=k + 1, std=2.0, dtype=rt)
    w = randn(k, seed=3, std=0.2, mean=1.0, dtype=BF if k % 16 else F32)
    x[5] = 0
    if res is not None:
        res[5] = 0
    check_norm(norm_all(x, res, w), x, res, w)
    if k in (1024, 16384):
        check_norm(norm_all(x, res), x, res, None)


def test_norm_many_rows():
    x, res, w = randn(4099, 2560, seed=1), randn(4099, 2560, seed=2, dtype=BF), randn(2560, seed=3, dtype=BF)
    check_norm(norm_all(x, res, w), x, res, w)
    # the stream in place, with the next row's loads under way
    stream = res.clone()
    xn = torch.empty_like(res)
    sbl.rmsnorm_forward(x, 4099, 2560, EPS, residual=stream, weight=w, h_out=stream, xn_out=xn)
    assert same_bits(stream, (x + res.float()).to(BF))


def test_norm_zero_rows_and_extreme_magnitudes():
    x = randn(6, 320, seed=4)
    x[0] = 0
    x[1] = 0
    x[1, 7] = 1e-30
    x[2] *= 1e30  # squares outside fp32
    x[3] *= 1e-20
    x[4] *= 3e37
    st = status()
    check_norm(norm_all(x, st=st), x, None, None)
    assert st.item() == 0
    b = randn(2, 320, seed=5, dtype=BF) * 1e38
    check_norm(norm_all(b), b, None, None)
    z = torch.zeros(3, 64, dtype=BF, device="cuda")
    out = norm_all(z, z.clone())
    assert not out["xq_out"].any() and not out["xn_out"].any()
    assert torch.equal(out["xscale_out"], torch.full((3,), 1e-5, device="cuda"))


@pytest.mark.parametrize("k", [64, 2560, 6912])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_norm_nonfinite_rows_are_flagged_and_stay_apart(k, value):
    x = randn(9, k, seed=6)
    clean = norm_all(x)
    x[4, k // 2] = value
    st = status()
    out = norm_all(x, st=st)
    assert st.item() == sbl.SBL_STATUS_NONFINITE_X
    rows = [0, 1, 2, 3, 5, 6, 7, 8]
    for name in out:
        assert same_bits(out[name][rows].contiguous(), clean[name][rows].contiguous()), name


def test_norm_overflowing_gain_is_flagged():
    x = randn(2, 64, seed=7)
    w = torch.full((64,), 3e38, device="cuda")
    st = status()
    xn = torch.empty(2, 64, dtype=BF, device="cuda")
    sbl.rmsnorm_forward(x, 2, 64, EPS, weight=w, xn_out=xn, status=st)
    assert st.item() == sbl.SBL_STATUS_NONFINITE_X


def test_norm_single_outputs_in_place_and_views():
    t, k = 7, 2560
    flat_x, flat_r = randn(t * k + 64, seed=8), randn(t * k + 64, seed=9, dtype=BF)
    x, res = flat_x[4:4 + t * k].view(t, k), flat_r[8:8 + t * k].view(t, k)  # 16-byte aligned, no more
    full = norm_all(x, res)
    for name, want in full.items():
        got = torch.empty_like(want)
        sbl.rmsnorm_forward(x, t, k, EPS, residual=res, **{name: got})
        assert same_bits(got, want), name
    stream = res.clone()
    sbl.rmsnorm_forward(x, t, k, EPS, residual=stream, h_out=stream, xn_out=full["xn_out"])  # the stream in place
    assert same_bits(stream, full["h_out"])
    # memory behind the last row stays as it was
    guard = torch.full((t * k + 64,), 7.0, dtype=BF, device="cuda")
    sbl.rmsnorm_forward(x, t, k, EPS, residual=res, xn_out=guard[:t * k].view(t, k))
    assert (guard[t * k:] == 7.0).all()


def test_norm_on_a_side_stream_and_in_a_graph():
    t, k = 65, 2560
    x, res, w = randn(t, k, seed=10), randn(t, k, seed=11, dtype=BF), randn(k, seed=12, dtype=BF)
    want = norm_all(x, res, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = norm_all(x, res, w, stream=side)
    torch.cuda.synchronize()
    assert all(same_bits(out[n], want[n]) for n in want)
    bufs = {n: torch.zeros_like(v) for n, v in want.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sbl.rmsnorm_forward(x, t, k, EPS, residual=res, weight=w, **bufs)
    x.mul_(-1.5)
    want = norm_all(x, res, w)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(same_bits(bufs[n], want[n]) for n in want)


def test_norm_codes_enter_the_products():
    n_out, k, t = 264, 320, 50
    layer = sbl.Layer.allocate(n_out, k, 2, 4)
    sbl.prepare_weights(layer, synth.master_weights(n_out, k, 1, "cuda"))
    x = randn(t, k, seed=13)
    out = norm_all(x)
    y, want = torch.empty(t, n_out, device="cuda"), torch.empty(t, n_out, device="cuda")
    sbl.forward_quantized(layer, out["xq_out"], out["xscale_out"], t, y)
    ws = torch.empty(sbl.workspace_bytes(t, k), dtype=torch.uint8, device="cuda")
    sbl.forward(layer, out["xn_out"], t, want, workspace=ws)
    assert torch.equal(y, want)


# ---------------------------------------------------------------------------
# Norm, backward
# ---------------------------------------------------------------------------
def norm_bwd(h, dys, w=None, dres=None, want_dx=True, want_dw=True, rstd=None, stream=None):
    t, k = h.shape
    if rstd is None:
        rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    out = {"dh": torch.empty_like(h), "dx": torch.empty(t, k, dtype=BF, device="cuda") if want_dx else None,
           "dw": torch.empty(k, device="cuda") if want_dw else None}
    ws = torch.empty(max(sbl.rmsnorm_backward_workspace_bytes(t, k), 1), dtype=torch.uint8, device="cuda")
    sbl.rmsnorm_backward(h, rstd, dys, t, k, out["dh"], weight=w, dres=dres, dx=out["dx"], dw=out["dw"], workspace=ws,
                         stream=stream)
    return out, rstd


def check_norm_bwd(out, rstd, h, dys, w, dres):
    t, k = h.shape
    hd, r = h.double(), rstd.double()[:, None]
    g = sum(d.double() for d in dys)
    ga = sum(d.double().abs() for d in dys)
    wd = w.double() if w is not None else torch.ones(k, dtype=torch.float64, device="cuda")
    n = hd * r
    c = (wd * g * n).mean(1, keepdim=True)
    ca = (wd.abs() * ga * n.abs()).mean(1, keepdim=True)
    dr = dres.double() if dres is not None else torch.zeros_like(hd)
    dh = dr + r * (wd * g - n * c)
    # dh: g 2 roundings, w g 1, n 1, the difference 1, the product 1, the sum 1; the mean's terms carry 5 and
    # its sum one for each of at most 32 elements a thread, 5 shuffles, 16 warps and the factor 1 / k
    tol = 8 * U * (dr.abs() + r * (wd.abs() * ga + n.abs() * c.abs())) + r * n.abs() * ca * (5 + 32 + 5 + 16 + 2) * U
    half = {BF: 2.0 ** -8, F32: 0.0}
    assert ((out["dh"].double() - dh).abs() <= tol + half[h.dtype] * (dh.abs() + tol)).all()
    if out["dx"] is not None:
        assert ((out["dx"].double() - dh).abs() <= tol + 2.0 ** -8 * (dh.abs() + tol)).all()
    if out["dw"] is not None:
        dw, dwa = (g * n).sum(0), (ga * n.abs()).sum(0)
        # a term 4 roundings; a thread adds at most all t rows, then 16 groups, 256 blocks
        assert ((out["dw"].double() - dw).abs() <= (4 + t + 16 + 256) * U * dwa).all()


@pytest.mark.parametrize("k", [8, 256, 264, 512, 1000, 1024, 1032, 2048, 2560, 4096, 4104, 6912, 8200, 12288, 16384])
@pytest.mark.parametrize("ht,dt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_norm_backward_row_lengths_and_types(k, ht, dt):
    for t, count, wt, with_res in ((1, 1, None, False), (6, 2, BF, True), (333, 3, F32, True)):
        h = randn(t, k, seed=k, std=2.0, dtype=ht)
        dys = [randn(t, k, seed=20 + i, dtype=dt) for i in range(count)]
        w = None if wt is None else randn(k, seed=3, std=0.2, mean=1.0, dtype=wt)
        dres = randn(t, k, seed=30, dtype=ht) if with_res else None
        out, rstd = norm_bwd(h, dys, w, dres)
        check_norm_bwd(out, rstd, h, dys, w, dres)


@pytest.mark.parametrize("k", [8, 256, 264, 1000, 1032, 2048, 2560, 4104, 6912, 12288, 16384])
@pytest.mark.parametrize("ht,dt", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_norm_backward_rings_of_many_rows(k, ht, dt):
    """Several rows a group and several groups a block, rings of every depth that the sizes give."""
    t = 5003 if k <= 1032 else 1801 if k <= 4104 else 601
    count = 1 + k // 8 % 3
    h = randn(t, k, seed=k, std=2.0, dtype=ht)
    dys = [randn(t, k, seed=20 + i, dtype=dt) for i in range(count)]
    w, dres = randn(k, seed=3, std=0.2, mean=1.0, dtype=BF), randn(t, k, seed=30, dtype=ht)
    out, rstd = norm_bwd(h, dys, w, dres)
    check_norm_bwd(out, rstd, h, dys, w, dres)
    out, rstd = norm_bwd(h, dys[:1], None, None, rstd=rstd)
    check_norm_bwd(out, rstd, h, dys[:1], None, None)


def test_norm_backward_many_rows_in_place_and_repeatable():
    t, k = 5003, 2560
    h, dys = randn(t, k, seed=1, dtype=BF), [randn(t, k, seed=2, dtype=BF)]
    w, dres = randn(k, seed=3, dtype=BF), randn(t, k, seed=4, dtype=BF)
    out, rstd = norm_bwd(h, dys, w, dres)
    check_norm_bwd(out, rstd, h, dys, w, dres)
    again, _ = norm_bwd(h, dys, w, dres)
    assert all(same_bits(out[n], again[n]) for n in out)  # fixed order of every sum
    stream = dres.clone()
    sbl.rmsnorm_backward(h, rstd, dys, t, k, stream, weight=w, dres=stream)
    assert same_bits(stream, out["dh"])
    # the same gradient given as two halves
    two, _ = norm_bwd(h, [dys[0] * 0.5, dys[0] * 0.5], w, dres)
    assert same_bits(two["dh"], out["dh"])


def test_norm_backward_against_differences():
    """dh against central differences of sum(G xn(h)) in 64 bits."""
    t, k = 3, 96
    h, w, G = randn(t, k, seed=5), randn(k, seed=6, std=0.3, mean=1.0), randn(t, k, seed=7)
    out, _ = norm_bwd(h, [G], w)

    def f(hd, wd):
        return (G.double() * hd * (hd.square().mean(1, keepdim=True) + EPS).rsqrt() * wd).sum()

    hd, wd, e = h.double(), w.double(), 1e-6
    for seed in range(8):
        d = torch.randn(t, k, generator=gen(100 + seed), device="cuda", dtype=torch.float64)
        got = (out["dh"].double() * d).sum()
        want = (f(hd + e * d, wd) - f(hd - e * d, wd)) / (2 * e)
        # differences: e^2 times third derivatives, and 1e-16 |f| / e; dh: some 70 u of its terms
        scale = (out["dh"].double().abs() * d.abs()).sum() + (G.double().abs() * d.abs()).sum()
        assert abs(got - want) <= 1e-5 * scale
        dv = torch.randn(k, generator=gen(200 + seed), device="cuda", dtype=torch.float64)
        want = (f(hd, wd + e * dv) - f(hd, wd - e * dv)) / (2 * e)
        assert abs((out["dw"].double() * dv).sum() - want) <= 1e-5 * (out["dw"].double().abs() * dv.abs()).sum()


def test_norm_backward_empty_and_graph():
    k = 64
    dw = torch.ones(k, device="cuda")
    e = torch.empty(0, k, dtype=BF, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    sbl.rmsnorm_backward(e, torch.empty(0, device="cuda"), [e], 0, k, e, dw=dw, workspace=ws)
    assert not dw.any()
    t, k = 129, 2560
    h, G, w = randn(t, k, seed=8, dtype=BF), randn(t, k, seed=9, dtype=BF), randn(k, seed=10, dtype=BF)
    want, rstd = norm_bwd(h, [G], w)
    dh, dw = torch.zeros_like(h), torch.zeros(k, device="cuda")
    ws = torch.empty(sbl.rmsnorm_backward_workspace_bytes(t, k), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sbl.rmsnorm_backward(h, rstd, [G], t, k, dh, weight=w, dw=dw, workspace=ws)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert same_bits(dh, want["dh"]) and same_bits(dw, want["dw"])


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
BLOCK = sbl.SBL_ADAMW_BLOCK


def adam_tensor(n, bits, gt, master, decay, seed, fresh=False):
    w32 = randn(n, seed=seed, std=0.02)
    grad = randn(n, seed=seed + 1, std=1e-3, dtype=gt)
    t = sbl.AdamWTensor.allocate(w32.to(BF), grad, bits=bits, master=master, decay=decay)
    if master:
        t.master.copy_(w32)
    if not fresh:
        m, r = randn(n, seed=seed + 2, std=5e-4), randn(n, seed=seed + 3, std=1e-3).abs()
        if bits == 32:
            t.m.copy_(m)
            t.v.copy_(r.square())
        else:
            for x, codes, scale in ((m, t.m, t.m_scale), (r, t.v, t.v_scale)):
                for b in range(0, n, BLOCK):
                    top = x[b:b + BLOCK].abs().max() / 448
                    scale[b // BLOCK] = top
                    codes[b:b + BLOCK] = (x[b:b + BLOCK] / top).to(torch.float8_e4m3fn)
    return t


def spread(scale, n):
    return scale.double().repeat_interleave(BLOCK)[:n]


def adam_before(t):
    n = t.w.numel()
    value = (t.master if t.master is not None else t.w).double().clone()
    if t.m_scale is None:
        return value, t.m.double().clone(), t.v.double().clone()
    m, r = t.m.view(torch.float8_e4m3fn).float().double(), t.v.view(torch.float8_e4m3fn).float().double()
    return value, m * spread(t.m_scale, n), (r * spread(t.v_scale, n)) ** 2


def check_adam(t, before, step, scale=1.0, lr=HYPER["lr"]):
    w, m0, v0 = before
    b1, b2, n = HYPER["beta1"], HYPER["beta2"], t.w.numel()
    g = t.grad.double() * scale
    m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
    ma = b1 * m0.abs() + (1 - b1) * g.abs()
    den = (v / (1 - b2 ** step)).sqrt() + HYPER["eps"]
    up = lr * m / (1 - b1 ** step) / den
    upa = lr * ma / (1 - b1 ** step) / den
    wd = HYPER["weight_decay"] if t.decay else 0.0
    value = w * (1 - lr * wd) - up
    # the step: m 5 roundings, v 7 under a root, root, factor, sum, quotient, rate 2 each; the value's own sum 2,
    # the decay's factor 2 and the product
    tol = U * (5 * w.abs() + 2 * value.abs()) + 24 * U * upa
    half = 2.0 ** -8
    if t.master is not None:
        assert ((t.master.double() - value).abs() <= tol).all()
        assert same_bits(t.w, t.master.to(BF))
    else:
        assert ((t.w.double() - value).abs() <= tol + half * (value.abs() + tol)).all()
    if t.m_scale is None:
        assert ((t.m.double() - m).abs() <= 5 * U * ma).all()
        # below 2^-126, fp32's smallest normal value, a rounding is off by up to 2^-150 whatever the value is:
        # with g around 1e-19 and less, g^2 gets there, and its roundings (7 at most) add 7 x 2^-150
        assert ((t.v.double() - v).abs() <= 7 * U * v + 7 * 2.0 ** -150).all()
        return
    for x, xa, codes, scales, low in ((m, ma, t.m, t.m_scale, 2.0 ** -10), (v.sqrt(), v.sqrt(), t.v, t.v_scale, 2.0 ** -9)):
        blocks = -(-n // BLOCK)
        pad, pada = torch.zeros(blocks * BLOCK, dtype=torch.float64, device="cuda"), None
        pad[:n] = x.abs()
        top = pad.view(-1, BLOCK).amax(1)
        pad[:n] = xa
        topa = pad.view(-1, BLOCK).amax(1)
        assert ((scales.double() - top / 448).abs() <= 8 * U * topa / 448).all()
        back = codes.view(torch.float8_e4m3fn).float().double() * spread(scales, n)
        # half a step of e4m3, at the bottom half its smallest step (all of it where zero is avoided)
        bound = 2.0 ** -4 * x.abs() + low * spread(top / 448, n) + 16 * U * spread(topa, n)
        assert ((back - x).abs() <= bound * (1 + 1e-6)).all()
    assert ((t.v.view(torch.uint8) != 0) | (v == 0) | (spread(t.v_scale, n) == 0)).all()


SIZES = [1, 3, 4, 255, 256, 257, 1000, 4095, 4096, 4097, 10007, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("master", [True, False])
def test_adamw_sizes(bits, gt, master):
    ts = [adam_tensor(n, bits, gt, master, i % 2 == 0, 10 * i) for i, n in enumerate(SIZES)]
    plan = sbl.AdamWTensors(ts)
    st = status()
    for step in (1, 2, 1000):
        before = [adam_before(t) for t in ts]
        sbl.adamw_step(plan, step, status=st, **HYPER)
        for t, b in zip(ts, before):
            check_adam(t, b, step)
    assert st.item() == 0


def test_adamw_8bit_states_equal_a_plain_form_bit_for_bit():
    """The moments' roundings are pinned (every product and sum by itself, the quotients through a reciprocal), so
    the codes, which sit behind one more rounding, are the same in any fp32 form written that way."""
    n = 1000 * BLOCK
    t = adam_tensor(n, 8, BF, True, True, 11)
    plan = sbl.AdamWTensors([t])
    c = {k: torch.tensor(v, device="cuda", dtype=F32) for k, v in
         dict(b1=0.9, a1=1 - 0.9, b2=0.95, a2=1 - 0.95, up=448.0, low=2.0 ** -9).items()}
    down = torch.ones((), device="cuda") / c["up"]
    for step in range(1, 6):
        m, r = (x.float().view(-1, BLOCK) * s[:, None] for x, s in ((t.m, t.m_scale), (t.v, t.v_scale)))
        g = t.grad.float().view(-1, BLOCK)
        m = c["b1"] * m + c["a1"] * g
        r = (c["b2"] * (r * r) + c["a2"] * g * g).sqrt()
        sbl.adamw_step(plan, step, **HYPER)
        for x, codes, scales in ((m, t.m, t.m_scale), (r, t.v, t.v_scale)):
            top = x.abs().amax(1)
            assert same_bits(scales, top * down)
            q = x * (top.reciprocal() * c["up"])[:, None]
            if codes is t.v:
                q = torch.where(q > 0, torch.maximum(q, c["low"]), q)
            assert same_bits(codes.view(torch.int8), q.to(torch.float8_e4m3fn).view(-1).view(torch.int8))


def test_adamw_mixed_tensors_over_several_launches():
    ts = []
    for i in range(300):
        ts.append(adam_tensor(1 + (i * 37) % 700, (32, 8)[i % 2], (BF, F32)[i // 2 % 2], i % 3 == 0, i % 5 != 0, i))
    ts.insert(7, sbl.AdamWTensor.allocate(torch.empty(0, dtype=BF, device="cuda"), torch.empty(0, device="cuda")))
    before = [adam_before(t) for t in ts]
    launched = sbl.launch_count()
    sbl.adamw_step(sbl.AdamWTensors(ts), 3, **HYPER)
    assert sbl.launch_count() - launched == 4  # 150 of each kind, 128 a launch, the empty one left out
    for t, b in zip(ts, before):
        if t.w.numel():
            check_adam(t, b, 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_from_zero_states_and_zero_gradients(bits):
    t = adam_tensor(1000, bits, F32, True, True, 5, fresh=True)
    t.grad[256:512] = 0
    t.grad[600:] *= 1e-12
    plan = sbl.AdamWTensors([t])
    for step in range(1, 4):
        before = adam_before(t)
        sbl.adamw_step(plan, step, **HYPER)
        check_adam(t, before, step)
    if bits == 8:
        assert t.m_scale[1].item() == 0 and t.v_scale[1].item() == 0


def test_adamw_tiny_blocks_hold_zeros():
    t = adam_tensor(256, 8, F32, True, True, 6, fresh=True)
    t.grad.fill_(1e-33)
    sbl.adamw_step(sbl.AdamWTensors([t]), 1, **HYPER)
    assert t.m_scale.item() == 0 and not t.m.view(torch.uint8).any()  # 1e-34 < 2^-100
    assert t.v_scale.item() == 0 and not t.v.view(torch.uint8).any()


def test_adamw_leaves_its_neighbours_alone():
    flat = {n: torch.full((3000,), 3.0, dtype=dt, device="cuda") for n, dt in
            (("w", BF), ("master", F32), ("grad", BF), ("m", F32), ("v", F32))}
    at = slice(512, 512 + 1003)
    t = sbl.AdamWTensor(flat["w"][at], flat["grad"][at], flat["m"][at], flat["v"][at], master=flat["master"][at])
    before = adam_before(t)
    sbl.adamw_step(sbl.AdamWTensors([t]), 2, **HYPER)
    check_adam(t, before, 2)
    for x in flat.values():
        assert (x[:512] == 3).all() and (x[512 + 1003:] == 3).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_device_scalars_in_a_replayed_graph(bits):
    a, b = (adam_tensor(5000, bits, BF, True, True, 8) for _ in range(2))
    lr, step = torch.tensor([1e-3], device="cuda"), torch.tensor([1], dtype=torch.int64, device="cuda")
    scale = torch.tensor([0.5], device="cuda")
    plan = sbl.AdamWTensors([a])
    keep = [x.clone() for x in (a.w, a.master, a.m.view(torch.uint8) if bits == 8 else a.m, a.v.view(torch.uint8) if bits == 8 else a.v)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sbl.adamw_step(plan, 0, lr_dev=lr, step_dev=step, grad_scale_dev=scale, **HYPER)
        step.add_(1)
    assert same_bits(a.w, keep[0])  # a capture runs nothing
    for i in range(1, 4):
        lr.fill_(1e-3 * i)
        before = adam_before(a)
        g.replay()
        torch.cuda.synchronize()
        check_adam(a, before, i, scale=0.5, lr=float(lr))
    b.grad.mul_(0.5)  # exact in bf16
    for i in range(1, 4):
        before = adam_before(b)
        sbl.adamw_step(sbl.AdamWTensors([b]), i, **{**HYPER, "lr": 1e-3 * i})
        check_adam(b, before, i, lr=1e-3 * i)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_flags_nonfinite_gradients(bits):
    for value in (float("nan"), float("inf")):
        t = adam_tensor(2000, bits, F32, True, True, 9)
        t.grad[1500] = value
        clean = adam_before(t)
        st = status()
        sbl.adamw_step(sbl.AdamWTensors([t]), 1, status=st, **HYPER)
        assert st.item() == sbl.SBL_STATUS_NONFINITE_G
        assert torch.isfinite(t.master[:1280]).all() and torch.isfinite(t.master[1536:]).all()
        assert not torch.equal(t.master[:1280].double(), clean[0][:1280])


# ---------------------------------------------------------------------------
# Linear cross entropy
# ---------------------------------------------------------------------------
def ce_inputs(t, v, d, seed, ignored=True, std=0.05):
    h, w = randn(t, d, seed=seed, dtype=BF), randn(v, d, seed=seed + 1, std=std, dtype=BF)
    y = torch.randint(0, v, (t,), generator=gen(seed + 2), device="cuda")
    if ignored and t > 2:
        y[::7] = -100
    return h, w, y


def ce_forward(h, w, y, st=None, stream=None, ignore=-100):
    (t, d), v = h.shape, w.shape[0]
    loss, lse = torch.full((t,), 9e9, device="cuda"), torch.full((t,), 9e9, device="cuda")
    ws = torch.empty(sbl.linear_ce_workspace_bytes(t, v, d), dtype=torch.uint8, device="cuda")
    sbl.linear_ce_forward(h, w, y, t, v, d, loss, lse, ws, ignore_index=ignore, status=st, stream=stream)
    return loss, lse


def logit_bound(h, w):
    """Largest error of a token's logits: products exact in fp32, d / 16 + 16 sums (the tensor core adds 16
    products at a time), each off by a step (2 u) of the magnitudes' sum."""
    d = h.shape[1]
    return (d / 16 + 16) * 2 * U * (h.double().abs() @ w.double().abs().T)


def check_ce(loss, lse, h, w, y, ignore=-100):
    z = h.double() @ w.double().T
    ref = torch.logsumexp(z, 1)
    live = y != ignore
    want = torch.where(live, ref - z.gather(1, torch.where(live, y, 0)[:, None])[:, 0], 0.0)
    zb = logit_bound(h, w).amax(1)
    # exponents off by 2 u of |z - max| (at most 2 max |z|), their sums' roundings, exp2 and log: 2^-20 in all
    tol = zb + 8 * U * z.abs().amax(1) + 2.0 ** -20
    assert ((lse.double() - ref).abs() <= tol).all()
    assert ((loss.double() - want).abs() <= 2 * tol).all()
    assert not loss[~live].any()


CE_SHAPES = [(1, 1, 8), (1, 17, 64), (2, 300, 8), (3, 255, 72), (63, 4099, 512), (257, 256, 264), (255, 257, 64),
             (300, 1000, 2560), (513, 5003, 128), (129, 40000, 64), (1, 32768, 2560)]


@pytest.mark.parametrize("t,v,d", CE_SHAPES)
def test_linear_ce_forward(t, v, d):
    h, w, y = ce_inputs(t, v, d, t + v)
    st = status()
    loss, lse = ce_forward(h, w, y, st)
    check_ce(loss, lse, h, w, y)
    assert st.item() == 0
    again = ce_forward(h, w, y)
    assert same_bits(again[0], loss) and same_bits(again[1], lse)


def test_linear_ce_large_logits_and_one_sided_rows():
    h, w, y = ce_inputs(70, 700, 128, 3, ignored=False, std=2.0)  # logits in the tens: most exponentials vanish
    h[0] = 0       # a uniform row
    h[1] = 30.0
    w[5] = 1.0     # a logit of 3840, far above the others
    y[1] = 5
    loss, lse = ce_forward(h, w, y)
    check_ce(loss, lse, h, w, y)
    assert abs(loss[0].item() - math.log(700)) < 1e-5
    assert loss[1].item() == 0


def test_linear_ce_ignored_and_bad_targets():
    h, w, y = ce_inputs(40, 100, 64, 4, ignored=False)
    y[:] = 7
    loss, lse = ce_forward(h, w, y, ignore=7)  # an index inside the vocabulary can be the ignored one
    assert not loss.any()
    y[3], y[4], y[5] = 100, -1, 2 ** 40
    st = status()
    loss, lse2 = ce_forward(h, w, y, st)
    assert st.item() == sbl.SBL_STATUS_BAD_TARGET
    assert torch.isnan(loss[3:6]).all() and torch.isfinite(loss[:3]).all() and torch.isfinite(loss[6:]).all()
    assert same_bits(lse, lse2)


def ce_backward(h, w, y, lse, dloss, st=None, ignore=-100, stream=None):
    (t, d), v = h.shape, w.shape[0]
    dh, dw = torch.full_like(h, 5.0), torch.full_like(w, 5.0)
    ws = torch.empty(sbl.linear_ce_workspace_bytes(t, v, d, True), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)  # what the workspace held before does not count
    sbl.linear_ce_backward(h, w, y, lse, dloss, t, v, d, dh, dw, ws, ignore_index=ignore, status=st, stream=stream)
    return dh, dw


def check_ce_bwd(dh, dw, h, w, y, lse, dloss, ignore=-100):
    hd, wd = h.double(), w.double()
    (t, d), v = h.shape, w.shape[0]
    z = hd @ wd.T
    good = (y != ignore) & (y >= 0) & (y < v)
    p = (z - lse.double()[:, None]).exp()
    hot = torch.zeros_like(p)
    hot[torch.arange(t, device="cuda")[good], y[good]] = 1
    g = torch.where(good, dloss.double().expand(t), 0.0)[:, None]
    dz = (p - hot) * g
    # dz: the exponential is off by the logit's error, 4 u of |z| + |lse| and 2^-20; then one rounding to bf16.
    # dh = dloss (dz w).  dw = dz^T (dloss h) takes dloss h rounded to bf16 too, once more 2^-8 of every term
    # (not where one dloss stands for all rows: it multiplies the sum).
    off = p * (logit_bound(h, w) + 4 * U * (z.abs() + lse.double().abs()[:, None]) + 2.0 ** -20) * g.abs() * 1.1
    zt = off + 2.0 ** -8 * (dz.abs() + off) + 1e-38
    zw = zt + (2.0 ** -8 * (dz.abs() + zt) if dloss.numel() > 1 else 0.0)
    for got, want, a, b, n in ((dh, dz @ wd, (dz.abs() + zt) @ wd.abs(), zt @ wd.abs(), v),
                               (dw, dz.T @ hd, (dz.abs() + zw).T @ hd.abs(), zw.T @ hd.abs(), t)):
        # the product: n / 16 + 64 sums of a step each (pieces and slices among them), the factor dloss one
        # rounding more, one rounding to bf16
        tol = b + (n / 16 + 65) * 2 * U * a
        assert ((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()


@pytest.mark.parametrize("t,v,d", CE_SHAPES)
def test_linear_ce_backward(t, v, d):
    h, w, y = ce_inputs(t, v, d, t + v)
    loss, lse = ce_forward(h, w, y)
    dloss = randn(t, seed=9, std=0.3, mean=1.0)
    dh, dw = ce_backward(h, w, y, lse, dloss)
    check_ce_bwd(dh, dw, h, w, y, lse, dloss)
    again = ce_backward(h, w, y, lse, dloss)
    assert same_bits(again[0], dh) and same_bits(again[1], dw)


@pytest.mark.parametrize("t,v,d", [(4100, 9001, 64), (9000, 8193, 264), (9000, 12001, 64), (300, 150001, 64)])
def test_linear_ce_backward_in_pieces(t, v, d):
    h, w, y = ce_inputs(t, v, d, 5)
    loss, lse = ce_forward(h, w, y)
    check_ce(loss, lse, h, w, y)
    dloss = randn(1, seed=9, std=0.1, mean=1.0 / t)  # one gradient for all rows
    launched = sbl.launch_count()
    dh, dw = ce_backward(h, w, y, lse, dloss)
    assert sbl.launch_count() - launched >= 3  # dz of the first piece, two pieces at least
    check_ce_bwd(dh, dw, h, w, y, lse, dloss)


@pytest.mark.parametrize("one", [False, True], ids=["each", "one"])
@pytest.mark.parametrize("t,v,d", [(3000, 40, 64), (5001, 300, 72), (9000, 2100, 64), (16384, 256, 136), (2100, 17, 2560)])
def test_linear_ce_backward_of_many_tokens(t, v, d, one):
    """dw has few tiles and a long sum over the tokens, which is split and joined."""
    h, w, y = ce_inputs(t, v, d, 12)
    loss, lse = ce_forward(h, w, y)
    dloss = randn(1 if one else t, seed=9, std=0.3, mean=1.0)
    launched = sbl.launch_count()
    dh, dw = ce_backward(h, w, y, lse, dloss)
    assert sbl.launch_count() - launched == 3
    check_ce_bwd(dh, dw, h, w, y, lse, dloss)
    again = ce_backward(h, w, y, lse, dloss)
    assert same_bits(again[0], dh) and same_bits(again[1], dw)


@pytest.mark.parametrize("t,v,d", [(33, 41, 120), (300, 365, 264), (1, 180, 1120), (2000, 2047, 64)])
def test_linear_ce_backward_of_few_entries_is_as_exact_as_its_outputs(t, v, d):
    """Below 2048 entries the products' operands are exact to 2^-17: what is left is the outputs' one rounding."""
    h, w, y = ce_inputs(t, v, d, 13)
    loss, lse = ce_forward(h, w, y)
    dloss = randn(t, seed=9, std=0.3, mean=1.0)
    dh, dw = ce_backward(h, w, y, lse, dloss)
    p = (h.double() @ w.double().T - lse.double()[:, None]).exp()
    live = y != -100
    p[live] -= torch.nn.functional.one_hot(y[live], v).double()
    dz = p * torch.where(live, dloss.double(), 0.0)[:, None]
    off = 2.0 ** -17 * dz.abs() + p.abs().clamp_max(1.0) * dloss.double().abs()[:, None] * (
        logit_bound(h, w) + 8 * U * lse.double().abs()[:, None] + 2.0 ** -20)
    for got, a, b, n in ((dh, dz, w.double(), v), (dw, dz.T, h.double(), t)):
        want, terms = a @ b, a.abs() @ b.abs()
        tol = (off if got is dh else off.T) @ b.abs() + (n / 8 + 65) * 2 * U * terms
        # the bound of every element: its own rounding, the operands' 2^-17, the logits' errors, the sums
        assert ((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()


def test_linear_ce_backward_of_many_tiles():
    """More output tiles than the launch's table of tiles holds: they are striped over the SMs instead."""
    t, v, d = 256, 40000, 8192
    h, w, y = ce_inputs(t, v, d, 7, std=0.01)
    loss, lse = ce_forward(h, w, y)
    check_ce(loss, lse, h, w, y)
    dloss = randn(t, seed=9, std=0.3, mean=1.0)
    dh, dw = ce_backward(h, w, y, lse, dloss)
    check_ce_bwd(dh, dw, h, w, y, lse, dloss)


def test_linear_ce_backward_rows_without_loss():
    h, w, y = ce_inputs(90, 333, 64, 6)
    loss, lse = ce_forward(h, w, y)
    dloss = torch.ones(90, device="cuda")
    dloss[::7] = float("nan")  # behind ignored targets
    lse[::7] = float("inf")
    dh, dw = ce_backward(h, w, y, lse, dloss)
    assert not dh[::7].any() and torch.isfinite(dh).all() and torch.isfinite(dw).all()
    y[:] = -100
    dh, dw = ce_backward(h, w, y, lse, dloss)
    assert not dh.any() and not dw.any()
    y[2] = 333
    st = status()
    dh, dw = ce_backward(h, w, y, lse, torch.ones(90, device="cuda"), st)
    assert st.item() == sbl.SBL_STATUS_BAD_TARGET and not dh.any() and not dw.any()
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    dw.fill_(3)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    sbl.linear_ce_backward(e, w, y[:0], lse[:0], dloss[:0], 0, 333, 64, e, dw, none)
    assert not dw.any()


@pytest.mark.parametrize("one", [False, True], ids=["each", "one"])
@pytest.mark.parametrize("t,v,d", [(90, 333, 64), (5, 9, 8), (700, 2500, 136), (4100, 9001, 64)])
def test_linear_ce_backward_of_padding_that_holds_anything(t, v, d, one):
    """Rows without loss may hold NaN and infinities: they reach no gradient."""
    h, w, y = ce_inputs(t, v, d, 11)  # every seventh row is ignored
    y[1], y[2] = v, -1                # and two targets are bad
    dead = (y < 0) | (y >= v)
    assert dead.sum() >= 3
    loss, lse = ce_forward(h, w, y)
    dloss = randn(1 if one else t, seed=9, std=0.3, mean=1.0)
    dh, dw = ce_backward(h, w, y, lse, dloss)
    check_ce_bwd(dh, dw, h, w, y, lse, dloss)
    dirty = h.clone()
    dirty[dead] = float("nan")
    dirty[0] = float("inf") if dead[0] else dirty[0]
    loss2, lse2 = ce_forward(dirty, w, y)
    assert same_bits(loss2[~dead], loss[~dead]) and same_bits(lse2[~dead], lse[~dead])
    got = ce_backward(dirty, w, y, lse2, dloss)
    assert same_bits(got[0], dh) and same_bits(got[1], dw)


def test_linear_ce_gradient_against_differences():
    """sum(dloss loss) along random directions, central differences in 64 bits."""
    t, v, d = 20, 300, 64
    h, w, y = ce_inputs(t, v, d, 8)
    loss, lse = ce_forward(h, w, y)
    dloss = randn(t, seed=9, std=0.3, mean=1.0)
    dh, dw = ce_backward(h, w, y, lse, dloss)
    live = y != -100

    def f(hd, wd):
        z = hd @ wd.T
        one = torch.logsumexp(z, 1) - z.gather(1, torch.where(live, y, 0)[:, None])[:, 0]
        return (torch.where(live, one, 0.0) * dloss.double()).sum()

    e = 1e-6
    for seed in range(6):
        a = torch.randn(t, d, generator=gen(seed), device="cuda", dtype=torch.float64)
        b = torch.randn(v, d, generator=gen(50 + seed), device="cuda", dtype=torch.float64)
        want = (f(h.double() + e * a, w.double()) - f(h.double() - e * a, w.double())) / (2 * e)
        # dz and the result are rounded to bf16: 2 x 2^-8 of the magnitudes
        assert abs((dh.double() * a).sum() - want) <= 2.0 ** -7 * (dh.double().abs() * a.abs()).sum() + 1e-4
        want = (f(h.double(), w.double() + e * b) - f(h.double(), w.double() - e * b)) / (2 * e)
        assert abs((dw.double() * b).sum() - want) <= 2.0 ** -7 * (dw.double().abs() * b.abs()).sum() + 1e-4


def test_linear_ce_on_a_side_stream_and_in_graphs():
    t, v, d = 130, 1000, 128
    h, w, y = ce_inputs(t, v, d, 10)
    dloss = torch.ones(t, device="cuda")
    loss, lse = ce_forward(h, w, y)
    dh, dw = ce_backward(h, w, y, lse, dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss2, lse2 = ce_forward(h, w, y)
        dh2, dw2 = ce_backward(h, w, y, lse2, dloss)
    torch.cuda.synchronize()
    assert same_bits(loss, loss2) and same_bits(dh, dh2) and same_bits(dw, dw2)
    # two graphs with a workspace each, replayed in turn on new inputs
    out = []
    for _ in range(2):
        o = {"h": h.clone(), "loss": torch.zeros(t, device="cuda"), "lse": torch.zeros(t, device="cuda"),
             "dh": torch.zeros_like(h), "dw": torch.zeros_like(w),
             "ws": torch.empty(max(sbl.linear_ce_workspace_bytes(t, v, d, b) for b in (False, True)), dtype=torch.uint8, device="cuda")}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sbl.linear_ce_forward(o["h"], w, y, t, v, d, o["loss"], o["lse"], o["ws"])
            sbl.linear_ce_backward(o["h"], w, y, o["lse"], dloss, t, v, d, o["dh"], o["dw"], o["ws"])
        out.append((g, o))
    out[1][1]["h"].neg_()
    for _ in range(2):
        for g, _o in out:
            g.replay()
    torch.cuda.synchronize()
    for _, o in out:
        loss, lse = ce_forward(o["h"], w, y)
        dh, dw = ce_backward(o["h"], w, y, lse, dloss)
        assert same_bits(o["loss"], loss) and same_bits(o["dh"], dh) and same_bits(o["dw"], dw)


# ---------------------------------------------------------------------------
# The operators as they are used: one training step of a small network
# ---------------------------------------------------------------------------
def test_training_step_of_a_small_network():
    """norm -> 2:4 product -> norm (with the residual) -> linear cross entropy, back through all of it, AdamW on
    every weight, and the updated masters prepared again; the gradients against a 64-bit autograd of the same
    network (straight through the quantisers, on the codes the GPU computed)."""
    t, k, v = 96, 320, 700
    x0 = randn(t, k, seed=1, dtype=BF)
    gain1, gain2 = randn(k, seed=2, std=0.1, mean=1.0, dtype=BF), randn(k, seed=3, std=0.1, mean=1.0, dtype=BF)
    w, head = synth.master_weights(k, k, 4, "cuda"), randn(v, k, seed=5, std=0.05, dtype=BF)
    y = torch.randint(0, v, (t,), generator=gen(6), device="cuda")
    y[::9] = -100
    layer = sbl.Layer.allocate(k, k, 2, 4)
    sbl.prepare_weights(layer, w)

    def buf(*shape, dtype=F32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    # forward
    n1, xq, xs, r1 = buf(t, k, dtype=BF), buf(t, k, dtype=torch.int8), buf(t), buf(t)
    sbl.rmsnorm_forward(x0, t, k, EPS, weight=gain1, xn_out=n1, xq_out=xq, xscale_out=xs, rstd_out=r1)
    out = buf(t, k)
    sbl.forward_quantized(layer, xq, xs, t, out)
    h, n2, r2 = buf(t, k, dtype=BF), buf(t, k, dtype=BF), buf(t)
    sbl.rmsnorm_forward(out, t, k, EPS, residual=x0, weight=gain2, h_out=h, xn_out=n2, rstd_out=r2)
    loss, lse = buf(t), buf(t)
    ws = buf(max(sbl.linear_ce_workspace_bytes(t, v, k, b) for b in (False, True)), dtype=torch.uint8)
    sbl.linear_ce_forward(n2, head, y, t, v, k, loss, lse, ws)
    # backward of the mean loss
    live = y != -100
    dloss = (1.0 / live.sum()).float().reshape(1)
    dn2, dhead = buf(t, k, dtype=BF), buf(v, k, dtype=BF)
    sbl.linear_ce_backward(n2, head, y, lse, dloss, t, v, k, dn2, dhead, ws)
    nws = buf(sbl.rmsnorm_backward_workspace_bytes(t, k), dtype=torch.uint8)
    dh, dgain2 = buf(t, k, dtype=BF), buf(k)
    sbl.rmsnorm_backward(h, r2, [dn2], t, k, dh, weight=gain2, dw=dgain2, workspace=nws)
    dn1, dw = buf(t, k, dtype=BF), buf(k, k, dtype=BF)
    sbl.backward(layer, n1, dh, t, dn1, dw)
    dx0, dgain1 = buf(t, k, dtype=BF), buf(k)
    sbl.rmsnorm_backward(x0, r1, [dn1], t, k, dx0, weight=gain1, dres=dh, dw=dgain1, workspace=nws)

    # the same in 64 bits
    _, g = sbl.read_scale(layer)
    weff = layer.section("weff_bf16", k * k * 2).view(BF).view(k, k).double() * g
    leaf = {n: p.double().requires_grad_() for n, p in dict(x0=x0, gain1=gain1, gain2=gain2, head=head).items()}
    wd = w.double().requires_grad_()

    def norm(a, gain):
        return a * (a.square().mean(1, keepdim=True) + EPS).rsqrt() * gain

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, wm):
            ctx.save_for_backward(a)
            return (xq.double() * xs.double()[:, None] / 127) @ weff.T

        @staticmethod
        def backward(ctx, dy):
            return dy @ weff, dy.T @ ctx.saved_tensors[0]

    a = norm(leaf["x0"], leaf["gain1"])
    z = norm(leaf["x0"] + Product.apply(a, wd), leaf["gain2"]) @ leaf["head"].T
    ref = torch.nn.functional.cross_entropy(z, y, ignore_index=-100)
    ref.backward()
    # each value on the way is rounded to bf16 (2^-8 at most): n1, h, n2, dz, dn2, dh, dn1 and the results
    assert abs(loss.sum().item() * dloss.item() - ref.item()) <= 4 * 2.0 ** -8 * ref.item()
    for name, got, want in (("head", dhead, leaf["head"].grad), ("gain2", dgain2, leaf["gain2"].grad), ("w", dw, wd.grad),
                            ("gain1", dgain1, leaf["gain1"].grad), ("x0", dx0, leaf["x0"].grad)):
        assert (got.double() - want).norm() <= 8 * 2.0 ** -8 * want.norm(), name

    # the update, and the next step's preparation from the updated masters
    ts = [sbl.AdamWTensor.allocate(w, dw, bits=8), sbl.AdamWTensor.allocate(head, dhead, bits=32),
          sbl.AdamWTensor.allocate(gain1, dgain1, decay=False), sbl.AdamWTensor.allocate(gain2, dgain2, decay=False)]
    before = [adam_before(p) for p in ts]
    ts_flat = [sbl.AdamWTensor(p.w.view(-1), p.grad.view(-1), p.m, p.v, p.m_scale, p.v_scale, p.master, p.decay) for p in ts]
    sbl.adamw_step(sbl.AdamWTensors(ts), 1, **HYPER)
    for p, b in zip(ts_flat, before):
        check_adam(p, tuple(q.reshape(-1) for q in b), 1)
    sbl.prepare_weights(layer, w)
    assert sbl.read_status(layer)[0] == sbl.SBL_OK
