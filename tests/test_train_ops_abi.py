"""Refusals and host-only functions of the norm, AdamW and linear cross entropy
entry points: no GPU, nothing is enqueued."""
import os
import re

import pytest
import torch

from sparse_linear_layers_bitlinear_b200 import build, sbl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return sbl.lib()


def norm(lib, x=A, res=None, w=None, t=4, k=64, eps=1e-5, flags=0, h=None, xn=A, xhat=None, xq=None, xs=None, rstd=None,
         status=None, reserved=0):
    return lib.sbl_rmsnorm_forward(sbl._RMSNORM_ARGS.pack(*(p or 0 for p in (x, res, w)), t, k, eps, *(
        p or 0 for p in (h, xn, xhat, xq, xs, rstd, status)), flags, reserved), None)


@pytest.mark.parametrize("bad,code", [
    (dict(k=0), sbl.SBL_ERR_SHAPE), (dict(k=12), sbl.SBL_ERR_SHAPE), (dict(k=-8), sbl.SBL_ERR_SHAPE),
    (dict(k=sbl.SBL_NORM_MAX_K + 8), sbl.SBL_ERR_SHAPE), (dict(t=-1), sbl.SBL_ERR_SHAPE),
    (dict(t=(1 << 30) + 1), sbl.SBL_ERR_SHAPE), (dict(x=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(xn=None), sbl.SBL_ERR_INVALID_ARG), (dict(flags=sbl.SBL_NORM_DY_F32), sbl.SBL_ERR_INVALID_ARG),
    (dict(reserved=1), sbl.SBL_ERR_INVALID_ARG), (dict(eps=0.0), sbl.SBL_ERR_INVALID_ARG), (dict(eps=float("nan")), sbl.SBL_ERR_INVALID_ARG),
    (dict(eps=2.0), sbl.SBL_ERR_INVALID_ARG), (dict(x=A + 8), sbl.SBL_ERR_ALIGN), (dict(w=A + 2), sbl.SBL_ERR_ALIGN),
    (dict(rstd=A + 4), sbl.SBL_ERR_ALIGN), (dict(xq=A + 8), sbl.SBL_ERR_ALIGN), (dict(status=A + 2), sbl.SBL_ERR_ALIGN),
])
def test_norm_forward_refusals(lib, bad, code):
    assert norm(lib, **bad) == code


def test_empty_batches_need_nothing(lib):
    assert norm(lib, t=0, x=None, xn=None) == sbl.SBL_OK
    assert ce(lib, t=0, v=5, h=None, w=None, y=None, loss=None, lse=None, ws=None) == sbl.SBL_OK
    assert norm_bwd(lib, t=0, h=None, rstd=None, dys=(None,), dh=None) == sbl.SBL_OK
    p = sbl._ADAMW_PARAMS.pack(1e-3, 0.9, 0.95, 1e-8, 0.1, 1, 0, 0, 0)
    assert lib.sbl_adamw_step(None, 0, p, None, None) == sbl.SBL_OK
    t = (sbl.sbl_adamw_tensor * 1)()
    assert lib.sbl_adamw_step(t, 1, p, None, None) == sbl.SBL_OK  # numel 0


def test_missing_argument_structs(lib):
    for call in (lib.sbl_rmsnorm_forward, lib.sbl_rmsnorm_backward, lib.sbl_linear_ce_forward, lib.sbl_linear_ce_backward):
        assert call(None, None) == sbl.SBL_ERR_INVALID_ARG
    assert lib.sbl_adamw_step(None, 0, None, None, None) == sbl.SBL_ERR_INVALID_ARG


def test_packed_structs_have_the_header_s_layout(tmp_path):
    """Sizes and field offsets of the packed forms against a C compiler's."""
    import struct
    import subprocess

    layouts = {"sbl_rmsnorm_args": (sbl._RMSNORM_ARGS, "x residual weight t k eps h_out xn_out xhat_out xq_out xscale_out "
                                    "rstd_out status_dev flags reserved"),
               "sbl_rmsnorm_backward_args": (sbl._RMSNORM_BACKWARD_ARGS, "h rstd weight dys[0] dys[1] dys[2] dres t k dh dx dw "
                                             "workspace flags dy_count"),
               "sbl_adamw_params": (sbl._ADAMW_PARAMS, "lr beta1 beta2 eps weight_decay step lr_dev step_dev grad_scale_dev"),
               "sbl_linear_ce_args": (sbl._LINEAR_CE_ARGS, "h w targets t v d ignore_index loss lse workspace status_dev"),
               "sbl_linear_ce_backward_args": (sbl._LINEAR_CE_BACKWARD_ARGS, "h w targets lse dloss dloss_stride t v d "
                                               "ignore_index dh dw workspace status_dev")}
    code = '#include <stddef.h>\n#include <stdio.h>\n#include "sbl.h"\nint main(void) {\n'
    for name, (_, fields) in layouts.items():
        code += f'printf("%zu", sizeof({name}));\n'
        for f in fields.split():
            code += f'printf(" %zu", offsetof({name}, {f}));\n'
        code += 'printf("\\n");\n'
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text(code + "return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    for line, (packed, fields) in zip(lines, layouts.values()):
        numbers = [int(x) for x in line.split()]
        assert numbers[0] == packed.size
        codes = "".join(c * int(n or 1) for n, c in re.findall(r"(\d*)([a-zA-Z])", packed.format))
        assert len(codes) == len(fields.split())
        assert numbers[1:] == [struct.calcsize("=" + codes[:i]) for i in range(len(codes))]


def norm_bwd(lib, h=A, rstd=A, w=None, dys=(A,), dres=None, t=4, k=64, flags=0, dh=A, dx=None, dw=None, ws=None,
             count=None):
    d = list(dys) + [None] * (3 - len(dys))
    return lib.sbl_rmsnorm_backward(sbl._RMSNORM_BACKWARD_ARGS.pack(*(p or 0 for p in (h, rstd, w, *d, dres)), t, k, *(
        p or 0 for p in (dh, dx, dw, ws)), flags, len(dys) if count is None else count), None)


@pytest.mark.parametrize("bad,code", [
    (dict(k=20), sbl.SBL_ERR_SHAPE), (dict(t=-1), sbl.SBL_ERR_SHAPE), (dict(count=0), sbl.SBL_ERR_INVALID_ARG),
    (dict(count=4), sbl.SBL_ERR_INVALID_ARG), (dict(dys=(A, None)), sbl.SBL_ERR_INVALID_ARG),
    (dict(dys=(A, A + 4)), sbl.SBL_ERR_ALIGN), (dict(h=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(rstd=None), sbl.SBL_ERR_INVALID_ARG), (dict(dh=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(dw=A), sbl.SBL_ERR_INVALID_ARG), (dict(dw=A + 8, ws=A), sbl.SBL_ERR_ALIGN),
    (dict(dw=A, ws=A + 8), sbl.SBL_ERR_ALIGN), (dict(flags=sbl.SBL_NORM_X_F32), sbl.SBL_ERR_INVALID_ARG),
])
def test_norm_backward_refusals(lib, bad, code):
    assert norm_bwd(lib, **bad) == code


def test_norm_workspace(lib):
    assert sbl.rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert sbl.rmsnorm_backward_workspace_bytes(5, 12) == 0
    assert sbl.rmsnorm_backward_workspace_bytes(3, 64) >= 64 * 4
    assert sbl.rmsnorm_backward_workspace_bytes(1 << 20, 2560) <= 256 * 2560 * 4


def adam(lib, n=8, flags=0, params=None, count=1, twice=False, **over):
    arr = (sbl.sbl_adamw_tensor * 2)()
    for i, c in enumerate(arr):
        off = 0 if twice else 0x1000 * i
        c.w, c.master, c.grad, c.m, c.v = A + off, None, A, A, A
        c.numel, c.flags = n, flags
    for key, value in over.items():
        setattr(arr[0], key, value)
    p = sbl._ADAMW_PARAMS.pack(*(params or (1e-3, 0.9, 0.95, 1e-8, 0.1, 1)), 0, 0, 0)
    return lib.sbl_adamw_step(arr, count, p, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(count=-1), sbl.SBL_ERR_INVALID_ARG), (dict(n=-1), sbl.SBL_ERR_SHAPE), (dict(n=(1 << 40) + 1), sbl.SBL_ERR_SHAPE),
    (dict(flags=8), sbl.SBL_ERR_INVALID_ARG), (dict(reserved=1), sbl.SBL_ERR_INVALID_ARG),
    (dict(w=None), sbl.SBL_ERR_INVALID_ARG), (dict(grad=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(m=None), sbl.SBL_ERR_INVALID_ARG), (dict(v=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(flags=sbl.SBL_ADAMW_STATE_8BIT), sbl.SBL_ERR_INVALID_ARG),
    (dict(w=A + 8), sbl.SBL_ERR_ALIGN), (dict(m=A + 4), sbl.SBL_ERR_ALIGN), (dict(master=A + 4), sbl.SBL_ERR_ALIGN),
    (dict(flags=sbl.SBL_ADAMW_STATE_8BIT, m_scale=A, v_scale=A + 2), sbl.SBL_ERR_ALIGN),
    (dict(count=2, twice=True), sbl.SBL_ERR_INVALID_ARG),
    (dict(params=(1e-3, 1.0, 0.95, 1e-8, 0.1, 1)), sbl.SBL_ERR_INVALID_ARG),
    (dict(params=(1e-3, 0.9, -0.1, 1e-8, 0.1, 1)), sbl.SBL_ERR_INVALID_ARG),
    (dict(params=(float("inf"), 0.9, 0.95, 1e-8, 0.1, 1)), sbl.SBL_ERR_INVALID_ARG),
    (dict(params=(1e-3, 0.9, 0.95, -1.0, 0.1, 1)), sbl.SBL_ERR_INVALID_ARG),
    (dict(params=(1e-3, 0.9, 0.95, 1e-8, 0.1, 0)), sbl.SBL_ERR_INVALID_ARG),
])
def test_adamw_refusals(lib, bad, code):
    assert adam(lib, **bad) == code


def ce(lib, h=A, w=A, y=A, t=4, v=9, d=64, loss=A, lse=A, ws=A):
    return lib.sbl_linear_ce_forward(sbl._LINEAR_CE_ARGS.pack(*(p or 0 for p in (h, w, y)), t, v, d, -100, *(
        p or 0 for p in (loss, lse, ws)), 0), None)


def ce_bwd(lib, h=A, w=A, y=A, lse=A, dloss=A, stride=1, t=4, v=9, d=64, dh=A, dw=A, ws=A):
    return lib.sbl_linear_ce_backward(sbl._LINEAR_CE_BACKWARD_ARGS.pack(*(p or 0 for p in (h, w, y, lse, dloss)), stride, t, v,
                                                                        d, -100, *(p or 0 for p in (dh, dw, ws)), 0), None)


CE_BAD = [
    (dict(d=0), sbl.SBL_ERR_SHAPE), (dict(d=20), sbl.SBL_ERR_SHAPE), (dict(d=131080), sbl.SBL_ERR_SHAPE),
    (dict(v=0), sbl.SBL_ERR_SHAPE), (dict(v=(1 << 22) + 1), sbl.SBL_ERR_SHAPE), (dict(t=-1), sbl.SBL_ERR_SHAPE),
    (dict(t=(1 << 22) + 1), sbl.SBL_ERR_SHAPE), (dict(h=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(w=None), sbl.SBL_ERR_INVALID_ARG), (dict(y=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(ws=None), sbl.SBL_ERR_INVALID_ARG), (dict(h=A + 8), sbl.SBL_ERR_ALIGN), (dict(w=A + 8), sbl.SBL_ERR_ALIGN),
    (dict(ws=A + 16), sbl.SBL_ERR_ALIGN)]


@pytest.mark.parametrize("bad,code", CE_BAD + [(dict(loss=None), sbl.SBL_ERR_INVALID_ARG),
                                               (dict(lse=None), sbl.SBL_ERR_INVALID_ARG)])
def test_linear_ce_forward_refusals(lib, bad, code):
    assert ce(lib, **bad) == code


@pytest.mark.parametrize("bad,code", CE_BAD + [
    (dict(stride=2), sbl.SBL_ERR_INVALID_ARG), (dict(dh=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(dw=None), sbl.SBL_ERR_INVALID_ARG), (dict(lse=None), sbl.SBL_ERR_INVALID_ARG),
    (dict(dloss=None), sbl.SBL_ERR_INVALID_ARG), (dict(dh=A + 8), sbl.SBL_ERR_ALIGN),
    (dict(dw=A + 8), sbl.SBL_ERR_ALIGN), (dict(lse=A + 2), sbl.SBL_ERR_ALIGN)])
def test_linear_ce_backward_refusals(lib, bad, code):
    assert ce_bwd(lib, **bad) == code


def test_linear_ce_workspace(lib):
    assert sbl.linear_ce_workspace_bytes(0, 5, 64) == 0
    assert sbl.linear_ce_workspace_bytes(5, 0, 64) == 0
    assert sbl.linear_ce_workspace_bytes(5, 5, 60, True) == 0
    for t, v, d in [(1, 1, 8), (8192, 32768, 2560), (63, 4099, 512), (100000, 1000, 64)]:
        assert 0 < sbl.linear_ce_workspace_bytes(t, v, d) < t * v * 4 + 4096 + 64 * t
        assert sbl.linear_ce_workspace_bytes(t, v, d, True) > 0
    # the backward pass keeps a piece of dz, never all of it
    assert sbl.linear_ce_workspace_bytes(8192, 131072, 2560, True) < 8192 * 131072 * 2 // 8


def test_binding_refuses_before_it_calls():
    """Tensors of the wrong type, length, layout or device raise, with the reason."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(sbl.SblError, match="not on the current CUDA device"):
        sbl.rmsnorm_forward(x, 4, 64, 1e-5, xn_out=x.clone())
    with pytest.raises(sbl.SblError, match="x is on cpu"):
        sbl.rmsnorm_forward(x.half(), 4, 64, 1e-5, xn_out=x.clone())
    with pytest.raises(sbl.SblError, match="4 gradients"):
        sbl.rmsnorm_backward(x, x, [x] * 4, 4, 64, x)
    with pytest.raises(sbl.SblError, match="is missing"):
        sbl.linear_ce_forward(None, x, x, 4, 4, 64, x, x, x)
    with pytest.raises(sbl.SblError, match="w, grad, m or v is missing"):
        sbl.AdamWTensors([sbl.AdamWTensor(x, None, x, x)])
    with pytest.raises(sbl.SblError, match="16 bits"):
        sbl.AdamWTensor.allocate(x, x, bits=16)
