"""ctypes binding of libsbl.so (include/sbl.h).

Argument marshalling only: every step of the operator runs in the CUDA
kernels of libsbl.so.  torch provides device memory and the current stream.
If the library is missing the import fails loudly; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import warnings
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsbl.so")

# sbl_status
SBL_OK = 0
SBL_ERR_INVALID_ARG = 1
SBL_ERR_UNSUPPORTED_NM = 2
SBL_ERR_SHAPE = 3
SBL_ERR_ALIGN = 4
SBL_ERR_CUDA = 5
SBL_ERR_NONFINITE = 6
SBL_ERR_TIMEOUT = 7
SBL_ERR_DEVICE = 8
SBL_ERR_SCRATCH = 9
STATUS_NAMES = {
    0: "SBL_OK", 1: "SBL_ERR_INVALID_ARG", 2: "SBL_ERR_UNSUPPORTED_NM", 3: "SBL_ERR_SHAPE",
    4: "SBL_ERR_ALIGN", 5: "SBL_ERR_CUDA", 6: "SBL_ERR_NONFINITE", 7: "SBL_ERR_TIMEOUT", 8: "SBL_ERR_DEVICE",
    9: "SBL_ERR_SCRATCH",
}
# Fixed scratch of sbl_forward_noalloc (SBL_NOALLOC_SCRATCH_BYTES in include/sbl.h).
NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024
# layer flags
SBL_PACK_GEMV = 1 << 0
SBL_MASK_FROM_QUANT = 1 << 1
SBL_PACK_GEMV_6BIT = 1 << 2
SBL_FUSE_ACT_QUANT = 1 << 3
# backward flags
SBL_GRAD_F32 = 1 << 1
SBL_NO_DX = 1 << 2
SBL_NO_DW = 1 << 3
SBL_MASKED_GRAD = 1 << 4
SBL_DW_QUANT_X = 1 << 5
# device status bits
SBL_STATUS_NONFINITE_W = 1 << 0
SBL_STATUS_NONFINITE_X = 1 << 1
SBL_STATUS_TIMEOUT = 1 << 2
SBL_STATUS_NONFINITE_G = 1 << 3
SBL_STATUS_BAD_TARGET = 1 << 4
# norm operand types
SBL_NORM_X_F32 = 1 << 0
SBL_NORM_STREAM_F32 = 1 << 1
SBL_NORM_W_F32 = 1 << 2
SBL_NORM_DY_F32 = 1 << 3
SBL_NORM_MAX_K = 16384
# AdamW tensor flags
SBL_ADAMW_GRAD_F32 = 1 << 0
SBL_ADAMW_STATE_8BIT = 1 << 1
SBL_ADAMW_NO_DECAY = 1 << 2
SBL_ADAMW_BLOCK = 256


class SblError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}")
        self.code = code


class sbl_layer(ctypes.Structure):
    _fields_ = [
        ("n_out", ctypes.c_int64),
        ("k", ctypes.c_int64),
        ("n", ctypes.c_int32),
        ("m", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("prepared", ctypes.c_void_p),
    ]


class sbl_blob_layout(ctypes.Structure):
    _fields_ = [(name, ctypes.c_uint64) for name in (
        "total_bytes", "header", "mask", "codes", "weff_bf16", "sp_values", "sp_meta", "sp_meta_bytes",
        "gemv", "gamma", "g", "status", "scratch", "gemv_bytes")]


class sbl_adamw_tensor(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("w", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("numel", ctypes.c_int64), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


# The argument structs of the entry points that take one, as packed bytes: a
# call then costs the host less than a ctypes argument for every field.
_RMSNORM_ARGS = struct.Struct("=3Q2qd7Q2I")
_RMSNORM_BACKWARD_ARGS = struct.Struct("=7Q2q4QIi")
_ADAMW_PARAMS = struct.Struct("=5dq3Q")
_LINEAR_CE_ARGS = struct.Struct("=3Q4q4Q")
_LINEAR_CE_BACKWARD_ARGS = struct.Struct("=5Q5q4Q")


# Every entry point of include/sbl.h with its ctypes signature.
_P, _I64, _I32, _U32, _U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64
_LP = ctypes.POINTER(sbl_layer)
SIGNATURES = {
    "sbl_prepared_layout": (_I32, [_I64, _I64, _I32, _I32, _U32, ctypes.POINTER(sbl_blob_layout)]),
    "sbl_prepared_bytes": (ctypes.c_size_t, [_I64, _I64, _I32, _I32, _U32]),
    "sbl_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "sbl_prepare_weights": (_I32, [_LP, _P, _P]),
    "sbl_prepare_weights_grouped": (_I32, [_LP, ctypes.POINTER(_P), _I32, _P]),
    "sbl_forward": (_I32, [_LP, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "sbl_backward": (_I32, [_LP, _P, _P, _I64, _P, _P, _U32, _P]),
    "sbl_backward_ws": (_I32, [_LP, _P, _P, _I64, _P, _P, _U32, _P, _P]),
    "sbl_backward_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _U32]),
    "sbl_forward_noalloc": (_I32, [_LP, _P, _I64, _P, _P, _P]),
    "sbl_read_status": (_I32, [_LP, _P, ctypes.POINTER(ctypes.c_uint32)]),
    "sbl_clear_status": (_I32, [_LP, _P]),
    "sbl_read_scale": (_I32, [_LP, _P, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float)]),
    "sbl_selftest_wait_timeout": (_I32, [_P, _U64, _P]),
    "sbl_selftest_chain_floor": (_I32, [_I32, _P]),
    "sbl_quantize_activations": (_I32, [_P, _I64, _I64, _P, _P, _P, _P]),
    "sbl_selftest_mma_rate": (_I32, [_I32, _I32, _I32, _P, ctypes.POINTER(ctypes.c_int64), _P]),
    "sbl_version": (ctypes.c_char_p, []),
    "sbl_launch_count": (ctypes.c_uint64, []),
    "sbl_forward_uses_gemv": (ctypes.c_int, [_LP, _I64]),
    "sbl_weight_abs_sum": (_I32, [_LP, _P, _P, _P]),
    "sbl_prepare_weights_from_sum": (_I32, [_LP, _P, _P, _I64, _P]),
    "sbl_forward_quantized": (_I32, [_LP, _P, _P, _I64, _P, _P, _P]),
    "sbl_rmsnorm_forward": (_I32, [ctypes.c_char_p, _P]),
    "sbl_rmsnorm_backward": (_I32, [ctypes.c_char_p, _P]),
    "sbl_rmsnorm_backward_workspace_bytes": (ctypes.c_size_t, [_I64, _I64]),
    "sbl_adamw_step": (_I32, [_P, _I32, ctypes.c_char_p, _P, _P]),
    "sbl_linear_ce_forward": (_I32, [ctypes.c_char_p, _P]),
    "sbl_linear_ce_backward": (_I32, [ctypes.c_char_p, _P]),
    "sbl_linear_ce_workspace_bytes": (ctypes.c_size_t, [_I64, _I64, _I64, _I32]),
}

_lib = None


def lib():
    """Load libsbl.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m sparse_linear_layers_bitlinear_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(code: int, what: str):
    if code != SBL_OK:
        raise SblError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def prepared_layout(n_out: int, k: int, n: int, m: int, flags: int = 0) -> sbl_blob_layout:
    out = sbl_blob_layout()
    _check(lib().sbl_prepared_layout(n_out, k, n, m, flags, ctypes.byref(out)), "sbl_prepared_layout")
    return out


def prepared_bytes(n_out: int, k: int, n: int, m: int, flags: int = 0) -> int:
    return int(lib().sbl_prepared_bytes(n_out, k, n, m, flags))


def workspace_bytes(t: int, k: int) -> int:
    return int(lib().sbl_workspace_bytes(t, k))


@dataclass
class Layer:
    """A Sparse-BitLinear layer: shapes, N:M pattern and its prepared device blob."""

    n_out: int
    k: int
    n: int
    m: int
    flags: int
    blob: "object"  # torch.uint8 CUDA tensor

    @classmethod
    def allocate(cls, n_out: int, k: int, n: int, m: int, flags: int = 0, device="cuda"):
        import torch

        nbytes = prepared_bytes(n_out, k, n, m, flags)
        if nbytes == 0:
            prepared_layout(n_out, k, n, m, flags)  # raises with the reason
        blob = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return cls(n_out, k, n, m, flags, blob)

    def c(self) -> sbl_layer:
        return sbl_layer(self.n_out, self.k, self.n, self.m, self.flags, self.blob.data_ptr())

    def layout(self) -> sbl_blob_layout:
        return prepared_layout(self.n_out, self.k, self.n, self.m, self.flags)

    def section(self, name: str, nbytes: int):
        off = getattr(self.layout(), name)
        return self.blob[off:off + nbytes]


def prepare_weights(layer: Layer, w_master, stream=None):
    cl = layer.c()
    _check(lib().sbl_prepare_weights(ctypes.byref(cl), _ptr(w_master), _stream(stream)), "sbl_prepare_weights")


def prepare_weights_grouped(layers, w_masters, stream=None):
    """sbl_prepare_weights_grouped: several layers (same m) prepared in one launch."""
    count = len(layers)
    arr = (sbl_layer * count)(*[L.c() for L in layers])
    ws = (_P * count)(*[_ptr(w) for w in w_masters])
    _check(lib().sbl_prepare_weights_grouped(arr, ws, count, _stream(stream)), "sbl_prepare_weights_grouped")


SBL_SUM_WORDS = 46


def weight_abs_sum(layer: Layer, w_shard, sum_out, stream=None):
    """sbl_weight_abs_sum: this shard's exact sum of |w| as SBL_SUM_WORDS words (int64 CUDA tensor)."""
    cl = layer.c()
    _check(lib().sbl_weight_abs_sum(ctypes.byref(cl), _ptr(w_shard), _ptr(sum_out), _stream(stream)),
           "sbl_weight_abs_sum")


def prepare_weights_from_sum(layer: Layer, w_shard, global_sum, global_numel: int, stream=None):
    """sbl_prepare_weights_from_sum: prepare this shard with the scale of the summed words."""
    cl = layer.c()
    _check(lib().sbl_prepare_weights_from_sum(ctypes.byref(cl), _ptr(w_shard), _ptr(global_sum), global_numel,
                                              _stream(stream)), "sbl_prepare_weights_from_sum")


def allreduce_sum_words(words, group=None):
    """Step 2 of the row-sharded scale: add every rank's sum words, word by
    word (an exact integer all-reduce; the words are below 2^63)."""
    import torch.distributed as dist

    dist.all_reduce(words, op=dist.ReduceOp.SUM, group=group)
    return words


def prepare_weights_row_sharded(layer: Layer, w_shard, global_rows: int, group=None, stream=None):
    """The three steps for this rank's row shard: its exact sum, the exact
    all-reduce of the words, and the preparation with the whole tensor's scale.

    The all-reduce is ordered on torch's current stream (as every collective
    is), so with an explicit ``stream`` the current stream first waits for the
    sum on ``stream``, and ``stream`` then waits for the all-reduce before the
    preparation reads the words.  No host synchronisation."""
    import torch

    words = torch.empty(SBL_SUM_WORDS, dtype=torch.int64, device=w_shard.device)
    weight_abs_sum(layer, w_shard, words, stream)
    cur = torch.cuda.current_stream(w_shard.device) if w_shard.is_cuda else None
    side = stream is not None and cur is not None and stream != cur
    if side:
        cur.wait_stream(stream)
    allreduce_sum_words(words, group)
    if side:
        stream.wait_stream(cur)
        words.record_stream(stream)
    prepare_weights_from_sum(layer, w_shard, words, global_rows * layer.k, stream)
    return words


def forward(layer: Layer, x, t: int, y, xq_out=None, xscale_out=None, acc_debug=None, workspace=None, stream=None):
    cl = layer.c()
    _check(lib().sbl_forward(ctypes.byref(cl), _ptr(x), t, _ptr(y), _ptr(xq_out), _ptr(xscale_out), _ptr(acc_debug),
                             _ptr(workspace), _stream(stream)), "sbl_forward")


def forward_quantized(layer: Layer, xq, xscale, t: int, y, acc_debug=None, stream=None):
    """sbl_forward_quantized: the forward from int8 codes and scales already at hand."""
    cl = layer.c()
    _check(lib().sbl_forward_quantized(ctypes.byref(cl), _ptr(xq), _ptr(xscale), t, _ptr(y), _ptr(acc_debug),
                                       _stream(stream)), "sbl_forward_quantized")


def quantize_activations(x, t: int, k: int, xq, xscale, status, stream=None):
    """sbl_quantize_activations: the forward's activation codes and scales
    alone; `status` is a device int32 tensor that receives the non-finite bit."""
    _check(lib().sbl_quantize_activations(_ptr(x), t, k, _ptr(xq), _ptr(xscale), _ptr(status), _stream(stream)),
           "sbl_quantize_activations")


def forward_noalloc(layer: Layer, x, t: int, y, acc_debug=None, stream=None):
    """sbl_forward_noalloc: the forward pass without any caller-provided scratch,
    for callers that cannot allocate device memory (see include/sbl.h)."""
    cl = layer.c()
    _check(lib().sbl_forward_noalloc(ctypes.byref(cl), _ptr(x), t, _ptr(y), _ptr(acc_debug), _stream(stream)),
           "sbl_forward_noalloc")


def backward(layer: Layer, x, dy, t: int, dx, dw, flags: int = 0, stream=None, workspace=None):
    """sbl_backward, or sbl_backward_ws when a workspace is given (SBL_DW_QUANT_X needs one)."""
    cl = layer.c()
    if workspace is None:
        _check(lib().sbl_backward(ctypes.byref(cl), _ptr(x), _ptr(dy), t, _ptr(dx), _ptr(dw), flags,
                                  _stream(stream)), "sbl_backward")
    else:
        _check(lib().sbl_backward_ws(ctypes.byref(cl), _ptr(x), _ptr(dy), t, _ptr(dx), _ptr(dw), flags,
                                     _ptr(workspace), _stream(stream)), "sbl_backward_ws")


def backward_workspace_bytes(t: int, k: int, flags: int) -> int:
    return int(lib().sbl_backward_workspace_bytes(t, k, flags))


def read_status(layer: Layer, stream=None):
    cl = layer.c()
    bits = ctypes.c_uint32(0)
    code = lib().sbl_read_status(ctypes.byref(cl), _stream(stream), ctypes.byref(bits))
    return code, int(bits.value)


def clear_status(layer: Layer, stream=None):
    cl = layer.c()
    _check(lib().sbl_clear_status(ctypes.byref(cl), _stream(stream)), "sbl_clear_status")


def read_scale(layer: Layer, stream=None):
    cl = layer.c()
    gamma, g = ctypes.c_float(0), ctypes.c_float(0)
    _check(lib().sbl_read_scale(ctypes.byref(cl), _stream(stream), ctypes.byref(gamma), ctypes.byref(g)),
           "sbl_read_scale")
    return gamma.value, g.value


def selftest_wait_timeout(status_dev, limit_ns: int, stream=None):
    _check(lib().sbl_selftest_wait_timeout(_ptr(status_dev), limit_ns, _stream(stream)), "sbl_selftest_wait_timeout")


def selftest_chain_floor(blocks: int, stream=None):
    """One empty kernel launched as the library launches its kernels (the
    per-call floor of a chain of dependent calls)."""
    _check(lib().sbl_selftest_chain_floor(blocks, _stream(stream)), "sbl_selftest_chain_floor")


def selftest_mma_rate(kind: int, stages: int, pairs: int, status, stream=None) -> int:
    """Resident-operand tensor-pipe rate launch of a GEMM stage (kind 0: 2:4
    int8 forward, 1: dense int8 forward, 2: bf16 backward); returns the
    multiply-adds of one pair's stage.  `status` is a device uint32 tensor."""
    macs = ctypes.c_int64(0)
    _check(lib().sbl_selftest_mma_rate(kind, stages, pairs, _ptr(status), ctypes.byref(macs), _stream(stream)),
           "sbl_selftest_mma_rate")
    return int(macs.value)


def version() -> str:
    return lib().sbl_version().decode()


def forward_uses_gemv(layer: Layer, t: int) -> bool:
    """Whether sbl_forward takes the decode kernel over the packed weights for t tokens on this layer."""
    cl = layer.c()
    return bool(lib().sbl_forward_uses_gemv(ctypes.byref(cl), t))


def launch_count() -> int:
    """Kernels the library has launched in this process (sbl_launch_count)."""
    return int(lib().sbl_launch_count())


# ---------------------------------------------------------------------------
# The operators around the products: norm, AdamW, linear cross entropy.  They
# take tensors of several types, so the tensors are checked here (type, length,
# dense layout, device) before their addresses go to the library.
# ---------------------------------------------------------------------------
_types = None  # torch's types, once torch is imported


class _Types:
    def __init__(self):
        import torch

        self.bf16, self.f32 = (torch.bfloat16,), (torch.float32,)
        self.float = (torch.bfloat16, torch.float32)
        self.i8, self.u8, self.i32, self.i64 = (torch.int8,), (torch.uint8,), (torch.int32,), (torch.int64,)
        self.code8 = (torch.float8_e4m3fn, torch.uint8)
        # the current device and the raw handle of its current stream without the objects around them: a call's
        # cost on the host is most of a small call's time
        self.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _torch_types() -> _Types:
    global _types
    if _types is None:
        _types = _Types()
    return _types


def _device(T: _Types, what: str, name: str, t) -> int:
    """The device of a call: that of its first tensor, which has to be the current one."""
    if t is None:
        raise SblError(SBL_ERR_INVALID_ARG, f"{what}: {name} is missing")
    dev = t.get_device()
    if dev < 0 or dev != T.current_device():
        raise SblError(SBL_ERR_DEVICE, f"{what}: {name} is on {t.device}, not on the current CUDA device")
    return dev


def _addr(what: str, name: str, t, dtypes, numel: int, dev: int):
    """The address of tensor `t` after its checks; 0 for None (the library refuses a NULL it needs)."""
    if t is None:
        return 0
    if t.dtype in dtypes and t.get_device() == dev and t.is_contiguous() and t.numel() == numel:
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise SblError(SBL_ERR_INVALID_ARG, f"{what}: {name} is {t.dtype}, not one of {dtypes}")
    if t.get_device() != dev:
        raise SblError(SBL_ERR_DEVICE, f"{what}: {name} is on {t.device}, the call on CUDA device {dev}")
    if not t.is_contiguous():
        raise SblError(SBL_ERR_SHAPE, f"{what}: {name} is not dense")
    raise SblError(SBL_ERR_SHAPE, f"{what}: {name} has {t.numel()} elements, not {numel}")


def _room(T: _Types, what: str, t, nbytes: int, dev: int):
    """The address of a uint8 workspace of `nbytes` or more."""
    return 0 if t is None else _addr(what, "workspace", t, T.u8, max(t.numel(), nbytes), dev)


def _raw_stream(T: _Types, stream, dev: int):
    if stream is not None:
        return stream.cuda_stream
    return T.raw_stream(dev) if T.raw_stream is not None else _stream().value


def rmsnorm_forward(x, t: int, k: int, eps: float, residual=None, weight=None, h_out=None, xn_out=None, xhat_out=None,
                    xq_out=None, xscale_out=None, rstd_out=None, status=None, stream=None):
    """sbl_rmsnorm_forward: h = x + residual, its root-mean-square norm (bf16
    ``xn_out``) and the norm's int8 codes and scales for ``forward_quantized``
    (``xq_out``, ``xscale_out``; ``xhat_out``: the values they stand for).
    x, the stream (residual, h_out) and weight are bf16 or fp32 each; without a
    residual h_out has x's type.  ``status``: a device int32 tensor or None."""
    T, me, n = _torch_types(), "sbl_rmsnorm_forward", t * k
    dev = _device(T, me, "x", x)
    xp = _addr(me, "x", x, T.float, n, dev)
    stream_type = T.f32 if (x if residual is None else residual).dtype in T.f32 else T.bf16
    flags = ((SBL_NORM_X_F32 if x.dtype in T.f32 else 0) | (SBL_NORM_STREAM_F32 if stream_type is T.f32 else 0)
             | (SBL_NORM_W_F32 if weight is not None and weight.dtype in T.f32 else 0))
    code = lib().sbl_rmsnorm_forward(_RMSNORM_ARGS.pack(
        xp, _addr(me, "residual", residual, stream_type, n, dev), _addr(me, "weight", weight, T.float, k, dev),
        t, k, eps, _addr(me, "h_out", h_out, stream_type, n, dev), _addr(me, "xn_out", xn_out, T.bf16, n, dev),
        _addr(me, "xhat_out", xhat_out, T.bf16, n, dev), _addr(me, "xq_out", xq_out, T.i8, n, dev),
        _addr(me, "xscale_out", xscale_out, T.f32, t, dev), _addr(me, "rstd_out", rstd_out, T.f32, t, dev),
        _addr(me, "status", status, T.i32, 1, dev), flags, 0), _raw_stream(T, stream, dev))
    if code:
        raise SblError(code, me)


def rmsnorm_backward_workspace_bytes(t: int, k: int) -> int:
    return int(lib().sbl_rmsnorm_backward_workspace_bytes(t, k))


def rmsnorm_backward(h, rstd, dys, t: int, k: int, dh, weight=None, dres=None, dx=None, dw=None, workspace=None,
                     stream=None):
    """sbl_rmsnorm_backward: the gradient dh of h (and so of x and of the
    residual) from ``dys`` (one to three gradients of the normalised rows, which
    are added) and ``dres`` (the residual stream's own gradient or None); dx: a
    bf16 copy of dh or None; dw: fp32 gradient of the weight or None (it needs
    ``workspace``, a uint8 tensor of rmsnorm_backward_workspace_bytes)."""
    T, me, n = _torch_types(), "sbl_rmsnorm_backward", t * k
    if not 1 <= len(dys) <= 3:
        raise SblError(SBL_ERR_INVALID_ARG, f"{me}: {len(dys)} gradients, not 1 to 3")
    dev = _device(T, me, "h", h)
    hp, stream_type = _addr(me, "h", h, T.float, n, dev), (h.dtype,)
    _device(T, me, "dys", dys[0])
    dy_type = (dys[0].dtype,)
    flags = ((SBL_NORM_STREAM_F32 if stream_type == T.f32 else 0) | (SBL_NORM_DY_F32 if dy_type == T.f32 else 0)
             | (SBL_NORM_W_F32 if weight is not None and weight.dtype in T.f32 else 0))
    if dy_type[0] not in T.float:
        dy_type = T.float
    dyp = [_addr(me, "dys", d, dy_type, n, dev) for d in dys] + [0] * (3 - len(dys))
    ws = _room(T, me, workspace, rmsnorm_backward_workspace_bytes(t, k), dev) if dw is not None else 0
    code = lib().sbl_rmsnorm_backward(_RMSNORM_BACKWARD_ARGS.pack(
        hp, _addr(me, "rstd", rstd, T.f32, t, dev), _addr(me, "weight", weight, T.float, k, dev), *dyp,
        _addr(me, "dres", dres, stream_type, n, dev), t, k, _addr(me, "dh", dh, stream_type, n, dev),
        _addr(me, "dx", dx, T.bf16, n, dev), _addr(me, "dw", dw, T.f32, k, dev), ws, flags, len(dys)),
        _raw_stream(T, stream, dev))
    if code:
        raise SblError(code, me)


@dataclass
class AdamWTensor:
    """One tensor of an AdamW step: bf16 weights ``w``, bf16 or fp32 ``grad``,
    states ``m`` and ``v`` (fp32, or float8_e4m3fn / uint8 with the fp32 scales
    ``m_scale`` and ``v_scale``, one per 256 elements), optional fp32 ``master``."""

    w: "object"
    grad: "object"
    m: "object"
    v: "object"
    m_scale: "object" = None
    v_scale: "object" = None
    master: "object" = None
    decay: bool = True

    @classmethod
    def allocate(cls, w, grad, bits: int = 32, master: bool = True, decay: bool = True):
        """Zeroed states for ``w`` (and an fp32 copy of it with ``master``)."""
        import torch

        n = w.numel()
        if bits not in (8, 32):
            raise SblError(SBL_ERR_INVALID_ARG, f"sbl.AdamWTensor: states of {bits} bits, not 8 or 32")
        dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
        blocks = (n + SBL_ADAMW_BLOCK - 1) // SBL_ADAMW_BLOCK
        m, v = (torch.zeros(n, dtype=dt, device=w.device) for _ in range(2))
        ms, vs = (torch.zeros(blocks, dtype=torch.float32, device=w.device) if bits == 8 else None for _ in range(2))
        return cls(w, grad, m, v, ms, vs, w.detach().float().reshape(-1) if master else None, decay)


class AdamWTensors:
    """The tensors of ``adamw_step``, checked once; keeps them alive.  Their
    addresses are taken here: a field of an AdamWTensor that is set later, or a
    tensor whose storage moves, is not seen.  Gradients that are allocated anew
    each step come in by ``set_grads``; for other tensors build a new one."""

    def __init__(self, tensors):
        T, me = _torch_types(), "sbl.AdamWTensors"
        self.tensors = list(tensors)
        self.count = len(self.tensors)
        self.array = (sbl_adamw_tensor * max(self.count, 1))()
        self.device = -1
        self.eight = False  # whether a tensor holds 8-bit states
        updated, grads = [], []
        for c, p in zip(self.array, self.tensors):
            if p.w is None or p.grad is None or p.m is None or p.v is None:
                raise SblError(SBL_ERR_INVALID_ARG, f"{me}: w, grad, m or v is missing")
            dev = self.device = _device(T, me, "w", p.w)
            n = p.w.numel()
            c.numel = n
            eight = p.m.dtype not in T.f32
            c.flags = ((SBL_ADAMW_GRAD_F32 if p.grad.dtype in T.f32 else 0) | (SBL_ADAMW_STATE_8BIT if eight else 0)
                       | (0 if p.decay else SBL_ADAMW_NO_DECAY))
            state = T.code8 if eight else T.f32
            c.w = w = _addr(me, "w", p.w, T.bf16, n, dev)
            c.grad = grad = _addr(me, "grad", p.grad, T.float, n, dev)
            c.m = m = _addr(me, "m", p.m, state, n, dev)
            c.v = v = _addr(me, "v", p.v, state, n, dev)
            c.master = master = _addr(me, "master", p.master, T.f32, n, dev)
            updated += (w, m, v, master)
            grads.append(grad)
            self.eight |= eight
            if eight:
                blocks = (n + SBL_ADAMW_BLOCK - 1) // SBL_ADAMW_BLOCK
                if p.m_scale is None or p.v_scale is None:
                    raise SblError(SBL_ERR_INVALID_ARG, f"{me}: 8-bit states without m_scale or v_scale")
                c.m_scale = ms = _addr(me, "m_scale", p.m_scale, T.f32, blocks, dev)
                c.v_scale = vs = _addr(me, "v_scale", p.v_scale, T.f32, blocks, dev)
                updated += (ms, vs)
        updated = [a for a in updated if a]  # no master, or an empty tensor: 0
        self.updated = set(updated)
        if len(self.updated) != len(updated) or not self.updated.isdisjoint(grads):
            raise SblError(SBL_ERR_INVALID_ARG, f"{me}: a tensor that is updated stands in two places")

    def set_grads(self, grads):
        """Other gradients from the next step on, one for each tensor in their order (bf16 or fp32, each of its
        tensor's length); nothing changes if one of them is refused.  A captured graph goes on reading those it was
        captured with: keep them for it."""
        T, me = _torch_types(), "sbl.AdamWTensors.set_grads"
        grads = list(grads)
        if len(grads) != self.count:
            raise SblError(SBL_ERR_INVALID_ARG, f"{me}: {len(grads)} gradients for {self.count} tensors")
        if any(g is None for g in grads):
            raise SblError(SBL_ERR_INVALID_ARG, f"{me}: a gradient is missing")
        at = [_addr(me, "grad", g, T.float, c.numel, self.device) for c, g in zip(self.array, grads)]
        if any(a % 16 for a in at):
            raise SblError(SBL_ERR_ALIGN, f"{me}: a gradient is not 16-byte aligned")
        if not self.updated.isdisjoint(at):
            raise SblError(SBL_ERR_INVALID_ARG, f"{me}: a gradient is a tensor that is updated")
        for c, p, g, a in zip(self.array, self.tensors, grads, at):
            p.grad, c.grad = g, a
            c.flags = c.flags & ~SBL_ADAMW_GRAD_F32 | (SBL_ADAMW_GRAD_F32 if g.dtype in T.f32 else 0)


def adamw_step(tensors: AdamWTensors, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.95,
               eps: float = 1e-8, weight_decay: float = 0.0, lr_dev=None, step_dev=None, grad_scale_dev=None,
               status=None, stream=None):
    """sbl_adamw_step: one step (the first is ``step`` 1) on every tensor.
    ``lr_dev`` (fp32), ``step_dev`` (int64) and ``grad_scale_dev`` (fp32) are
    device scalars that a captured graph reads at each replay, or None.  With
    8-bit states a ``beta2`` above 0.99 warns: nearest rounding then keeps
    nearly every second moment where it is (see sbl_adamw_step)."""
    T, me = _torch_types(), "sbl_adamw_step"
    if tensors.count == 0:
        return
    dev = tensors.device
    if dev != T.current_device():
        raise SblError(SBL_ERR_DEVICE, f"{me}: the tensors are not on the current CUDA device")
    if tensors.eight and beta2 > 0.99:
        warnings.warn(f"{me}: 8-bit second moments hardly move with beta2 = {beta2}; take 0.95 or less", stacklevel=2)
    params = _ADAMW_PARAMS.pack(lr, beta1, beta2, eps, weight_decay, step, _addr(me, "lr_dev", lr_dev, T.f32, 1, dev),
                                _addr(me, "step_dev", step_dev, T.i64, 1, dev),
                                _addr(me, "grad_scale_dev", grad_scale_dev, T.f32, 1, dev))
    code = lib().sbl_adamw_step(tensors.array, tensors.count, params,
                                _addr(me, "status", status, T.i32, 1, dev), _raw_stream(T, stream, dev))
    if code:
        raise SblError(code, me)


def linear_ce_workspace_bytes(t: int, v: int, d: int, backward: bool = False) -> int:
    return int(lib().sbl_linear_ce_workspace_bytes(t, v, d, 1 if backward else 0))


def linear_ce_forward(h, w, targets, t: int, v: int, d: int, loss, lse, workspace, ignore_index: int = -100,
                      status=None, stream=None):
    """sbl_linear_ce_forward: loss[i] = log sum exp(h[i] w^T) - (h[i] w^T)[targets[i]]
    and lse, the logits never in memory.  h: bf16 [t, d], w: bf16 [v, d],
    targets: int64 [t], workspace: uint8, linear_ce_workspace_bytes(t, v, d)."""
    T, me = _torch_types(), "sbl_linear_ce_forward"
    dev = _device(T, me, "h", h)
    code = lib().sbl_linear_ce_forward(_LINEAR_CE_ARGS.pack(
        _addr(me, "h", h, T.bf16, t * d, dev), _addr(me, "w", w, T.bf16, v * d, dev),
        _addr(me, "targets", targets, T.i64, t, dev), t, v, d, ignore_index, _addr(me, "loss", loss, T.f32, t, dev),
        _addr(me, "lse", lse, T.f32, t, dev), _room(T, me, workspace, linear_ce_workspace_bytes(t, v, d), dev),
        _addr(me, "status", status, T.i32, 1, dev)), _raw_stream(T, stream, dev))
    if code:
        raise SblError(code, me)


def linear_ce_backward(h, w, targets, lse, dloss, t: int, v: int, d: int, dh, dw, workspace,
                       ignore_index: int = -100, status=None, stream=None):
    """sbl_linear_ce_backward: dh (bf16 [t, d]) and dw (bf16 [v, d]) from the
    forward's lse and ``dloss``, fp32 of t elements (each loss's gradient) or of
    one (the same for all).  workspace: linear_ce_workspace_bytes(t, v, d, True)."""
    T, me = _torch_types(), "sbl_linear_ce_backward"
    dev = _device(T, me, "h", h)
    one = dloss is not None and dloss.numel() == 1
    code = lib().sbl_linear_ce_backward(_LINEAR_CE_BACKWARD_ARGS.pack(
        _addr(me, "h", h, T.bf16, t * d, dev), _addr(me, "w", w, T.bf16, v * d, dev),
        _addr(me, "targets", targets, T.i64, t, dev), _addr(me, "lse", lse, T.f32, t, dev),
        _addr(me, "dloss", dloss, T.f32, 1 if one else t, dev), 0 if one else 1, t, v, d, ignore_index,
        _addr(me, "dh", dh, T.bf16, t * d, dev), _addr(me, "dw", dw, T.bf16, v * d, dev),
        _room(T, me, workspace, linear_ce_workspace_bytes(t, v, d, True), dev),
        _addr(me, "status", status, T.i32, 1, dev)), _raw_stream(T, stream, dev))
    if code:
        raise SblError(code, me)


class SparseBitLinear:
    """Convenience wrapper: one layer, its blob and its forward/backward buffers.

    All arithmetic happens in libsbl.so; this class only allocates torch
    tensors and calls the C ABI.
    """

    def __init__(self, n_out: int, k: int, n: int = 2, m: int = 4, flags: int = 0, device="cuda"):
        self.layer = Layer.allocate(n_out, k, n, m, flags, device)
        self.device = device

    def prepare(self, w_master):
        prepare_weights(self.layer, w_master)

    def forward(self, x, acc_debug: bool = False):
        import torch

        t = x.shape[0]
        y = torch.empty((t, self.layer.n_out), dtype=torch.float32, device=self.device)
        xq = torch.empty((t, self.layer.k), dtype=torch.int8, device=self.device)
        ap = torch.empty((max(t, 1),), dtype=torch.float32, device=self.device)
        acc = torch.empty((t, self.layer.n_out), dtype=torch.int32, device=self.device) if acc_debug else None
        forward(self.layer, x, t, y, xq, ap, acc)
        return y, xq, ap[:t], acc

    def backward(self, x, dy, f32: bool = False):
        import torch

        t = dy.shape[0]
        dt = torch.float32 if f32 else torch.bfloat16
        dx = torch.empty((t, self.layer.k), dtype=dt, device=self.device)
        dw = torch.empty((self.layer.n_out, self.layer.k), dtype=dt, device=self.device)
        backward(self.layer, x, dy, t, dx, dw, SBL_GRAD_F32 if f32 else 0)
        return dx, dw
