"""Python binding of libfp8q (the block-scaled FP8 linear layer for B200, sm_100a).

Argument marshalling only: each function checks dtypes/shapes, allocates nothing
unless asked to (the ``*_alloc`` helpers), and calls the C entry point of the same
name with device pointers and the current CUDA stream. Every step of the path runs
in libfp8q's kernels; there is no CPU or PyTorch fallback. If libfp8q.so is missing
or stale the import fails loudly: build it with ``python fp8_block_scaled_08_b200/build.py``.

The operations follow "Resumen Técnico: Jet-RL" (gist.science, paper 2601.14243),
section "Esquema de Cuantización"; see include/fp8q.h for layouts and semantics.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8q.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libfp8q.so is not built (%s); run `python fp8_block_scaled_08_b200/build.py`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

FP8Q_OK = 0
FP8Q_ERR_NULL = 1
FP8Q_ERR_SHAPE = 2
FP8Q_ERR_ALIGN = 3
FP8Q_ERR_CUDA = 4
FP8Q_ERR_TIMEOUT = 5
FP8Q_ERR_UNSUPPORTED = 6
FP8Q_ERR_OFFSETS = 7

_P = ctypes.c_void_p
_I = ctypes.c_int64
_F = ctypes.c_float

_SIGS = {
    "fp8q_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "fp8q_version": ([], ctypes.c_int),
    "fp8q_last_error_message": ([], ctypes.c_char_p),
    "fp8q_device_error": ([_P, ctypes.c_int], ctypes.c_int),
    "fp8q_last_device_error": ([_P], ctypes.c_int),
    "fp8q_quant_act_1x128": ([_P, _I, _I, _I, _P, _P, _I, _P], ctypes.c_int),
    "fp8q_quant_weight_128x128": ([_P, _I, _I, _I, _P, _P, _P, _P], ctypes.c_int),
    "fp8q_rmsnorm_quant": ([_P, _P, _I, _I, _I, _F, _P, _P, _I, _P], ctypes.c_int),
    "fp8q_swiglu_quant": ([_P, _I, _I, _I, _P, _P, _I, _P], ctypes.c_int),
    "fp8q_transpose_quant_bf16": ([_P, _I, _I, _I, _P, _P, _I, _P, _P, _P], ctypes.c_int),
    "fp8q_transpose_quant_fp8": ([_P, _P, _I, _I, _I, _P, _P, _P], ctypes.c_int),
    "fp8q_rmsnorm_quant_dual": ([_P, _P, _I, _I, _I, _F, _P, _P, _I, _P, _P, _P, _P],
                                ctypes.c_int),
    "fp8q_swiglu_quant_dual": ([_P, _I, _I, _I, _P, _P, _I, _P, _P, _P], ctypes.c_int),
    "fp8q_swiglu_bwd_quant_dual": ([_P, _P, _I, _I, _P, _P, _P, _I, _P, _P, _P], ctypes.c_int),
    "fp8q_rmsnorm_bwd_workspace_bytes": ([_I, _I], ctypes.c_int64),
    "fp8q_rmsnorm_bwd_quant_dual": ([_P, _P, _P, _P, _I, _I, _F, _P, _P, _P, _I, _P, _P, _P,
                                     _P, _I, _P], ctypes.c_int),
    "fp8q_linear_fwd": ([_P, _P, _I, _P, _P, _I, _I, _I, _P, _I, _P], ctypes.c_int),
    "fp8q_linear_fwd_splitk_workspace": ([_I, _I, _I], ctypes.c_int64),
    "fp8q_linear_fwd_splitk_counter_bytes": ([_I, _I], ctypes.c_int64),
    "fp8q_linear_fwd_splitk": ([_P, _P, _I, _P, _P, _I, _I, _I, _P, _I, _P, _I, _P],
                               ctypes.c_int),
    "fp8q_linear_fwd_splitk_noalloc": ([_P, _P, _I, _P, _P, _I, _I, _I, _P, _I, _P],
                                       ctypes.c_int),
    "fp8q_linear_dgrad": ([_P, _P, _I, _P, _P, _I, _I, _I, _P, _I, _P], ctypes.c_int),
    "fp8q_linear_wgrad": ([_P, _P, _P, _P, _I, _I, _I, _P, _I, _P], ctypes.c_int),
    "fp8q_linear_wgrad_acc_f32": ([_P, _P, _P, _P, _I, _I, _I, _P, _I, _P], ctypes.c_int),
    "fp8q_add_rmsnorm_quant": ([_P, _P, _P, _I, _I, _I, _I, _F, _P, _I, _P, _P, _I, _P],
                               ctypes.c_int),
    "fp8q_grouped_padded_rows": ([_I, _I], ctypes.c_int64),
    "fp8q_grouped_linear_fwd": ([_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P],
                                ctypes.c_int),
    "fp8q_grouped_linear_dgrad": ([_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P],
                                  ctypes.c_int),
    "fp8q_grouped_linear_wgrad": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P],
                                  ctypes.c_int),
    "fp8q_grouped_transpose_quant_bf16": ([_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _I, _P],
                                          ctypes.c_int),
    "fp8q_grouped_transpose_quant_fp8": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P],
                                         ctypes.c_int),
    "fp8q_debug_wait_timeout": ([_I, _P], ctypes.c_int),
}
for _name, (_args, _res) in _SIGS.items():
    try:
        _fn = getattr(_lib, _name)
    except AttributeError as _e:
        raise ImportError("libfp8q.so is stale (no %s); rebuild it with "
                          "`python fp8_block_scaled_08_b200/build.py`" % _name) from _e
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)


class Fp8qError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if status in (FP8Q_ERR_CUDA, FP8Q_ERR_UNSUPPORTED):
            detail = " [%s]" % last_error_message()
        super().__init__("%s: %s%s" % (where, status_string(status), detail))


def status_string(status: int) -> str:
    return _lib.fp8q_status_string(int(status)).decode()


def last_error_message() -> str:
    return _lib.fp8q_last_error_message().decode()


def version() -> int:
    return int(_lib.fp8q_version())


def _check(status: int, where: str) -> None:
    if status != FP8Q_OK:
        raise Fp8qError(status, where)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("libfp8q takes CUDA tensors (device pointers)")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _want(t, dtype, ndim, name):
    if t.dtype != dtype or t.dim() != ndim:
        raise ValueError("%s must be a %d-D %s tensor, got %s %s" % (
            name, ndim, dtype, tuple(t.shape), t.dtype))


def _rows_dense(t, name):
    if t.stride(-1) != 1:
        raise ValueError("%s must have unit column stride" % name)
    return t.stride(0)


def _dense(t, name):
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _groups(n: int) -> int:
    """Number of 128-wide groups covering n elements."""
    return (int(n) + 127) // 128


def _shape(t, shape, dtype, name):
    """Operand `name` must be a `dtype` tensor of exactly `shape` (checked before any
    pointer reaches the C side, whose tensor maps and stores trust these extents)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype or tuple(t.shape) != tuple(int(d) for d in shape):
        raise ValueError("%s must be a %s tensor of shape %s, got %s %s" % (
            name, dtype, tuple(int(d) for d in shape), tuple(t.shape), t.dtype))


def _scales_1x128(s, groups, rows, name):
    """1x128 scale array: fp32 [groups, lds] with lds >= rows (a multiple of 4 is
    checked by the library)."""
    if not isinstance(s, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if s.dtype != torch.float32 or s.dim() != 2 or s.shape[0] != groups or s.shape[1] < rows:
        raise ValueError("%s must be a float32 tensor [%d, >=%d], got %s %s" % (
            name, groups, rows, tuple(s.shape), s.dtype))


def lds_for(m: int) -> int:
    """Smallest legal leading dimension of a 1x128 scale array for M rows."""
    return (max(m, 1) + 3) // 4 * 4


# --------------------------------------------------------------------------
# Raw entry points (caller-owned outputs)
# --------------------------------------------------------------------------

def device_error(stream=None, clear: bool = True) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(_lib.fp8q_device_error(_stream(stream), 1 if clear else 0))


def quant_act_1x128(x, q, s, stream=None):
    """a1: x BF16 [M,K] -> q uint8 [M,K], s float32 [K/128, lds]."""
    _want(x, torch.bfloat16, 2, "x"); _want(q, torch.uint8, 2, "q"); _want(s, torch.float32, 2, "s")
    _dense(q, "q"); _dense(s, "s")
    M, K = x.shape
    _shape(q, (M, K), torch.uint8, "q")
    _scales_1x128(s, _groups(K), M, "s")
    _check(_lib.fp8q_quant_act_1x128(_ptr(x), M, K, _rows_dense(x, "x"), _ptr(q), _ptr(s),
                                     s.shape[1], _stream(stream)), "fp8q_quant_act_1x128")


def quant_weight_128x128(w, q, s, qT=None, stream=None):
    """a2: w BF16 [N,K] -> q [N,K], s [N/128,K/128], optional qT [K,N]."""
    _want(w, torch.bfloat16, 2, "w"); _want(q, torch.uint8, 2, "q"); _want(s, torch.float32, 2, "s")
    _dense(q, "q"); _dense(s, "s")
    if qT is not None:
        _want(qT, torch.uint8, 2, "qT"); _dense(qT, "qT")
    N, K = w.shape
    _shape(q, (N, K), torch.uint8, "q")
    _shape(s, (_groups(N), _groups(K)), torch.float32, "s")
    if qT is not None:
        _shape(qT, (K, N), torch.uint8, "qT")
    _check(_lib.fp8q_quant_weight_128x128(_ptr(w), N, K, _rows_dense(w, "w"), _ptr(q), _ptr(s),
                                          _ptr(qT), _stream(stream)), "fp8q_quant_weight_128x128")


def rmsnorm_quant(x, gamma, eps, q, s, stream=None):
    """a3: RMSNorm(x)*gamma rounded to BF16, then 1x128 quantization."""
    _want(x, torch.bfloat16, 2, "x"); _want(gamma, torch.bfloat16, 1, "gamma")
    _want(q, torch.uint8, 2, "q"); _want(s, torch.float32, 2, "s")
    _dense(gamma, "gamma"); _dense(q, "q"); _dense(s, "s")
    M, H = x.shape
    _shape(gamma, (H,), torch.bfloat16, "gamma")
    _shape(q, (M, H), torch.uint8, "q")
    _scales_1x128(s, _groups(H), M, "s")
    _check(_lib.fp8q_rmsnorm_quant(_ptr(x), _ptr(gamma), M, H, _rows_dense(x, "x"), float(eps),
                                   _ptr(q), _ptr(s), s.shape[1], _stream(stream)),
           "fp8q_rmsnorm_quant")


def swiglu_quant(gu, q, s, stream=None):
    """a4: gu BF16 [M,2I] (gate | up) -> SwiGLU BF16 -> 1x128 quantization."""
    _want(gu, torch.bfloat16, 2, "gu"); _want(q, torch.uint8, 2, "q"); _want(s, torch.float32, 2, "s")
    _dense(q, "q"); _dense(s, "s")
    M, I2 = gu.shape
    if I2 % 2:
        raise ValueError("gu must be [M, 2I] (gate | up), got %s" % (tuple(gu.shape),))
    _shape(q, (M, I2 // 2), torch.uint8, "q")
    _scales_1x128(s, _groups(I2 // 2), M, "s")
    _check(_lib.fp8q_swiglu_quant(_ptr(gu), M, I2 // 2, _rows_dense(gu, "gu"), _ptr(q), _ptr(s),
                                  s.shape[1], _stream(stream)), "fp8q_swiglu_quant")


def transpose_quant_bf16(dy, q_row, s_row, q_colT, s_col, stream=None):
    """a6: dY BF16 [M,N] -> row-wise (q_row [M,N], s_row [N/128,lds]) and column-wise
    transposed (q_colT [N,M], s_col [M/128,N]). q_row/s_row may be None."""
    _want(dy, torch.bfloat16, 2, "dy")
    _want(q_colT, torch.uint8, 2, "q_colT"); _want(s_col, torch.float32, 2, "s_col")
    _dense(q_colT, "q_colT"); _dense(s_col, "s_col")
    lds_row = 0
    if q_row is not None:
        _want(q_row, torch.uint8, 2, "q_row"); _want(s_row, torch.float32, 2, "s_row")
        _dense(q_row, "q_row"); _dense(s_row, "s_row")
        lds_row = s_row.shape[1]
    M, N = dy.shape
    if q_row is not None:
        _shape(q_row, (M, N), torch.uint8, "q_row")
        _scales_1x128(s_row, _groups(N), M, "s_row")
    _shape(q_colT, (N, M), torch.uint8, "q_colT")
    _shape(s_col, (_groups(M), N), torch.float32, "s_col")
    _check(_lib.fp8q_transpose_quant_bf16(_ptr(dy), M, N, _rows_dense(dy, "dy"), _ptr(q_row),
                                          _ptr(s_row), lds_row, _ptr(q_colT), _ptr(s_col),
                                          _stream(stream)), "fp8q_transpose_quant_bf16")


def transpose_quant_fp8(q, s, qT, sT, stream=None):
    """a8: saved FP8 (q [M,K], s [K/128,lds]) -> 128x1 requantized transposed (qT [K,M],
    sT [M/128,K])."""
    _want(q, torch.uint8, 2, "q"); _want(s, torch.float32, 2, "s")
    _want(qT, torch.uint8, 2, "qT"); _want(sT, torch.float32, 2, "sT")
    for t, n in ((q, "q"), (s, "s"), (qT, "qT"), (sT, "sT")):
        _dense(t, n)
    M, K = q.shape
    _scales_1x128(s, _groups(K), M, "s")
    _shape(qT, (K, M), torch.uint8, "qT")
    _shape(sT, (_groups(M), K), torch.float32, "sT")
    _check(_lib.fp8q_transpose_quant_fp8(_ptr(q), _ptr(s), M, K, s.shape[1], _ptr(qT), _ptr(sT),
                                         _stream(stream)), "fp8q_transpose_quant_fp8")


def rmsnorm_quant_dual(x, gamma, eps, q_row, s_row, q_colT, s_col, rstd, stream=None):
    """Option B: RMSNorm(x)*gamma in BF16, emitted 1x128 (rows) and 128x1 (transposed),
    plus the per-row reciprocal RMS."""
    _want(x, torch.bfloat16, 2, "x"); _want(gamma, torch.bfloat16, 1, "gamma")
    for t, n in ((q_row, "q_row"), (s_row, "s_row"), (q_colT, "q_colT"), (s_col, "s_col"),
                 (rstd, "rstd")):
        _dense(t, n)
    M, H = x.shape
    _shape(gamma, (H,), torch.bfloat16, "gamma")
    _shape(q_row, (M, H), torch.uint8, "q_row")
    _scales_1x128(s_row, _groups(H), M, "s_row")
    _shape(q_colT, (H, M), torch.uint8, "q_colT")
    _shape(s_col, (_groups(M), H), torch.float32, "s_col")
    _shape(rstd, (M,), torch.float32, "rstd")
    _check(_lib.fp8q_rmsnorm_quant_dual(_ptr(x), _ptr(gamma), M, H, _rows_dense(x, "x"),
                                        float(eps), _ptr(q_row), _ptr(s_row), s_row.shape[1],
                                        _ptr(q_colT), _ptr(s_col), _ptr(rstd), _stream(stream)),
           "fp8q_rmsnorm_quant_dual")


def rmsnorm_quant_dual_alloc(x, gamma, eps, stream=None):
    M, H = x.shape
    q = _empty((M, H), torch.uint8, x.device, stream)
    s = _empty((_groups(H), lds_for(M)), torch.float32, x.device, stream)
    qT = _empty((H, M), torch.uint8, x.device, stream)
    sT = _empty((_groups(M), H), torch.float32, x.device, stream)
    r = _empty((M,), torch.float32, x.device, stream)
    rmsnorm_quant_dual(x, gamma, eps, q, s, qT, sT, r, stream)
    return q, s, qT, sT, r


def swiglu_quant_dual(gu, q_row, s_row, q_colT, s_col, stream=None):
    """Option B: SwiGLU(gate, up) in BF16, emitted 1x128 (rows) and 128x1 (transposed)."""
    _want(gu, torch.bfloat16, 2, "gu")
    for t, n in ((q_row, "q_row"), (s_row, "s_row"), (q_colT, "q_colT"), (s_col, "s_col")):
        _dense(t, n)
    M, I2 = gu.shape
    if I2 % 2:
        raise ValueError("gu must be [M, 2I] (gate | up), got %s" % (tuple(gu.shape),))
    I = I2 // 2
    _shape(q_row, (M, I), torch.uint8, "q_row")
    _scales_1x128(s_row, _groups(I), M, "s_row")
    _shape(q_colT, (I, M), torch.uint8, "q_colT")
    _shape(s_col, (_groups(M), I), torch.float32, "s_col")
    _check(_lib.fp8q_swiglu_quant_dual(_ptr(gu), M, I2 // 2, _rows_dense(gu, "gu"), _ptr(q_row),
                                       _ptr(s_row), s_row.shape[1], _ptr(q_colT), _ptr(s_col),
                                       _stream(stream)), "fp8q_swiglu_quant_dual")


def swiglu_quant_dual_alloc(gu, stream=None):
    M, I2 = gu.shape
    I = I2 // 2
    q = _empty((M, I), torch.uint8, gu.device, stream)
    s = _empty((_groups(I), lds_for(M)), torch.float32, gu.device, stream)
    qT = _empty((I, M), torch.uint8, gu.device, stream)
    sT = _empty((_groups(M), I), torch.float32, gu.device, stream)
    swiglu_quant_dual(gu, q, s, qT, sT, stream)
    return q, s, qT, sT


def swiglu_bwd_quant_dual(gu, dh, q_row, s_row, q_colT, s_col, dgu=None, stream=None):
    """SwiGLU backward in BF16 (gu [M, 2I] = [gate | up], dh [M, I]) with the gradient
    [d_gate | d_up] quantized 1x128 (rows) and 128x1 (transposed); dgu optionally receives
    the BF16 gradient."""
    _want(gu, torch.bfloat16, 2, "gu"); _want(dh, torch.bfloat16, 2, "dh")
    for t, n in ((gu, "gu"), (dh, "dh"), (q_row, "q_row"), (s_row, "s_row"),
                 (q_colT, "q_colT"), (s_col, "s_col")):
        _dense(t, n)
    if dgu is not None:
        _want(dgu, torch.bfloat16, 2, "dgu"); _dense(dgu, "dgu")
    M, I2 = gu.shape
    if dh.shape != (M, I2 // 2):
        raise ValueError("dh must be [M, I] for gu [M, 2I]")
    _shape(q_row, (M, I2), torch.uint8, "q_row")
    _scales_1x128(s_row, _groups(I2), M, "s_row")
    _shape(q_colT, (I2, M), torch.uint8, "q_colT")
    _shape(s_col, (_groups(M), I2), torch.float32, "s_col")
    if dgu is not None:
        _shape(dgu, (M, I2), torch.bfloat16, "dgu")
    _check(_lib.fp8q_swiglu_bwd_quant_dual(_ptr(gu), _ptr(dh), M, I2 // 2, _ptr(dgu), _ptr(q_row),
                                           _ptr(s_row), s_row.shape[1], _ptr(q_colT),
                                           _ptr(s_col), _stream(stream)),
           "fp8q_swiglu_bwd_quant_dual")


def swiglu_bwd_quant_dual_alloc(gu, dh, want_dgu=False, stream=None):
    M, I2 = gu.shape
    q = _empty((M, I2), torch.uint8, gu.device, stream)
    s = _empty((_groups(I2), lds_for(M)), torch.float32, gu.device, stream)
    qT = _empty((I2, M), torch.uint8, gu.device, stream)
    sT = _empty((_groups(M), I2), torch.float32, gu.device, stream)
    dgu = _empty((M, I2), torch.bfloat16, gu.device, stream) if want_dgu else None
    swiglu_bwd_quant_dual(gu, dh, q, s, qT, sT, dgu, stream)
    return q, s, qT, sT, dgu


def rmsnorm_bwd_workspace_bytes(M: int, H: int) -> int:
    return int(_lib.fp8q_rmsnorm_bwd_workspace_bytes(int(M), int(H)))


def rmsnorm_bwd_quant_dual(x, gamma, dy, dres, eps, out, q_row, s_row, q_colT, s_col, dgamma,
                           workspace, stream=None):
    """RMSNorm backward in BF16 plus the residual gradient dres (may be None): out [M, H]
    BF16, its 1x128 and 128x1 (transposed) quantizations, dgamma [H] fp32 (may be None).
    workspace: a uint8 CUDA tensor of rmsnorm_bwd_workspace_bytes(M, H) bytes."""
    _want(x, torch.bfloat16, 2, "x"); _want(gamma, torch.bfloat16, 1, "gamma")
    _want(dy, torch.bfloat16, 2, "dy"); _want(out, torch.bfloat16, 2, "out")
    if dres is not None:
        _want(dres, torch.bfloat16, 2, "dres")
    for t, n in ((x, "x"), (dy, "dy"), (dres, "dres"), (out, "out"), (q_row, "q_row"),
                 (s_row, "s_row"), (q_colT, "q_colT"), (s_col, "s_col"), (dgamma, "dgamma"),
                 (workspace, "workspace")):
        if t is not None:
            _dense(t, n)
    M, H = x.shape
    for t, n in ((dy, "dy"), (dres, "dres"), (out, "out")):
        if t is not None and t.shape != (M, H):
            raise ValueError("%s must have the shape of x" % n)
    _shape(gamma, (H,), torch.bfloat16, "gamma")
    _shape(q_row, (M, H), torch.uint8, "q_row")
    _scales_1x128(s_row, _groups(H), M, "s_row")
    _shape(q_colT, (H, M), torch.uint8, "q_colT")
    _shape(s_col, (_groups(M), H), torch.float32, "s_col")
    if dgamma is not None:
        _shape(dgamma, (H,), torch.float32, "dgamma")
    if workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    _check(_lib.fp8q_rmsnorm_bwd_quant_dual(
        _ptr(x), _ptr(gamma), _ptr(dy), _ptr(dres), M, H, float(eps), _ptr(out), _ptr(q_row),
        _ptr(s_row), s_row.shape[1], _ptr(q_colT), _ptr(s_col), _ptr(dgamma), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "fp8q_rmsnorm_bwd_quant_dual")


def rmsnorm_bwd_quant_dual_alloc(x, gamma, dy, dres, eps, stream=None):
    M, H = x.shape
    dev = x.device
    out = _empty((M, H), torch.bfloat16, dev, stream)
    q = _empty((M, H), torch.uint8, dev, stream)
    s = _empty((_groups(H), lds_for(M)), torch.float32, dev, stream)
    qT = _empty((H, M), torch.uint8, dev, stream)
    sT = _empty((_groups(M), H), torch.float32, dev, stream)
    dg = _empty((H,), torch.float32, dev, stream)
    nbytes = rmsnorm_bwd_workspace_bytes(M, H)
    ws = _empty((max(nbytes, 16),), torch.uint8, dev, stream)
    rmsnorm_bwd_quant_dual(x, gamma, dy, dres, eps, out, q, s, qT, sT, dg, ws, stream)
    return out, q, s, qT, sT, dg


def _gemm_operands(qa, sa, qw, name_a, name_sa, name_w):
    """Extents of a block-scaled product [M, N] = qa [M, K] x qw [N, K]^T: checks the
    two code operands and the 1x128 row scales sa [K/128, >= M]; returns (M, N, K) for
    the caller to check the block scales and the output against."""
    if not isinstance(qa, torch.Tensor) or qa.dim() != 2 or qa.dtype != torch.uint8:
        raise ValueError("%s must be a 2-D uint8 tensor" % name_a)
    if not isinstance(qw, torch.Tensor) or qw.dim() != 2 or qw.dtype != torch.uint8:
        raise ValueError("%s must be a 2-D uint8 tensor" % name_w)
    M, K = qa.shape
    N = qw.shape[0]
    _shape(qw, (N, K), torch.uint8, name_w)
    _scales_1x128(sa, _groups(K), M, name_sa)
    return M, N, K


def linear_fwd(qa, sa, qw, sw, y, stream=None):
    """a5: y BF16 [M,N] = block-scaled qa [M,K] x qw [N,K]^T."""
    for t, n in ((qa, "qa"), (sa, "sa"), (qw, "qw"), (sw, "sw")):
        _dense(t, n)
    M, N, K = _gemm_operands(qa, sa, qw, "qa", "sa", "qw")
    _shape(sw, (_groups(N), _groups(K)), torch.float32, "sw")
    _shape(y, (M, N), torch.bfloat16, "y")
    _check(_lib.fp8q_linear_fwd(_ptr(qa), _ptr(sa), sa.shape[1], _ptr(qw), _ptr(sw), M, N, K,
                                _ptr(y), _rows_dense(y, "y"), _stream(stream)), "fp8q_linear_fwd")


def linear_fwd_splitk_workspace_bytes(M, N, K):
    """Bytes of workspace fp8q_linear_fwd_splitk needs for this shape (0 if unsupported)."""
    return int(_lib.fp8q_linear_fwd_splitk_workspace(M, N, K))


def splitk_workspace(M, N, K, device):
    """A workspace for fp8q_linear_fwd_splitk, zero-filled (its counters must start at
    zero; the kernel leaves them at zero)."""
    n = linear_fwd_splitk_workspace_bytes(M, N, K)
    if n <= 0:
        raise ValueError("no split-K workspace for M=%d N=%d K=%d" % (M, N, K))
    return torch.zeros(n, dtype=torch.uint8, device=device)


def linear_fwd_splitk(qa, sa, qw, sw, y, workspace, stream=None):
    """a5 at decode sizes with K split over CTAs (same bits as linear_fwd); `workspace`
    is a uint8 device tensor from splitk_workspace (not shared by concurrent calls)."""
    for t, n in ((qa, "qa"), (sa, "sa"), (qw, "qw"), (sw, "sw")):
        _dense(t, n)
    M, N, K = _gemm_operands(qa, sa, qw, "qa", "sa", "qw")
    _shape(sw, (_groups(N), _groups(K)), torch.float32, "sw")
    _shape(y, (M, N), torch.bfloat16, "y")
    _want(workspace, torch.uint8, 1, "workspace")
    _check(_lib.fp8q_linear_fwd_splitk(_ptr(qa), _ptr(sa), sa.shape[1], _ptr(qw), _ptr(sw), M, N,
                                       K, _ptr(y), _rows_dense(y, "y"), _ptr(workspace),
                                       workspace.numel(), _stream(stream)),
           "fp8q_linear_fwd_splitk")


def linear_fwd_splitk_noalloc(qa, sa, qw, sw, y, stream=None):
    """linear_fwd_splitk on the library's static workspace (no allocation; calls on one
    device must not overlap)."""
    for t, n in ((qa, "qa"), (sa, "sa"), (qw, "qw"), (sw, "sw")):
        _dense(t, n)
    M, N, K = _gemm_operands(qa, sa, qw, "qa", "sa", "qw")
    _shape(sw, (_groups(N), _groups(K)), torch.float32, "sw")
    _shape(y, (M, N), torch.bfloat16, "y")
    _check(_lib.fp8q_linear_fwd_splitk_noalloc(_ptr(qa), _ptr(sa), sa.shape[1], _ptr(qw),
                                               _ptr(sw), M, N, K, _ptr(y), _rows_dense(y, "y"),
                                               _stream(stream)),
           "fp8q_linear_fwd_splitk_noalloc")


def linear_dgrad(qdy, sdy, qwT, sw, dx, stream=None):
    """a7: dx BF16 [M,K] = block-scaled qdy [M,N] x W [N,K] (weights passed transposed,
    qwT [K,N])."""
    for t, n in ((qdy, "qdy"), (sdy, "sdy"), (qwT, "qwT"), (sw, "sw")):
        _dense(t, n)
    # dx [M, K] = qdy [M, N] x qwT [K, N]^T: the product's reduction runs over N
    M, K, N = _gemm_operands(qdy, sdy, qwT, "qdy", "sdy", "qwT")
    _shape(sw, (_groups(N), _groups(K)), torch.float32, "sw")
    _shape(dx, (M, K), torch.bfloat16, "dx")
    _check(_lib.fp8q_linear_dgrad(_ptr(qdy), _ptr(sdy), sdy.shape[1], _ptr(qwT), _ptr(sw), M, N,
                                  K, _ptr(dx), _rows_dense(dx, "dx"), _stream(stream)),
           "fp8q_linear_dgrad")


def _wgrad_operands(qdyT, sdy_c, qxT, sx_c):
    """Shapes of WGrad: qdyT [N, M] and qxT [K, M] (128x1 codes, transposed) with their
    scales sdy_c [M/128, N] and sx_c [M/128, K]. Returns (N, M, K)."""
    for t, n in ((qdyT, "qdyT"), (qxT, "qxT")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype != torch.uint8:
            raise ValueError("%s must be a 2-D uint8 tensor" % n)
    N, M = qdyT.shape
    K = qxT.shape[0]
    _shape(qxT, (K, M), torch.uint8, "qxT")
    _shape(sdy_c, (_groups(M), N), torch.float32, "sdy_c")
    _shape(sx_c, (_groups(M), K), torch.float32, "sx_c")
    return N, M, K


def linear_wgrad(qdyT, sdy_c, qxT, sx_c, dw, stream=None):
    """a9: dw BF16 [N,K] = sum over 128-token groups of (qdyT [N,M]) x (qxT [K,M])^T with
    the 128x1 scales sdy_c [M/128,N] and sx_c [M/128,K]."""
    for t, n in ((qdyT, "qdyT"), (sdy_c, "sdy_c"), (qxT, "qxT"), (sx_c, "sx_c")):
        _dense(t, n)
    N, M, K = _wgrad_operands(qdyT, sdy_c, qxT, sx_c)
    _shape(dw, (N, K), torch.bfloat16, "dw")
    _check(_lib.fp8q_linear_wgrad(_ptr(qdyT), _ptr(sdy_c), _ptr(qxT), _ptr(sx_c), M, N, K,
                                  _ptr(dw), _rows_dense(dw, "dw"), _stream(stream)),
           "fp8q_linear_wgrad")


def linear_wgrad_acc_f32(qdyT, sdy_c, qxT, sx_c, dw, stream=None):
    """WGrad accumulated in fp32: dw [N,K] (fp32) += the fp32 accumulator of linear_wgrad."""
    for t, n in ((qdyT, "qdyT"), (sdy_c, "sdy_c"), (qxT, "qxT"), (sx_c, "sx_c")):
        _dense(t, n)
    N, M, K = _wgrad_operands(qdyT, sdy_c, qxT, sx_c)
    _shape(dw, (N, K), torch.float32, "dw")
    _check(_lib.fp8q_linear_wgrad_acc_f32(_ptr(qdyT), _ptr(sdy_c), _ptr(qxT), _ptr(sx_c), M, N,
                                          K, _ptr(dw), _rows_dense(dw, "dw"), _stream(stream)),
           "fp8q_linear_wgrad_acc_f32")


# --------------------------------------------------------------------------
# One weight per expert (ragged row groups), and the norm in front of it
# --------------------------------------------------------------------------

def _row_stride(t, rows, cols, name):
    """Row stride of a matrix [rows, cols] that is not contiguous, with dense rows (a single
    row has none: its length)."""
    r, c = t.stride()
    if c != 1 and cols > 1:
        raise ValueError("%s must have unit column stride" % name)
    return r if rows > 1 else cols


def _raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


# The same without a Stream object, and the device without the check that CUDA is up (it is:
# the operands lie there): 3 us of a small call, where torch has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(fn, where, stream, dev, *args):
    """Call `fn` on device `dev` (the current one or not), on `stream` or that device's
    current stream."""
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if status != FP8Q_OK:
        raise Fp8qError(status, where)


def _device(names, *operands):
    """Refuse operands (None: not given) that do not lie on one CUDA device, by name; the
    callers compare the devices themselves first."""
    dev = operands[0].get_device()
    if dev < 0:
        raise ValueError("libfp8q takes CUDA tensors (device pointers)")
    for t in operands:
        if t is not None and t.get_device() != dev:
            name = [n for n, o in zip(names.split(), operands) if o is t][0]
            raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))


_T, _BF16, _U8, _F32 = torch.Tensor, torch.bfloat16, torch.uint8, torch.float32


def _scales_dense(s, groups, rows, name):
    """Dense 1x128 scales fp32 [groups, lds >= rows]; returns lds."""
    if isinstance(s, torch.Tensor) and s.dtype == _F32 and s.dim() == 2 and s.is_contiguous():
        g, lds = s.shape
        if g == groups and lds >= rows:
            return lds
    _scales_1x128(s, groups, rows, name)
    _dense(s, name)
    return s.shape[1]


def _exact(t, shape, dtype, name):
    """_shape for a tuple of ints, with the failing case left to it."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape:
        _shape(t, shape, dtype, name)


def _exact_dense(t, shape, dtype, name):
    _exact(t, shape, dtype, name)
    if not t.is_contiguous():
        _dense(t, name)


def _offsets(offsets):
    """int32 [E + 1]; returns E."""
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a torch.Tensor")
    n = offsets.numel()
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or n < 2:
        raise ValueError("offsets must be an int32 tensor [E + 1], got %s %s" % (
            tuple(offsets.shape), offsets.dtype))
    if not offsets.is_contiguous():
        _dense(offsets, "offsets")
    return n - 1


def grouped_padded_rows(M, E) -> int:
    """Columns P of the transposed arrays of a grouped call over M rows and E experts that
    are enough whatever the offsets are (a multiple of 128)."""
    n = int(_lib.fp8q_grouped_padded_rows(int(M), int(E)))
    if n < 0:
        raise ValueError("grouped_padded_rows: M=%d E=%d" % (M, E))
    return n


def add_rmsnorm_quant(x, res, gamma, eps, h, q, s, stream=None):
    """a3 behind a residual addition: h = bf16(x + res) [M,H] (may be x or res itself), then
    RMSNorm(h)*gamma in BF16 -> q [M,H], s [H/128, lds]; H % 16 == 0. Its backward is
    rmsnorm_bwd_quant_dual on h, for H % 128 == 0 and rows rounded up to a multiple of 128
    (zeros in h, dy and dres behind row M)."""
    _want(x, _BF16, 2, "x")
    M, H = shape = x.shape
    # one comparison of everything on the way of a correct call; the checks one by one (and
    # their messages) only where it fails
    if not (isinstance(res, _T) and isinstance(h, _T) and isinstance(gamma, _T)
            and isinstance(q, _T) and res.dtype == h.dtype == gamma.dtype == _BF16
            and q.dtype == _U8 and res.shape == h.shape == q.shape == shape and gamma.shape == (H,)
            and gamma.is_contiguous() and q.is_contiguous()):
        _exact(res, shape, _BF16, "res")
        _exact(h, shape, _BF16, "h")
        _exact_dense(gamma, (H,), _BF16, "gamma")
        _exact_dense(q, shape, _U8, "q")
    lds = _scales_dense(s, _groups(H), M, "s")
    dev = x.get_device()
    if not (0 <= dev == res.get_device() == gamma.get_device() == h.get_device()
            == q.get_device() == s.get_device()):
        _device("x res gamma h q s", x, res, gamma, h, q, s)
    if M == 0:  # a rank without tokens, as in the grouped calls
        return
    _run(_lib.fp8q_add_rmsnorm_quant, "fp8q_add_rmsnorm_quant", stream, dev, x.data_ptr(),
         res.data_ptr(), gamma.data_ptr(), M, H,
         H if x.is_contiguous() else _row_stride(x, M, H, "x"),
         H if res.is_contiguous() else _row_stride(res, M, H, "res"), float(eps), h.data_ptr(),
         H if h.is_contiguous() else _row_stride(h, M, H, "h"),
         q.data_ptr(), s.data_ptr(), lds)


def add_rmsnorm_quant_alloc(x, res, gamma, eps, stream=None):
    """add_rmsnorm_quant into new tensors: (h, q, s)."""
    M, H = x.shape
    h = _empty((M, H), torch.bfloat16, x.device, stream)
    q = _empty((M, H), torch.uint8, x.device, stream)
    s = _empty((_groups(H), lds_for(M)), torch.float32, x.device, stream)
    add_rmsnorm_quant(x, res, gamma, eps, h, q, s, stream)
    return h, q, s


def grouped_quant_weight_alloc(w, want_t=True, stream=None):
    """The weights w BF16 [E,N,K] of E experts, quantized per 128x128 block by one
    quant_weight_128x128 over the stacked [E*N,K] matrix: (qw [E,N,K], sw
    [E,N/128,K/128], qwT [K,E,N] or None), the operands of the grouped products."""
    _want(w, torch.bfloat16, 3, "w")
    _dense(w, "w")
    E, N, K = w.shape
    if N % 128 or K % 128:
        raise ValueError("w must be [E, N, K] with N and K multiples of 128, got %s" % (
            tuple(w.shape),))
    dev = w.get_device()
    if dev < 0:
        raise ValueError("libfp8q takes CUDA tensors (device pointers)")
    with torch.cuda.device(dev):  # as the grouped calls: on w's device, the current one or not
        q, s, qT = quant_weight_alloc(w.view(E * N, K), want_t, stream)
    return (q.view(E, N, K), s.view(E, N // 128, K // 128),
            qT.view(K, E, N) if want_t else None)


def _grouped_weight(qw, sw, offsets, name, N_at):
    """Stacked weight codes (qw [E,N,K] with N_at = 1, qwT [K,E,N] with N_at = 2) and their
    block scales sw [E,N/128,K/128], for offsets [E+1]; returns (E, N, K)."""
    _want(qw, torch.uint8, 3, name)
    _dense(qw, name)
    shape = qw.shape
    E, N, K = shape if N_at == 1 else (shape[1], shape[2], shape[0])
    if _offsets(offsets) != E:
        raise ValueError("%s holds %d experts, offsets %d" % (name, E, offsets.numel() - 1))
    _exact_dense(sw, (E, _groups(N), _groups(K)), torch.float32, "sw")
    return E, N, K


def _grouped_rows(q, s, width, name_q, name_s):
    """Row operand q [M,width] with its 1x128 scales; returns M and the scales' lds."""
    _want(q, _U8, 2, name_q)
    M, cols = q.shape
    if cols != width or not q.is_contiguous():
        _exact_dense(q, (M, width), _U8, name_q)
    return M, _scales_dense(s, _groups(width), M, name_s)


def grouped_linear_fwd(qa, sa, qw, sw, offsets, y, stream=None):
    """linear_fwd with one weight per expert: rows offsets[e] .. offsets[e+1]-1 of qa [M,K]
    times qw[e] ([E,N,K], see grouped_quant_weight_alloc) -> the same rows of y BF16 [M,N].
    Rows of no expert are left as they are. offsets: int32 [E+1] on the device."""
    E, N, K = _grouped_weight(qw, sw, offsets, "qw", 1)
    M, lds = _grouped_rows(qa, sa, K, "qa", "sa")
    _exact(y, (M, N), torch.bfloat16, "y")
    dev = qa.get_device()
    if not (0 <= dev == sa.get_device() == qw.get_device() == sw.get_device()
            == offsets.get_device() == y.get_device()):
        _device("qa sa qw sw offsets y", qa, sa, qw, sw, offsets, y)
    _run(_lib.fp8q_grouped_linear_fwd, "fp8q_grouped_linear_fwd", stream, dev, qa.data_ptr(),
         sa.data_ptr(), lds, qw.data_ptr(), sw.data_ptr(), offsets.data_ptr(), E, M, N, K,
         y.data_ptr(), N if y.is_contiguous() else _row_stride(y, M, N, "y"))


def grouped_linear_dgrad(qdy, sdy, qwT, sw, offsets, dx, stream=None):
    """linear_dgrad with one weight per expert: qdy [M,N] x W[e] -> dx BF16 [M,K] (weights
    transposed and stacked, qwT [K,E,N]). Rows of no expert are left as they are."""
    E, N, K = _grouped_weight(qwT, sw, offsets, "qwT", 2)
    M, lds = _grouped_rows(qdy, sdy, N, "qdy", "sdy")
    _exact(dx, (M, K), torch.bfloat16, "dx")
    dev = qdy.get_device()
    if not (0 <= dev == sdy.get_device() == qwT.get_device() == sw.get_device()
            == offsets.get_device() == dx.get_device()):
        _device("qdy sdy qwT sw offsets dx", qdy, sdy, qwT, sw, offsets, dx)
    _run(_lib.fp8q_grouped_linear_dgrad, "fp8q_grouped_linear_dgrad", stream, dev, qdy.data_ptr(),
         sdy.data_ptr(), lds, qwT.data_ptr(), sw.data_ptr(), offsets.data_ptr(), E, M, N, K,
         dx.data_ptr(), K if dx.is_contiguous() else _row_stride(dx, M, K, "dx"))


def _grouped_columns(qT, sT, rows, name_q, name_s):
    """Transposed codes [rows,P] with their 128x1 scales [P/128,rows]; returns P."""
    _want(qT, _U8, 2, name_q)
    n, P = qT.shape
    if P % 128:
        raise ValueError("%s must have a multiple of 128 columns, got %s" % (
            name_q, tuple(qT.shape)))
    if n != rows or not qT.is_contiguous():
        _exact_dense(qT, (rows, P), _U8, name_q)
    _exact_dense(sT, (P // 128, rows), _F32, name_s)
    return P


def grouped_transpose_quant_bf16(dy, offsets, q_row, s_row, q_colT, s_col, stream=None):
    """a6 with 128x1 groups that restart at each expert: dy BF16 [M,N] -> q_row [M,N], s_row
    [N/128,lds] (both may be None) and q_colT [N,P], s_col [P/128,N], with
    P >= grouped_padded_rows(M, E)."""
    _want(dy, torch.bfloat16, 2, "dy")
    E = _offsets(offsets)
    M, N = shape = dy.shape
    lds_row = 0
    if (q_row is None) != (s_row is None):
        raise ValueError("q_row and s_row must be given together")
    if q_row is not None:
        _exact_dense(q_row, shape, _U8, "q_row")
        lds_row = _scales_dense(s_row, _groups(N), M, "s_row")
    P = _grouped_columns(q_colT, s_col, N, "q_colT", "s_col")
    dev = dy.get_device()
    if not (0 <= dev == offsets.get_device() == q_colT.get_device() == s_col.get_device()
            and (q_row is None or dev == q_row.get_device() == s_row.get_device())):
        _device("dy offsets q_colT s_col q_row s_row", dy, offsets, q_colT, s_col, q_row, s_row)
    _run(_lib.fp8q_grouped_transpose_quant_bf16, "fp8q_grouped_transpose_quant_bf16", stream, dev,
         dy.data_ptr(), offsets.data_ptr(), E, M, N,
         N if dy.is_contiguous() else _row_stride(dy, M, N, "dy"),
         None if q_row is None else q_row.data_ptr(), None if s_row is None else s_row.data_ptr(),
         lds_row, q_colT.data_ptr(), s_col.data_ptr(), P)


def grouped_transpose_quant_bf16_alloc(dy, offsets, want_row=True, stream=None):
    """grouped_transpose_quant_bf16 into new tensors: (q_row, s_row, q_colT, s_col). Rows of
    no expert and columns past the last group hold whatever the memory held."""
    M, N = dy.shape
    P = grouped_padded_rows(M, _offsets(offsets))
    q_row = _empty((M, N), torch.uint8, dy.device, stream) if want_row else None
    s_row = _empty((_groups(N), lds_for(M)), torch.float32, dy.device, stream) if want_row else None
    q_colT = _empty((N, P), torch.uint8, dy.device, stream)
    s_col = _empty((P // 128, N), torch.float32, dy.device, stream)
    grouped_transpose_quant_bf16(dy, offsets, q_row, s_row, q_colT, s_col, stream)
    return q_row, s_row, q_colT, s_col


def grouped_transpose_quant_fp8(q, s, offsets, qT, sT, stream=None):
    """a8 with 128x1 groups that restart at each expert: saved FP8 (q [M,K], s [K/128,lds])
    -> qT [K,P], sT [P/128,K], with P >= grouped_padded_rows(M, E)."""
    _want(q, torch.uint8, 2, "q")
    E = _offsets(offsets)
    K = q.shape[1]
    M, lds = _grouped_rows(q, s, K, "q", "s")
    P = _grouped_columns(qT, sT, K, "qT", "sT")
    dev = q.get_device()
    if not (0 <= dev == s.get_device() == offsets.get_device() == qT.get_device()
            == sT.get_device()):
        _device("q s offsets qT sT", q, s, offsets, qT, sT)
    _run(_lib.fp8q_grouped_transpose_quant_fp8, "fp8q_grouped_transpose_quant_fp8", stream, dev,
         q.data_ptr(), s.data_ptr(), offsets.data_ptr(), E, M, K, lds, qT.data_ptr(),
         sT.data_ptr(), P)


def grouped_transpose_quant_fp8_alloc(q, s, offsets, stream=None):
    """grouped_transpose_quant_fp8 into new tensors: (qT, sT)."""
    M, K = q.shape
    P = grouped_padded_rows(M, _offsets(offsets))
    qT = _empty((K, P), torch.uint8, q.device, stream)
    sT = _empty((P // 128, K), torch.float32, q.device, stream)
    grouped_transpose_quant_fp8(q, s, offsets, qT, sT, stream)
    return qT, sT


def grouped_linear_wgrad(qdyT, sdy_c, qxT, sx_c, offsets, dw, stream=None):
    """linear_wgrad per expert: dw[e] BF16 [N,K] = expert e's groups of qdyT [N,P] x qxT
    [K,P]^T (the outputs of the grouped quantizers, one P for both); zeros for an expert
    without rows. dw is [E,N,K], dense. Of the offsets only the order and the groups' total
    against P are checked on the device (the quantizers check them against their rows)."""
    _want(qdyT, torch.uint8, 2, "qdyT"); _want(qxT, torch.uint8, 2, "qxT")
    N, K = qdyT.shape[0], qxT.shape[0]
    if qxT.shape[1] != qdyT.shape[1]:
        raise ValueError("qxT must have the columns of qdyT (%d), got %s" % (
            qdyT.shape[1], tuple(qxT.shape)))
    P = _grouped_columns(qdyT, sdy_c, N, "qdyT", "sdy_c")
    _grouped_columns(qxT, sx_c, K, "qxT", "sx_c")
    E = _offsets(offsets)
    _want(dw, torch.bfloat16, 3, "dw")
    if dw.shape[0] != E:
        raise ValueError("dw holds %d experts, offsets %d" % (dw.shape[0], E))
    _exact_dense(dw, (E, N, K), torch.bfloat16, "dw")
    dev = qdyT.get_device()
    if not (0 <= dev == sdy_c.get_device() == qxT.get_device() == sx_c.get_device()
            == offsets.get_device() == dw.get_device()):
        _device("qdyT sdy_c qxT sx_c offsets dw", qdyT, sdy_c, qxT, sx_c, offsets, dw)
    _run(_lib.fp8q_grouped_linear_wgrad, "fp8q_grouped_linear_wgrad", stream, dev,
         qdyT.data_ptr(), sdy_c.data_ptr(), qxT.data_ptr(), sx_c.data_ptr(), offsets.data_ptr(),
         E, P, N, K, dw.data_ptr(), K)


def debug_wait_timeout(limit_ns: int, stream=None) -> int:
    """Launch the bounded-wait probe (gives up after limit_ns); returns the launch status."""
    return int(_lib.fp8q_debug_wait_timeout(int(limit_ns), _stream(stream)))


# --------------------------------------------------------------------------
# Allocating helpers (torch allocates; the kernels are the ones above)
# --------------------------------------------------------------------------

def _empty(shape, dtype, device, stream=None):
    """A new tensor for a call on `stream`: its memory is taken from that stream's pool. From
    the current stream's, the call could write what is still in use there (a block freed
    before the work on it was done), and a workspace could be given away before the call's
    kernels have used it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def quant_act_1x128_alloc(x, stream=None):
    M, K = x.shape
    q = _empty((M, K), torch.uint8, x.device, stream)
    s = _empty((_groups(K), lds_for(M)), torch.float32, x.device, stream)
    quant_act_1x128(x, q, s, stream)
    return q, s


def quant_weight_alloc(w, want_t=True, stream=None):
    N, K = w.shape
    q = _empty((N, K), torch.uint8, w.device, stream)
    s = _empty((_groups(N), _groups(K)), torch.float32, w.device, stream)
    qT = _empty((K, N), torch.uint8, w.device, stream) if want_t else None
    quant_weight_128x128(w, q, s, qT, stream)
    return q, s, qT


def rmsnorm_quant_alloc(x, gamma, eps, stream=None):
    M, H = x.shape
    q = _empty((M, H), torch.uint8, x.device, stream)
    s = _empty((_groups(H), lds_for(M)), torch.float32, x.device, stream)
    rmsnorm_quant(x, gamma, eps, q, s, stream)
    return q, s


def swiglu_quant_alloc(gu, stream=None):
    M, I2 = gu.shape
    q = _empty((M, I2 // 2), torch.uint8, gu.device, stream)
    s = _empty((_groups(I2 // 2), lds_for(M)), torch.float32, gu.device, stream)
    swiglu_quant(gu, q, s, stream)
    return q, s


def transpose_quant_bf16_alloc(dy, want_row=True, stream=None):
    M, N = dy.shape
    q_row = _empty((M, N), torch.uint8, dy.device, stream) if want_row else None
    s_row = _empty((_groups(N), lds_for(M)), torch.float32, dy.device, stream) if want_row else None
    q_colT = _empty((N, M), torch.uint8, dy.device, stream)
    s_col = _empty((_groups(M), N), torch.float32, dy.device, stream)
    transpose_quant_bf16(dy, q_row, s_row, q_colT, s_col, stream)
    return q_row, s_row, q_colT, s_col


def transpose_quant_fp8_alloc(q, s, stream=None):
    M, K = q.shape
    qT = _empty((K, M), torch.uint8, q.device, stream)
    sT = _empty((_groups(M), K), torch.float32, q.device, stream)
    transpose_quant_fp8(q, s, qT, sT, stream)
    return qT, sT


def linear_fwd_alloc(qa, sa, qw, sw, stream=None):
    y = _empty((qa.shape[0], qw.shape[0]), torch.bfloat16, qa.device, stream)
    linear_fwd(qa, sa, qw, sw, y, stream)
    return y


def linear_dgrad_alloc(qdy, sdy, qwT, sw, stream=None):
    dx = _empty((qdy.shape[0], qwT.shape[0]), torch.bfloat16, qdy.device, stream)
    linear_dgrad(qdy, sdy, qwT, sw, dx, stream)
    return dx


def linear_wgrad_alloc(qdyT, sdy_c, qxT, sx_c, stream=None):
    dw = _empty((qdyT.shape[0], qxT.shape[0]), torch.bfloat16, qdyT.device, stream)
    linear_wgrad(qdyT, sdy_c, qxT, sx_c, dw, stream)
    return dw
