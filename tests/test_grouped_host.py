"""Host side of the expert-layer operators (no GPU): the C entry points refuse bad sizes,
alignments, NULL pointers and overlaps before any CUDA call, and the binding refuses
mismatched operands by name before it takes a pointer."""
import ctypes

import pytest
import torch

import fp8_block_scaled_08_b200 as fq

# never dereferenced: every call below is refused (or has nothing to do) on the host
A, B, C, D, E_, F_ = (ctypes.c_void_p(0x100000 * i) for i in range(1, 7))
ODD = ctypes.c_void_p(0x100008)
NUL = None
NULL, SHAPE, ALIGN, OK = 1, 2, 3, 0
FLT = ctypes.c_float


def call(name, *args):
    return getattr(fq._lib, name)(*args)


def test_status_string_of_bad_offsets():
    assert fq.status_string(fq.FP8Q_ERR_OFFSETS).startswith("FP8Q_ERR_OFFSETS")


@pytest.mark.parametrize("M", [0, 1, 5, 127, 128, 129, 1000])
@pytest.mark.parametrize("E", [1, 2, 7, 64, 1024])
def test_padded_rows_cover_every_routing(M, E):
    P = fq.grouped_padded_rows(M, E)
    assert P % 128 == 0
    # the routing that needs most: one row to as many experts as possible, the rest to one
    k = min(E, M)
    most = [1] * k
    if k:
        left = M - k
        for i in range(k):  # the fewest rows that open another group
            add = min(left, 0 if i else left // 128 * 128)
            most[i] += add
            left -= add
        most[0] += left
    need = 128 * sum(-(-n // 128) for n in most)
    assert need <= P
    assert P < need + 128 * max(1, k) + 128


def test_padded_rows_refuses():
    for m, e in [(-1, 4), (4, 0), (4, 1025), (1 << 31, 4)]:
        assert call("fp8q_grouped_padded_rows", m, e) == -1
        with pytest.raises(ValueError):
            fq.grouped_padded_rows(m, e)


def fwd(M=8, N=256, K=128, E=4, lds=8, ldy=256, qa=A, sa=B, qw=C, sw=D, off=E_, y=F_):
    return call("fp8q_grouped_linear_fwd", qa, sa, lds, qw, sw, off, E, M, N, K, y, ldy, NUL)


def dgrad(M=8, N=256, K=128, E=4, lds=8, ldx=128, qa=A, sa=B, qw=C, sw=D, off=E_, y=F_):
    return call("fp8q_grouped_linear_dgrad", qa, sa, lds, qw, sw, off, E, M, N, K, y, ldx, NUL)


@pytest.mark.parametrize("f", [fwd, dgrad])
def test_validation_grouped_products(f):
    assert f(N=200) == SHAPE and f(K=64) == SHAPE and f(N=0) == SHAPE and f(K=-128) == SHAPE
    assert f(M=-1) == SHAPE and f(E=0) == SHAPE and f(E=1025) == SHAPE
    assert f(lds=4) == SHAPE
    assert f(lds=10) == ALIGN
    assert f(M=0) == OK and f(M=0, qa=NUL, y=NUL) == OK
    for k in ("qa", "sa", "qw", "sw", "off", "y"):
        assert f(**{k: NUL}) == NULL, k
    for k in ("qa", "sa", "qw", "sw", "y"):
        assert f(**{k: ODD}) == ALIGN, k
    assert f(off=ctypes.c_void_p(0x100002)) == ALIGN
    assert fwd(ldy=248) == SHAPE and fwd(ldy=260) == ALIGN
    assert dgrad(ldx=120) == SHAPE and dgrad(ldx=132) == ALIGN


def wgrad(P=256, N=256, K=128, E=4, ld=128, a=A, sa=B, b=C, sb=D, off=E_, dw=F_):
    return call("fp8q_grouped_linear_wgrad", a, sa, b, sb, off, E, P, N, K, dw, ld, NUL)


def test_validation_grouped_wgrad():
    assert wgrad(P=100) == SHAPE and wgrad(P=-128) == SHAPE and wgrad(N=200) == SHAPE
    assert wgrad(K=96) == SHAPE and wgrad(E=0) == SHAPE and wgrad(ld=120) == SHAPE
    assert wgrad(ld=132) == ALIGN
    assert wgrad(dw=NUL) == NULL and wgrad(P=0, dw=NUL) == NULL
    for k in ("a", "sa", "b", "sb", "off"):
        assert wgrad(**{k: NUL}) == NULL, k
    for k in ("a", "sa", "b", "sb", "dw"):
        assert wgrad(**{k: ODD}) == ALIGN, k


def tq_bf16(M=100, N=256, E=4, ld=256, lds=100, P=512, dy=A, off=B, q=C, s=D, qT=E_, sT=F_):
    return call("fp8q_grouped_transpose_quant_bf16", dy, off, E, M, N, ld, q, s, lds, qT, sT, P,
                NUL)


def tq_fp8(M=100, N=256, E=4, lds=100, P=512, q=A, s=B, off=C, qT=D, sT=E_):
    return call("fp8q_grouped_transpose_quant_fp8", q, s, off, E, M, N, lds, qT, sT, P, NUL)


def test_validation_grouped_quantizers():
    for f in (tq_bf16, tq_fp8):
        assert f(N=100) == SHAPE and f(M=-1) == SHAPE and f(E=0) == SHAPE and f(E=2000) == SHAPE
        assert f(P=384) == SHAPE and f(P=500) == SHAPE      # fewer columns than the rows may need
        assert f(lds=96) == SHAPE
        assert f(M=0) == OK
        for k in ("off", "qT", "sT", "s"):
            assert f(**{k: NUL}) == NULL, k
        for k in ("qT", "sT", "s", "q"):
            assert f(**{k: ODD}) == ALIGN, k
    assert tq_bf16(ld=200) == SHAPE and tq_bf16(ld=260) == ALIGN and tq_bf16(dy=ODD) == ALIGN
    assert tq_fp8(q=NUL) == NULL and tq_bf16(dy=NUL) == NULL
    assert tq_fp8(lds=102) == ALIGN


def norm(x=A, r=B, g=C, M=4, H=256, ldx=256, ldr=256, eps=1e-5, h=D, ldh=256, q=E_, s=F_, lds=4):
    return call("fp8q_add_rmsnorm_quant", x, r, g, M, H, ldx, ldr, FLT(eps), h, ldh, q, s, lds, NUL)


def test_validation_add_rmsnorm():
    assert norm(H=100) == SHAPE and norm(H=32768, ldx=32768, ldr=32768, ldh=32768) == SHAPE
    assert norm(M=0) == SHAPE and norm(eps=-1.0) == SHAPE and norm(eps=float("nan")) == SHAPE
    assert norm(ldx=128) == SHAPE and norm(ldr=128) == SHAPE and norm(ldh=128) == SHAPE
    assert norm(lds=2) == SHAPE
    assert norm(ldx=260) == ALIGN and norm(ldr=260) == ALIGN and norm(ldh=260) == ALIGN
    for k in ("x", "r", "g", "h", "q", "s"):
        assert norm(**{k: NUL}) == NULL, k
        assert norm(**{k: ODD}) == ALIGN, k


def test_add_rmsnorm_refuses_a_partial_overlap():
    # h one row behind x, or shifted by some columns of the same rows
    assert norm(h=ctypes.c_void_p(0x100000 + 512)) == SHAPE
    assert norm(h=ctypes.c_void_p(0x100000 + 32)) == SHAPE
    assert norm(h=ctypes.c_void_p(0x200000 + 32)) == SHAPE              # over res
    assert norm(h=A, ldh=264) == SHAPE                                  # in place, other stride


# ---------------------------------------------------------------------------- binding
M, N, K, E = 200, 256, 384, 3
P = 128 * ((M + 127 * E) // 128)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(s)


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def off(n=E):
    return torch.zeros(n + 1, dtype=torch.int32)


def good():
    return {
        fq.grouped_linear_fwd: dict(qa=u8(M, K), sa=f32(K // 128, M), qw=u8(E, N, K),
                                    sw=f32(E, N // 128, K // 128), offsets=off(), y=bf16(M, N)),
        fq.grouped_linear_dgrad: dict(qdy=u8(M, N), sdy=f32(N // 128, M), qwT=u8(K, E, N),
                                      sw=f32(E, N // 128, K // 128), offsets=off(),
                                      dx=bf16(M, K)),
        fq.grouped_linear_wgrad: dict(qdyT=u8(N, P), sdy_c=f32(P // 128, N), qxT=u8(K, P),
                                      sx_c=f32(P // 128, K), offsets=off(), dw=bf16(E, N, K)),
        fq.grouped_transpose_quant_bf16: dict(dy=bf16(M, N), offsets=off(), q_row=u8(M, N),
                                              s_row=f32(N // 128, M), q_colT=u8(N, P),
                                              s_col=f32(P // 128, N)),
        fq.grouped_transpose_quant_fp8: dict(q=u8(M, K), s=f32(K // 128, M), offsets=off(),
                                             qT=u8(K, P), sT=f32(P // 128, K)),
        fq.add_rmsnorm_quant: dict(x=bf16(M, K), res=bf16(M, K), gamma=bf16(K), eps=1e-5,
                                   h=bf16(M, K), q=u8(M, K), s=f32(K // 128, M)),
    }


WRONG = [
    (fq.grouped_linear_fwd, "qa", u8(M, K + 128)), (fq.grouped_linear_fwd, "sa", f32(K // 128, M - 4)),
    (fq.grouped_linear_fwd, "qw", u8(E * N, K)), (fq.grouped_linear_fwd, "sw", f32(E, K // 128, N // 128)),
    (fq.grouped_linear_fwd, "offsets", off(E + 1)), (fq.grouped_linear_fwd, "offsets", off().long()),
    (fq.grouped_linear_fwd, "y", bf16(M, K)), (fq.grouped_linear_fwd, "y", f32(M, N)),
    (fq.grouped_linear_fwd, "qw", u8(E, N, 2 * K)[:, :, ::2]),
    (fq.grouped_linear_dgrad, "qwT", u8(E, N, K)), (fq.grouped_linear_dgrad, "dx", bf16(M, N)),
    (fq.grouped_linear_dgrad, "sdy", f32(N // 128, M - 4)), (fq.grouped_linear_dgrad, "offsets", off(1)),
    (fq.grouped_linear_wgrad, "qdyT", u8(N, P - 64)), (fq.grouped_linear_wgrad, "qxT", u8(K, P + 128)),
    (fq.grouped_linear_wgrad, "sdy_c", f32(P // 128 + 1, N)), (fq.grouped_linear_wgrad, "sx_c", f32(P // 128, N)),
    (fq.grouped_linear_wgrad, "dw", bf16(E, K, N)), (fq.grouped_linear_wgrad, "offsets", off(E - 1)),
    (fq.grouped_transpose_quant_bf16, "q_row", u8(M + 1, N)), (fq.grouped_transpose_quant_bf16, "s_row", f32(1, M)),
    (fq.grouped_transpose_quant_bf16, "s_row", None),
    (fq.grouped_transpose_quant_bf16, "q_colT", u8(N, P + 1)), (fq.grouped_transpose_quant_bf16, "s_col", f32(P // 128, K)),
    (fq.grouped_transpose_quant_bf16, "offsets", torch.zeros(2 * E + 2, dtype=torch.int32)[::2]),
    (fq.grouped_transpose_quant_fp8, "s", f32(K // 128, M - 1)), (fq.grouped_transpose_quant_fp8, "qT", u8(N, P)),
    (fq.grouped_transpose_quant_fp8, "sT", f32(P // 128 - 1, K)),
    (fq.grouped_transpose_quant_fp8, "offsets", torch.zeros(1, dtype=torch.int32)),
    (fq.add_rmsnorm_quant, "res", bf16(M, K + 128)), (fq.add_rmsnorm_quant, "h", bf16(M + 1, K)),
    (fq.add_rmsnorm_quant, "gamma", bf16(K - 16)), (fq.add_rmsnorm_quant, "q", u8(K, M)),
    (fq.add_rmsnorm_quant, "s", f32(K // 128, M - 4)), (fq.add_rmsnorm_quant, "h", f32(M, K)),
]


@pytest.mark.parametrize("i", range(len(WRONG)),
                         ids=["%s-%s-%d" % (w[0].__name__, w[1], i) for i, w in enumerate(WRONG)])
def test_binding_refuses_a_mismatched_operand(i):
    fn, name, wrong = WRONG[i]
    args = good()[fn]
    args[name] = wrong
    with pytest.raises(ValueError, match=r"\b%s\b" % name):
        fn(**args)


@pytest.mark.parametrize("i", range(6))
def test_binding_accepts_matching_operands(i):
    fn, args = list(good().items())[i]
    with pytest.raises(ValueError, match="CUDA tensors"):
        fn(**args)


def test_grouped_quant_weight_refuses_ragged_weights():
    for shape in [(2, 200, 128), (2, 128, 192), (256, 128)]:
        with pytest.raises(ValueError, match=r"\bw\b"):
            fq.grouped_quant_weight_alloc(bf16(*shape))
