"""The expert layer on the GPU, against the oracle applied expert by expert: quantizers bit
for bit, products within one BF16 ulp + 1e-5 * sum |a b|, and bit for bit equal to the
dense entry points on each expert's rows. Row counts cover experts without rows, single
rows, groups that end inside a tile, exact multiples, and rows that belong to nobody
(never written)."""
import numpy as np
import pytest
import torch

import workloads
from gpu_util import (assert_codes_equal, assert_gemm_close, assert_scales_equal, bf16_values,
                      bits, np_f32, np_u8)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import fp8_block_scaled_08_b200 as f
    return f


# (rows before the first expert, rows of each expert, rows behind the last one)
ROUTINGS = {
    "one": (0, [1], 0),
    "single_expert": (0, [300], 0),
    "empty_ends": (0, [0, 5, 0, 0, 130, 0], 0),
    "ragged": (0, [1, 3, 257, 0, 128, 64, 31], 0),
    "spare": (3, [17, 0, 255, 2], 70),
    "exact": (0, [256, 128, 384], 0),
    "nobody": (0, [0, 0, 0], 40),
    "many": (0, [(7 * i) % 5 for i in range(70)], 1),
    "long": (1, [700, 1, 1300], 5),
}


def route(name):
    lead, counts, spare = ROUTINGS[name]
    off = np.concatenate([[0], np.cumsum(counts)]) + lead
    return off.astype(np.int32), int(off[-1]) + spare, len(counts)


def dev_offsets(off):
    return torch.tensor(off, dtype=torch.int32, device=DEV)


def owned(off, M):
    m = np.zeros(M, bool)
    m[off[0]:off[-1]] = True
    return m


def weights(fq, E, N, K, tid):
    w = workloads.normal_bf16((E, N, K), 0.02, 0, tid, DEV)
    return fq.grouped_quant_weight_alloc(w)


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


# ---------------------------------------------------------------- products

@pytest.mark.parametrize("N,K", [(128, 128), (384, 640), (256, 1152)])
@pytest.mark.parametrize("name", list(ROUTINGS))
def test_fwd(fq, oracle_mod, name, N, K):
    off, M, E = route(name)
    qw, sw, _ = weights(fq, E, N, K, 3000)
    x = workloads.activations_bf16((M, K), 0, 3001, DEV, outlier_count=4, outlier_scale=30.0)
    qa, sa = fq.quant_act_1x128_alloc(x)
    y = torch.full((M, N), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, sa, qw, sw, dev_offsets(off), y)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    assert torch.all(y[torch.tensor(~owned(off, M), device=DEV)] == 7.5)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        ref, ab = oracle_mod.linear_fwd(np_u8(qa[lo:hi]), np_f32(sa[:, lo:hi]), np_u8(qw[e]),
                                        np_f32(sw[e]))
        assert_gemm_close(bf16_values(y[lo:hi]), ref, ab, "expert %d" % e)
        qe, se = fq.quant_act_1x128_alloc(x[lo:hi].contiguous())
        assert same_bits(y[lo:hi], fq.linear_fwd_alloc(qe, se, qw[e], sw[e].clone())), e


@pytest.mark.parametrize("N,K", [(128, 128), (640, 384), (1152, 256)])
@pytest.mark.parametrize("name", list(ROUTINGS))
def test_dgrad(fq, oracle_mod, name, N, K):
    off, M, E = route(name)
    qw, sw, qwT = weights(fq, E, N, K, 3010)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3011, DEV, small_row_frac=0.1,
                                  small_row_scale=1e-3)
    q, s = fq.quant_act_1x128_alloc(dy)
    dx = torch.full((M, K), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_dgrad(q, s, qwT, sw, dev_offsets(off), dx)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    assert torch.all(dx[torch.tensor(~owned(off, M), device=DEV)] == 7.5)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        ref, ab = oracle_mod.linear_dgrad(np_u8(q[lo:hi]), np_f32(s[:, lo:hi]), np_u8(qw[e]),
                                          np_f32(sw[e]))
        assert_gemm_close(bf16_values(dx[lo:hi]), ref, ab, "expert %d" % e)
        qe, se = fq.quant_act_1x128_alloc(dy[lo:hi].contiguous())
        assert same_bits(dx[lo:hi], fq.linear_dgrad_alloc(qe, se, qwT[:, e].contiguous(), sw[e].clone())), e


@pytest.mark.parametrize("N,K", [(128, 128), (384, 640), (512, 256)])
@pytest.mark.parametrize("name", list(ROUTINGS))
def test_wgrad(fq, oracle_mod, name, N, K):
    off, M, E = route(name)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3020, DEV)
    x = workloads.activations_bf16((M, K), 0, 3021, DEV, outlier_count=4, outlier_scale=30.0)
    o = dev_offsets(off)
    _, _, qdyT, sdy = fq.grouped_transpose_quant_bf16_alloc(dy, o, want_row=False)
    qxT, sx = fq.grouped_transpose_quant_fp8_alloc(*fq.quant_act_1x128_alloc(x), o)
    dw = torch.full((E, N, K), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qdyT, sdy, qxT, sx, o, dw)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    g = 0
    for e in range(E):
        n = -(-int(off[e + 1] - off[e]) // 128)
        if n == 0:
            assert torch.all(dw[e] == 0), e
            continue
        a, sa = qdyT[:, 128 * g:128 * (g + n)].contiguous(), sdy[g:g + n].contiguous()
        b, sb = qxT[:, 128 * g:128 * (g + n)].contiguous(), sx[g:g + n].contiguous()
        ref, ab = oracle_mod.linear_wgrad(np_u8(a), np_f32(sa), np_u8(b), np_f32(sb))
        assert_gemm_close(bf16_values(dw[e]), ref, ab, "expert %d" % e)
        assert same_bits(dw[e], fq.linear_wgrad_alloc(a, sa, b, sb)), e
        g += n


@pytest.mark.parametrize("counts", [[1, 0, 9, 33, 2, 0, 0, 5], [30, 64, 1, 0, 67, 20, 31, 40],
                                    [128, 40, 129, 0, 100, 61, 90, 96]])
@pytest.mark.parametrize("N,K", [(640, 4224), (1280, 128), (2560, 384), (128, 8448)])
def test_products_over_strip_shapes(fq, counts, N, K):
    """Few rows per expert: every token-tile width, strip height and odd or long reduction,
    bit for bit the dense products."""
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1])
    o = dev_offsets(off)
    qw, sw, qwT = weights(fq, E, N, K, 3045)
    x = workloads.activations_bf16((M, K), 0, 3046, DEV)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3047, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)
    q, s = fq.quant_act_1x128_alloc(dy)
    y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    dx = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, sa, qw, sw, o, y)
    fq.grouped_linear_dgrad(q, s, qwT, sw, o, dx)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        qe, se = fq.quant_act_1x128_alloc(x[lo:hi].contiguous())
        assert same_bits(y[lo:hi], fq.linear_fwd_alloc(qe, se, qw[e], sw[e].clone())), e
        qe, se = fq.quant_act_1x128_alloc(dy[lo:hi].contiguous())
        assert same_bits(dx[lo:hi], fq.linear_dgrad_alloc(qe, se, qwT[:, e].contiguous(),
                                                          sw[e].clone())), e


@pytest.mark.parametrize("avg", [12, 40, 57, 100, 190, 230])
@pytest.mark.parametrize("N,K", [(1280, 640), (896, 1408)])
def test_products_over_many_tiles(fq, avg, N, K):
    """More tiles than SMs at every choice of kernel: 40 ragged experts, one of them without
    rows and one with a single row."""
    rng = np.random.RandomState(avg)
    counts = [int(c) for c in rng.randint(0, 2 * avg, 40)]
    counts[7], counts[23] = 0, 1
    test_products_over_strip_shapes(fq, counts, N, K)


def test_strided_outputs_and_wide_scales(fq):
    """Row strides of y and dx, and scale arrays longer than the rows."""
    off, M, E = route("ragged")
    N, K = 256, 384
    qw, sw, qwT = weights(fq, E, N, K, 3030)
    o = dev_offsets(off)
    x = workloads.activations_bf16((M, K), 0, 3031, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)
    ref = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, sa, qw, sw, o, ref)
    wide = torch.full((K // 128, M + 60), -1.0, device=DEV)
    wide[:, :M] = sa[:, :M]
    wide = torch.nn.functional.pad(wide, (0, -(M + 60) % 4)).contiguous()
    big = torch.full((M, N + 136), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, wide, qw, sw, o, big[:, 64:64 + N])
    assert same_bits(big[:, 64:64 + N].contiguous(), ref)
    assert torch.all(big[:, :64] == 7.5) and torch.all(big[:, 64 + N:] == 7.5)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3032, DEV)
    q, s = fq.quant_act_1x128_alloc(dy)
    ref = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_dgrad(q, s, qwT, sw, o, ref)
    big = torch.full((M, K + 8), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_dgrad(q, s, qwT, sw, o, big[:, 8:])
    assert same_bits(big[:, 8:].contiguous(), ref) and torch.all(big[:, :8] == 7.5)


@pytest.mark.parametrize("counts", [[2, 0, 1, 0, 3, 1, 1, 0], [16] * 8, [40, 9, 64, 65, 1, 0, 129, 33],
                                    [500, 2, 300, 40]])
def test_fwd_rows_do_not_depend_on_the_batch(fq, counts):
    """A row's bits are the same in a call of its own and in any batch (rollout and training
    share the product), whatever kernel the sizes select."""
    E, N, K = len(counts), 512, 1280
    qw, sw, qwT = weights(fq, E, N, K, 3040)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1])
    x = workloads.activations_bf16((M, K), 0, 3041, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)
    y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, sa, qw, sw, dev_offsets(off), y)
    for m in sorted({0, 1, M // 2, M - 1}):
        e = int(np.searchsorted(off, m, side="right")) - 1
        q1, s1 = fq.quant_act_1x128_alloc(x[m:m + 1].contiguous())
        o1 = torch.tensor([0] * (e + 1) + [1] * (E - e), dtype=torch.int32, device=DEV)
        y1 = torch.zeros((1, N), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_fwd(q1, s1, qw, sw, o1, y1)
        assert same_bits(y1, y[m:m + 1]), m


# ---------------------------------------------------------------- quantizers

@pytest.mark.parametrize("N", [16, 128, 400, 640])
@pytest.mark.parametrize("name", list(ROUTINGS))
def test_transpose_quant_bf16(fq, oracle_mod, name, N):
    off, M, E = route(name)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3050, DEV, small_row_frac=0.05,
                                  small_row_scale=1e-3)
    dy[:, N // 2] = 0                       # an all-zero column: scale 1
    if M > 2:
        dy[M // 2] = 0
    P = fq.grouped_padded_rows(M, E) + 128  # more columns than needed
    G = -(-N // 128)
    q = torch.full((M, N), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((G, fq.lds_for(M) + 4), -1.0, device=DEV)
    qT = torch.full((N, P), 77, dtype=torch.uint8, device=DEV)
    sT = torch.full((P // 128, N), -1.0, device=DEV)
    fq.grouped_transpose_quant_bf16(dy, dev_offsets(off), q, s, qT, sT)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    check_rows_and_columns(oracle_mod, dy, off, q, s, qT, sT)
    qT2, sT2 = torch.full_like(qT, 77), torch.full_like(sT, -1.0)
    fq.grouped_transpose_quant_bf16(dy, dev_offsets(off), None, None, qT2, sT2)
    assert torch.equal(qT2, qT) and torch.equal(sT2, sT)


def check_rows_and_columns(oracle_mod, dy, off, q, s, qT, sT):
    M = dy.shape[0]
    mask = owned(off, M)
    assert np.all(np_u8(q)[~mask] == 77) and np.all(np_f32(s)[:, :M][:, ~mask] == -1.0)
    assert np.all(np_f32(s)[:, M:] == -1.0)
    g = 0
    for e in range(len(off) - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        rq, rs, rqT, rsT = oracle_mod.transpose_quant_bf16(bits(dy[lo:hi]))
        n = -(-(hi - lo) // 128)
        assert_codes_equal(q[lo:hi], rq, "rows of %d" % e)
        assert_scales_equal(s[:, lo:hi], rs[:, :hi - lo], "row scales of %d" % e)
        assert_codes_equal(qT[:, 128 * g:128 * g + hi - lo], rqT, "columns of %d" % e)
        assert torch.all(qT[:, 128 * g + hi - lo:128 * (g + n)] == 0)
        assert_scales_equal(sT[g:g + n], rsT, "column scales of %d" % e)
        g += n
    assert torch.all(qT[:, 128 * g:] == 77) and torch.all(sT[g:] == -1.0)


@pytest.mark.parametrize("K", [16, 128, 400, 640])
@pytest.mark.parametrize("name", list(ROUTINGS))
def test_transpose_quant_fp8(fq, oracle_mod, name, K):
    off, M, E = route(name)
    x = workloads.activations_bf16((M, K), 0, 3060, DEV, outlier_count=2, outlier_scale=30.0)
    x[:, K // 2] = 0
    q, s = fq.quant_act_1x128_alloc(x)
    P = fq.grouped_padded_rows(M, E) + 128
    qT = torch.full((K, P), 77, dtype=torch.uint8, device=DEV)
    sT = torch.full((P // 128, K), -1.0, device=DEV)
    fq.grouped_transpose_quant_fp8(q, s, dev_offsets(off), qT, sT)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    g = 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        rqT, rsT = oracle_mod.transpose_quant_fp8(np_u8(q[lo:hi]), np.ascontiguousarray(np_f32(s)[:, lo:hi]))
        n = -(-(hi - lo) // 128)
        assert_codes_equal(qT[:, 128 * g:128 * g + hi - lo], rqT, "columns of %d" % e)
        assert torch.all(qT[:, 128 * g + hi - lo:128 * (g + n)] == 0)
        assert_scales_equal(sT[g:g + n], rsT, "column scales of %d" % e)
        g += n
    assert torch.all(qT[:, 128 * g:] == 77) and torch.all(sT[g:] == -1.0)


def test_tiny_scales(fq, oracle_mod):
    """Columns and rows whose scale is below 2^-80 take the kernels' division path, beside
    others that do not."""
    off, M, E = route("ragged")
    N = 384
    x = workloads.activations_bf16((M, N), 0, 3065, DEV)
    x[:, 5:300:7] *= 1e-30
    x[:, 128:256] *= 1e-33
    x[3:40] *= 1e-28
    o = dev_offsets(off)
    P = fq.grouped_padded_rows(M, E)
    q = torch.full((M, N), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((N // 128, fq.lds_for(M)), -1.0, device=DEV)
    qT = torch.full((N, P), 77, dtype=torch.uint8, device=DEV)
    sT = torch.full((P // 128, N), -1.0, device=DEV)
    fq.grouped_transpose_quant_bf16(x, o, q, s, qT, sT)
    check_rows_and_columns(oracle_mod, x, off, q, s, qT, sT)
    qa, sa = fq.quant_act_1x128_alloc(x)
    xT, xs = fq.grouped_transpose_quant_fp8_alloc(qa, sa, o)
    g = 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        rqT, rsT = oracle_mod.transpose_quant_fp8(np_u8(qa[lo:hi]),
                                                  np.ascontiguousarray(np_f32(sa)[:, lo:hi]))
        assert_codes_equal(xT[:, 128 * g:128 * g + hi - lo], rqT, "columns of %d" % e)
        n = -(-(hi - lo) // 128)
        assert_scales_equal(xs[g:g + n], rsT, "column scales of %d" % e)
        g += n


def test_huge_scales(fq, oracle_mod):
    """Values over 2^60 take the division path, beside ordinary ones and zeros."""
    off, M, E = route("spare")
    N = 272
    x = workloads.activations_bf16((M, N), 0, 3066, DEV)
    x[:, 3:200:5] *= 1e22
    x[10:30] *= 1e10
    x[40, :] = 0
    x[41, ::2] = -0.0
    o = dev_offsets(off)
    P = fq.grouped_padded_rows(M, E)
    q = torch.full((M, N), 77, dtype=torch.uint8, device=DEV)
    s = torch.full((-(-N // 128), fq.lds_for(M)), -1.0, device=DEV)
    qT = torch.full((N, P), 77, dtype=torch.uint8, device=DEV)
    sT = torch.full((P // 128, N), -1.0, device=DEV)
    fq.grouped_transpose_quant_bf16(x, o, q, s, qT, sT)
    check_rows_and_columns(oracle_mod, x, off, q, s, qT, sT)


def test_values_of_other_experts_do_not_leak(fq, oracle_mod):
    """NaN in the neighbours' rows (and in nobody's) changes nothing in an expert's groups."""
    off, M, E = route("spare")
    N = 256
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3070, DEV)
    o = dev_offsets(off)
    _, _, qT, sT = fq.grouped_transpose_quant_bf16_alloc(dy, o)
    lo, hi = int(off[2]), int(off[3])
    bad = torch.full_like(dy, float("nan"))
    bad[lo:hi] = dy[lo:hi]
    q2, s2, qT2, sT2 = fq.grouped_transpose_quant_bf16_alloc(bad, o)
    g0, g1 = 1, 1 + -(-(hi - lo) // 128)     # expert 0 has one group, expert 1 none
    assert torch.equal(qT[:, 128 * g0:128 * g1], qT2[:, 128 * g0:128 * g1])
    assert torch.equal(sT[g0:g1], sT2[g0:g1])
    rq, rs, _, _ = oracle_mod.transpose_quant_bf16(bits(dy[lo:hi]))
    assert_codes_equal(q2[lo:hi], rq)
    # and in the products: NaN codes in the rows around
    K = 384
    qw, sw, _ = weights(fq, E, N, K, 3071)
    qa, sa = fq.quant_act_1x128_alloc(workloads.activations_bf16((M, K), 0, 3172, DEV))
    y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, sa, qw, sw, o, y)
    qb, sb = torch.full_like(qa, 0x7F), torch.full_like(sa, float("nan"))
    qb[lo:hi] = qa[lo:hi]
    sb[:, lo:hi] = sa[:, lo:hi]
    y2 = torch.zeros_like(y)
    fq.grouped_linear_fwd(qb, sb, qw, sw, o, y2)
    assert same_bits(y[lo:hi], y2[lo:hi])


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("M,H", [(1, 128), (1, 16), (3, 4096), (5, 400), (33, 3584), (17, 5120),
                                 (9, 8192), (2, 16384), (7, 12304), (1100, 640), (1300, 2064),
                                 (1025, 4096), (2049, 5120), (1030, 8192), (1027, 8320)])
def test_add_rmsnorm(fq, oracle_mod, M, H):
    x = workloads.activations_bf16((M, H), 0, 3080, DEV, outlier_count=min(4, H // 16),
                                   outlier_scale=30.0)
    res = workloads.activations_bf16((M, H), 0, 3081, DEV)
    gamma = workloads.gamma_bf16(H, 0, 3082, DEV)
    h, q, s = fq.add_rmsnorm_quant_alloc(x, res, gamma, 1e-5)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    ref = (x.float() + res.float()).to(torch.bfloat16)
    assert same_bits(h, ref)
    rq, rs = oracle_mod.rmsnorm_quant(bits(ref), bits(gamma), 1e-5)
    assert_codes_equal(q, rq, "codes")
    assert_scales_equal(s, rs, "scales", cols=M)
    # the same bits as the norm of the stored stream
    q2, s2 = fq.rmsnorm_quant_alloc(h, gamma, 1e-5)
    assert torch.equal(q, q2) and torch.equal(s[:, :M], s2[:, :M])


@pytest.mark.parametrize("M", [6, 1500])
def test_add_rmsnorm_strides_and_in_place(fq, M):
    H = 1024
    wide = workloads.activations_bf16((M, 3 * H + 24), 0, 3090, DEV)
    x, res = wide[:, 8:8 + H], wide[:, 2 * H:3 * H]
    gamma = workloads.gamma_bf16(H, 0, 3091, DEV)
    h, q, s = fq.add_rmsnorm_quant_alloc(x.contiguous(), res.contiguous(), gamma, 1e-6)
    for target in ("apart", "x", "res", "columns"):
        w = wide.clone()
        xs, rs = w[:, 8:8 + H], w[:, 2 * H:3 * H]
        out = {"apart": torch.empty_like(h), "x": xs, "res": rs, "columns": w[:, H + 8:2 * H + 8]}[target]
        if target == "columns":
            out = w[:, H + 8:2 * H + 8][:, :H - 8]  # would overlap res: refused
            with pytest.raises((ValueError, fq.Fp8qError)):
                fq.add_rmsnorm_quant(xs, rs, gamma, 1e-6, w[:, H + 16:2 * H + 16], q, s)
            continue
        q1, s1 = torch.zeros_like(q), torch.full((H // 128, fq.lds_for(M) + 8), -1.0, device=DEV)
        fq.add_rmsnorm_quant(xs, rs, gamma, 1e-6, out, q1, s1)
        assert same_bits(out.contiguous(), h), target
        assert torch.equal(q1, q) and torch.equal(s1[:, :M], s[:, :M])
        assert torch.all(s1[:, M:] == -1.0)
        keep = torch.ones(w.shape[1], dtype=torch.bool, device=DEV)
        if target == "x":
            keep[8:8 + H] = False
        elif target == "res":
            keep[2 * H:3 * H] = False
        assert torch.equal(w[:, keep].view(torch.int16), wide[:, keep].view(torch.int16)), target


def test_add_rmsnorm_zero_rows_and_extremes(fq, oracle_mod):
    """Rows that cancel to zero (scale 1), tiny and huge values."""
    M, H = 12, 640
    x = workloads.activations_bf16((M, H), 0, 3100, DEV)
    res = workloads.activations_bf16((M, H), 0, 3101, DEV)
    res[0] = -x[0]
    x[1], res[1] = 1e-30, 1e-30
    x[2] *= 1e15
    x[3, :128] = 0
    res[3, :128] = 0
    gamma = workloads.gamma_bf16(H, 0, 3102, DEV)
    for eps in (0.0, 1e-5):
        xe, re = (x, res) if eps else (x[1:], res[1:])  # a zero row needs eps
        h, q, s = fq.add_rmsnorm_quant_alloc(xe.contiguous(), re.contiguous(), gamma, eps)
        ref = (xe.float() + re.float()).to(torch.bfloat16)
        assert same_bits(h, ref)
        rq, rs = oracle_mod.rmsnorm_quant(bits(ref), bits(gamma), eps)
        assert_codes_equal(q, rq)
        assert_scales_equal(s, rs, cols=xe.shape[0])


def test_add_rmsnorm_gradient(fq):
    """The documented backward: rmsnorm_bwd_quant_dual on h with the stream's gradient as
    dres gives the gradient of both addends, against 64-bit autograd of the formula and
    against central differences of it."""
    M, H = 128, 256
    x = workloads.activations_bf16((M, H), 0, 3110, DEV)
    res = workloads.activations_bf16((M, H), 0, 3111, DEV)
    gamma = workloads.gamma_bf16(H, 0, 3112, DEV)
    dy = workloads.gradients_bf16((M, H), 1.0, 0, 3113, DEV)
    dh = workloads.gradients_bf16((M, H), 1.0, 0, 3114, DEV)
    h, _, _ = fq.add_rmsnorm_quant_alloc(x, res, gamma, 1e-5)
    out = fq.rmsnorm_bwd_quant_dual_alloc(h, gamma, dy, dh, 1e-5)[0].double()

    def loss(a, b):  # the formula on the stored stream's point
        t = a + b
        y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-5) * gamma.double()
        return (y * dy.double()).sum() + (t * dh.double()).sum()

    a = (h.double() - res.double()).requires_grad_()
    b = res.double().requires_grad_()
    loss(a, b).backward()
    # two BF16 roundings (dx and out) and the fp32 steps: half a step each of |dx|, |out|
    dx = a.grad - dh.double()
    tol = 2.0 ** -8 * (dx.abs() + a.grad.abs()) + 1e-5 * (dx.abs() + dh.double().abs()) + 1e-6
    assert torch.all((out - a.grad).abs() <= tol)
    assert torch.all((out - b.grad).abs() <= tol)
    v = torch.randn(M, H, generator=torch.Generator(DEV).manual_seed(5), device=DEV, dtype=torch.float64)
    t = 1e-5
    with torch.no_grad():
        diff = (loss(a + t * v, b) - loss(a - t * v, b)) / (2 * t)
    assert abs(float(diff - (out * v).sum())) <= float((tol * v.abs()).sum())


# ---------------------------------------------------------------- together

def expert_mlp(fq, x, res, gamma, wgu, wd, o, dout):
    """Norm -> gate/up -> SwiGLU -> down of every expert, and the backward of the products;
    returns all that a training step keeps."""
    qgu, sgu, qguT = fq.grouped_quant_weight_alloc(wgu)
    qd, sd, qdT = fq.grouped_quant_weight_alloc(wd)
    E, H, I = wd.shape[0], wd.shape[1], wd.shape[2]
    M = x.shape[0]
    h, q, s = fq.add_rmsnorm_quant_alloc(x, res, gamma, 1e-5)
    gu = torch.zeros((M, 2 * I), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(q, s, qgu, sgu, o, gu)
    qh, sh = fq.swiglu_quant_alloc(gu)
    y = torch.zeros((M, H), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qh, sh, qd, sd, o, y)
    qr, sr, qc, sc = fq.grouped_transpose_quant_bf16_alloc(dout, o)
    dh = torch.zeros((M, I), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_dgrad(qr, sr, qdT, sd, o, dh)
    hT, hTs = fq.grouped_transpose_quant_fp8_alloc(qh, sh, o)
    dwd = torch.empty((E, H, I), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qc, sc, hT, hTs, o, dwd)
    return h, gu, y, dh, dwd


def mlp_inputs(M, H, I, E):
    return (workloads.activations_bf16((M, H), 0, 3120, DEV),
            workloads.activations_bf16((M, H), 0, 3121, DEV), workloads.gamma_bf16(H, 0, 3122, DEV),
            workloads.normal_bf16((E, 2 * I, H), 0.02, 0, 3123, DEV),
            workloads.normal_bf16((E, H, I), 0.02, 0, 3124, DEV),
            workloads.gradients_bf16((M, H), 1e-3, 0, 3125, DEV))


def test_expert_mlp_equals_the_dense_layer_per_expert(fq):
    off, M, E = route("ragged")
    H, I = 512, 256
    x, res, gamma, wgu, wd, dout = mlp_inputs(M, H, I, E)
    h, gu, y, dh, dwd = expert_mlp(fq, x, res, gamma, wgu, wd, dev_offsets(off), dout)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            assert torch.all(dwd[e] == 0)
            continue
        q, s = fq.rmsnorm_quant_alloc(h[lo:hi].contiguous(), gamma, 1e-5)
        qgu, sgu, _ = fq.quant_weight_alloc(wgu[e])
        qd, sd, qdT = fq.quant_weight_alloc(wd[e])
        g = fq.linear_fwd_alloc(q, s, qgu, sgu)
        assert same_bits(g, gu[lo:hi])
        qh, sh = fq.swiglu_quant_alloc(g)
        assert same_bits(fq.linear_fwd_alloc(qh, sh, qd, sd), y[lo:hi])
        qr, sr = fq.quant_act_1x128_alloc(dout[lo:hi].contiguous())
        assert same_bits(fq.linear_dgrad_alloc(qr, sr, qdT, sd), dh[lo:hi])


def test_products_are_the_gradients(fq):
    """DGrad and WGrad against differences of the bilinear form that the forward product
    computes, on the dequantized operands in 64 bits: L(x, W) = sum dy * (x W^T)."""
    off, M, E = route("ragged")
    N, K = 256, 384
    qw, sw, qwT = weights(fq, E, N, K, 3130)
    o = dev_offsets(off)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3131, DEV)
    x = workloads.activations_bf16((M, K), 0, 3132, DEV)
    qr, sr, qc, sc = fq.grouped_transpose_quant_bf16_alloc(dy, o)
    qxT, sx = fq.grouped_transpose_quant_fp8_alloc(*fq.quant_act_1x128_alloc(x), o)
    dx = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_dgrad(qr, sr, qwT, sw, o, dx)
    dw = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qc, sc, qxT, sx, o, dw)
    f8 = torch.float8_e4m3fn
    W = qw.view(f8).double() * sw.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    dyr = qr.view(f8).double() * sr[:, :M].double().t().repeat_interleave(128, 1)
    g = torch.Generator(DEV).manual_seed(7)
    lead = 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        n = -(-(hi - lo) // 128) * 128
        # direction in x: (L(x + v) - L(x - v)) / 2 = sum dy * (v W^T)
        v = torch.randn(hi - lo, K, generator=g, device=DEV, dtype=torch.float64)
        diff = (dyr[lo:hi] * (v @ W[e].t())).sum()
        ab = dyr[lo:hi].abs() @ W[e].abs()
        tol = ((2.0 ** -8 * dx[lo:hi].double().abs() + 1e-5 * ab) * v.abs()).sum()
        assert abs(float(diff - (dx[lo:hi].double() * v).sum())) <= float(tol) + 1e-30
        # direction in W
        dyc = qc[:, lead:lead + n].view(f8).double().t() * sc[lead // 128:(lead + n) // 128].double().repeat_interleave(128, 0)
        xc = qxT[:, lead:lead + n].view(f8).double().t() * sx[lead // 128:(lead + n) // 128].double().repeat_interleave(128, 0)
        v = torch.randn(N, K, generator=g, device=DEV, dtype=torch.float64)
        diff = (dyc * (xc @ v.t())).sum()
        ab = dyc.abs().t() @ xc.abs()
        tol = ((2.0 ** -8 * dw[e].double().abs() + 1e-5 * ab) * v.abs()).sum()
        assert abs(float(diff - (dw[e].double() * v).sum())) <= float(tol) + 1e-30
        lead += n


def test_captured_graph_follows_new_offsets(fq):
    """One capture, replayed with other routings written into the same offsets tensor, on a
    stream of its own; and two graphs that share nothing but the inputs."""
    M, H, I, E = 600, 256, 128, 5
    inputs = mlp_inputs(M, H, I, E)
    routings = [[100, 0, 300, 1, 150], [0, 0, 0, 600, 0], [1, 2, 3, 4, 5], [0, 0, 0, 0, 0]]
    offs = [torch.tensor(np.concatenate([[0], np.cumsum(r)]), dtype=torch.int32, device=DEV)
            for r in routings]
    want = [[t.clone() for t in expert_mlp(fq, *inputs[:5], o, inputs[5])] for o in offs]
    o = offs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        expert_mlp(fq, *inputs[:5], o, inputs[5])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(expert_mlp(fq, *inputs[:5], o, inputs[5]))
        graphs.append(g)
    for k in (1, 2, 3, 0):
        o.copy_(offs[k])
        for g, out in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want[k]):
                assert same_bits(a, b), k
    assert fq.device_error() == fq.FP8Q_OK


def test_capture_between_copies_and_joined_streams(fq):
    """Captured calls whose predecessors are copies, fills and events of another stream: the
    launches that overlap the kernel before them wait for those as well."""
    M, N, K, E = 400, 256, 384, 3
    qw, sw, _ = weights(fq, E, N, K, 3145)
    gamma = workloads.gamma_bf16(K, 0, 3146, DEV)
    o = dev_offsets(np.array([0, 128, 129, 400], np.int32))
    x = workloads.activations_bf16((M, K), 0, 3147, DEV)
    res = workloads.activations_bf16((M, K), 0, 3148, DEV)
    stage, h = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty((M, K), dtype=torch.uint8, device=DEV)
    s = torch.empty((K // 128, M), device=DEV)
    P = fq.grouped_padded_rows(M, E)
    t = torch.empty((K, P), dtype=torch.uint8, device=DEV)
    ts = torch.empty((P // 128, K), device=DEV)
    g_row, g_s = torch.empty((M, N), dtype=torch.uint8, device=DEV), torch.empty((2, M), device=DEV)
    c, cs = torch.empty((N, P), dtype=torch.uint8, device=DEV), torch.empty((P // 128, N), device=DEV)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    dw = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    main, other = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        stage.copy_(x)                                            # memcpy -> kernel
        fq.add_rmsnorm_quant(stage, res, gamma, 1e-5, h, q, s)
        stage.zero_()                                             # behind its reader
        other.wait_stream(torch.cuda.current_stream())            # fork
        y.zero_()
        fq.grouped_linear_fwd(q, s, qw, sw, o, y)
        with torch.cuda.stream(other):
            fq.grouped_transpose_quant_fp8(q, s, o, t, ts)
        fq.grouped_transpose_quant_bf16(y, o, g_row, g_s, c, cs)
        torch.cuda.current_stream().wait_stream(other)            # join
        fq.grouped_linear_wgrad(c, cs, t, ts, o, dw)
        q.fill_(0x7F)
        t.fill_(0x7F)
        c.fill_(0x7F)

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        step()
    torch.cuda.synchronize()
    hq, hs = fq.rmsnorm_quant_alloc((x.float() + res.float()).to(torch.bfloat16), gamma, 1e-5)
    want = [torch.zeros_like(y), torch.zeros_like(dw)]
    torch.cuda.synchronize()
    fq.grouped_linear_fwd(hq, hs, qw, sw, o, want[0])
    torch.cuda.synchronize()
    _, _, wc, wcs = fq.grouped_transpose_quant_bf16_alloc(want[0], o)
    wt, wts = fq.grouped_transpose_quant_fp8_alloc(hq, hs, o)
    torch.cuda.synchronize()
    fq.grouped_linear_wgrad(wc, wcs, wt, wts, o, want[1])
    torch.cuda.synchronize()
    assert same_bits(y, want[0]) and same_bits(dw, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        step()
    for _ in range(20):
        y.fill_(7.5)
        dw.fill_(7.5)
        torch.cuda.synchronize()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert same_bits(y, want[0]) and same_bits(dw, want[1])
    assert fq.device_error() == fq.FP8Q_OK


def test_two_streams_at_once(fq):
    off, M, E = route("long")
    N, K = 512, 640
    qw, sw, qwT = weights(fq, E, N, K, 3140)
    o = dev_offsets(off)
    x = workloads.activations_bf16((M, K), 0, 3141, DEV)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3142, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)
    q, s = fq.quant_act_1x128_alloc(dy)
    y0 = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    dx0 = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, sa, qw, sw, o, y0)
    fq.grouped_linear_dgrad(q, s, qwT, sw, o, dx0)
    y1, dx1 = torch.zeros_like(y0), torch.zeros_like(dx0)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        fq.grouped_linear_fwd(qa, sa, qw, sw, o, y1, stream=a)
        fq.grouped_linear_dgrad(q, s, qwT, sw, o, dx1, stream=b)
    torch.cuda.synchronize()
    assert same_bits(y0, y1) and same_bits(dx0, dx1)


@pytest.mark.parametrize("bad", [[0, 50, 20, 100], [0, 10, 20, 5000], [-7, 10, 20, 30],
                                 [90, 90, 10, 0], [2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1]])
def test_offsets_out_of_order_are_clamped_and_reported(fq, bad):
    """Device-side input: the kernels clamp it (as a running maximum within [0, M]) and the
    device error word says so; the results are those of the clamped offsets."""
    M, N, K, E = 100, 128, 256, 3
    fixed, run = [], 0
    for b in bad:
        run = min(max(b, run), M)
        fixed.append(run)
    qw, sw, qwT = weights(fq, E, N, K, 3150)
    x = workloads.activations_bf16((M, K), 0, 3151, DEV)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3152, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)

    def calls(o):
        y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_fwd(qa, sa, qw, sw, o, y)
        yield y.view(torch.int16)
        P = fq.grouped_padded_rows(M, E)
        q, s = torch.zeros((M, N), dtype=torch.uint8, device=DEV), torch.zeros((1, M), device=DEV)
        qT, sT = torch.zeros((N, P), dtype=torch.uint8, device=DEV), torch.zeros((P // 128, N), device=DEV)
        fq.grouped_transpose_quant_bf16(dy, o, q, s, qT, sT)
        yield torch.cat([t.view(torch.uint8).flatten() for t in (q, s, qT, sT)])
        dx = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_dgrad(q, s, qwT, sw, o, dx)
        yield dx.view(torch.int16)
        xT, xs = torch.zeros((K, P), dtype=torch.uint8, device=DEV), torch.zeros((P // 128, K), device=DEV)
        fq.grouped_transpose_quant_fp8(qa, sa, o, xT, xs)
        yield torch.cat([t.view(torch.uint8).flatten() for t in (xT, xs)])
        dw = torch.zeros((E, N, K), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_wgrad(qT, sT, xT, xs, o, dw)
        yield None  # WGrad clamps to its own columns: only that it reports and stays inside

    want = []
    for r in calls(torch.tensor(fixed, dtype=torch.int32, device=DEV)):
        assert fq.device_error() == fq.FP8Q_OK
        want.append(r)
    for r, w in zip(calls(torch.tensor(bad, dtype=torch.int32, device=DEV)), want):
        assert fq.device_error() == fq.FP8Q_ERR_OFFSETS
        assert w is None or torch.equal(r, w)
    assert fq.device_error() == fq.FP8Q_OK


def test_wgrad_drops_groups_past_its_columns(fq):
    """Operands with fewer columns than the offsets need: the groups past the end are left
    out and reported, the others are as they would be."""
    N, K, E = 128, 256, 3
    off = np.array([0, 130, 300, 420], np.int32)          # 2, 2 and 1 groups
    o = dev_offsets(off)
    M = int(off[-1])
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3185, DEV)
    x = workloads.activations_bf16((M, K), 0, 3186, DEV)
    _, _, c, cs = fq.grouped_transpose_quant_bf16_alloc(dy, o, want_row=False)
    t, ts = fq.grouped_transpose_quant_fp8_alloc(*fq.quant_act_1x128_alloc(x), o)
    dw = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(c, cs, t, ts, o, dw)
    assert fq.device_error() == fq.FP8Q_OK
    short = torch.full_like(dw, 7.5)
    P = 3 * 128                                           # expert 1 keeps one of two, 2 none
    fq.grouped_linear_wgrad(c[:, :P].contiguous(), cs[:3].contiguous(), t[:, :P].contiguous(),
                            ts[:3].contiguous(), o, short)
    assert fq.device_error() == fq.FP8Q_ERR_OFFSETS
    assert same_bits(short[0], dw[0]) and torch.all(short[2] == 0)
    one = fq.linear_wgrad_alloc(c[:, 256:P].contiguous(), cs[2:3].contiguous(),
                                t[:, 256:P].contiguous(), ts[2:3].contiguous())
    assert same_bits(short[1], one)


def test_elements_past_32_bits(fq):
    """Arrays of more than 2^31 elements: the last rows and columns against small calls."""
    M, wide, N, K = 70000, 32768, 128, 256
    counts = [M - 300, 300]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    o, lo = dev_offsets(off), int(off[1])
    o_last = dev_offsets(np.array([0, 0, 300], np.int32))
    qw, sw, qwT = weights(fq, 2, N, K, 3190)
    x = workloads.activations_bf16((M, K), 0, 3191, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)
    big = torch.zeros((M, wide), dtype=torch.bfloat16, device=DEV)   # 2.29e9 elements
    fq.grouped_linear_fwd(qa, sa, qw, sw, o, big[:, wide - N:])
    q1, s1 = fq.quant_act_1x128_alloc(x[lo:].contiguous())
    y1 = torch.zeros((300, N), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(q1, s1, qw, sw, o_last, y1)
    assert same_bits(big[lo:, wide - N:].contiguous(), y1)
    # the same rows through the strip kernel (few rows per expert of a large buffer)
    o_many = dev_offsets(np.concatenate([[lo] * 1000, [M] * 25]).astype(np.int32))
    many_w = qw[1:].expand(1024, N, K).contiguous()
    many_s = sw[1:].expand(1024, 1, K // 128).contiguous()
    big.zero_()
    fq.grouped_linear_fwd(qa, sa, many_w, many_s, o_many, big[:, wide - N:])
    assert same_bits(big[lo:, wide - N:].contiguous(), y1)
    assert fq.device_error() == fq.FP8Q_OK
    # quantizers: 2.29e9 codes each way
    for i in range(0, M, 7000):
        big[i:i + 7000].normal_()
    q, s, qT, sT = fq.grouped_transpose_quant_bf16_alloc(big, o)
    r = fq.grouped_transpose_quant_bf16_alloc(big[lo:].contiguous(), o_last)
    g0 = -(-lo // 128)
    assert torch.equal(q[lo:], r[0]) and torch.equal(s[:, lo:M], r[1][:, :300])
    assert torch.equal(qT[-3:, 128 * g0:128 * g0 + 384], r[2][-3:, :384])
    assert torch.equal(sT[g0:g0 + 3], r[3][:3])
    t, ts = fq.grouped_transpose_quant_fp8_alloc(q, s, o)
    s_last = torch.empty((wide // 128, 300), device=DEV)
    s_last.copy_(s[:, lo:M])
    t1, ts1 = fq.grouped_transpose_quant_fp8_alloc(q[lo:].contiguous(), s_last, o_last)
    assert torch.equal(t[-3:, 128 * g0:128 * g0 + 384], t1[-3:, :384])
    assert torch.equal(ts[g0:g0 + 3], ts1[:3])
    # the norm: rows of more than 2^31 elements in all, in place
    gamma = workloads.gamma_bf16(16384, 0, 3192, DEV)
    view = big[:, :16384]
    last = big[-5:, :16384].clone()
    qn = torch.empty((M, 16384), dtype=torch.uint8, device=DEV)
    sn = torch.empty((128, M), device=DEV)
    fq.add_rmsnorm_quant(view, view, gamma, 1e-5, view, qn, sn)
    h, q5, s5 = fq.add_rmsnorm_quant_alloc(last, last, gamma, 1e-5)
    assert same_bits(big[-5:, :16384].contiguous(), h) and torch.equal(qn[-5:], q5)
    assert torch.equal(sn[:, -5:], s5[:, :5]) and fq.device_error() == fq.FP8Q_OK


def test_most_experts(fq):
    """1024 experts (the table's limit), most of them without rows, against the same rows in
    a call with only the experts that have some."""
    E, N, K = 1024, 128, 256
    counts = np.zeros(E, np.int64)
    counts[[0, 3, 31, 32, 500, 1022, 1023]] = [2, 1, 140, 5, 33, 1, 7]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M, used = int(off[-1]), np.flatnonzero(counts)
    o = dev_offsets(off)
    o_used = dev_offsets(np.concatenate([[0], np.cumsum(counts[used])]).astype(np.int32))
    qw, sw, qwT = weights(fq, E, N, K, 3170)
    qw1, sw1 = qw[used].contiguous(), sw[used].contiguous()
    qwT1 = qwT[:, used].contiguous()
    x = workloads.activations_bf16((M, K), 0, 3171, DEV)
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3172, DEV)

    def run(qw, sw, qwT, o):
        qa, sa = fq.quant_act_1x128_alloc(x)
        y, dx = torch.zeros_like(dy), torch.zeros_like(x)
        fq.grouped_linear_fwd(qa, sa, qw, sw, o, y)
        qr, sr, qc, sc = fq.grouped_transpose_quant_bf16_alloc(dy, o)
        fq.grouped_linear_dgrad(qr, sr, qwT, sw, o, dx)
        xT, xs = fq.grouped_transpose_quant_fp8_alloc(qa, sa, o)
        dw = torch.empty((o.numel() - 1, N, K), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_wgrad(qc, sc, xT, xs, o, dw)
        torch.cuda.synchronize()
        assert fq.device_error() == fq.FP8Q_OK
        return y, dx, dw

    y, dx, dw = run(qw, sw, qwT, o)
    y1, dx1, dw1 = run(qw1, sw1, qwT1, o_used)
    assert same_bits(y, y1) and same_bits(dx, dx1) and same_bits(dw[used].contiguous(), dw1)
    rest = np.setdiff1d(np.arange(E), used)
    assert torch.all(dw[rest] == 0)
    with pytest.raises(ValueError):  # one more does not fit the table
        fq.grouped_transpose_quant_bf16_alloc(dy, torch.zeros(E + 2, dtype=torch.int32, device=DEV))


def test_calls_in_a_row_see_each_other(fq):
    """Kernels whose launches overlap the end of the one before: a stream updated in place
    forty times without a wait, a consumer after every step, inputs overwritten behind it."""
    M, H, N, E = 300, 1024, 256, 3
    x = workloads.activations_bf16((M, H), 0, 3180, DEV)
    gamma = workloads.gamma_bf16(H, 0, 3181, DEV)
    qw, sw, _ = weights(fq, E, N, H, 3182)
    o = dev_offsets(np.array([0, 100, 101, 300], np.int32))
    res = torch.zeros_like(x)
    q = torch.empty((M, H), dtype=torch.uint8, device=DEV)
    s = torch.empty((H // 128, M), device=DEV)
    ys = [torch.zeros((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(40)]
    for y in ys:
        fq.add_rmsnorm_quant(x, res, gamma, 1e-5, res, q, s)
        fq.grouped_linear_fwd(q, s, qw, sw, o, y)
        q.fill_(0x7F)
    want = torch.zeros_like(x)
    for y in ys:
        want = (want.float() + x.float()).to(torch.bfloat16)
        q1, s1 = fq.rmsnorm_quant_alloc(want, gamma, 1e-5)
        torch.cuda.synchronize()
        y1 = torch.zeros_like(y)
        fq.grouped_linear_fwd(q1, s1, qw, sw, o, y1)
        torch.cuda.synchronize()
        assert same_bits(y, y1)
    assert same_bits(res, want)


def test_no_rows_at_all(fq):
    M, N, K, E = 0, 256, 128, 3
    o = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    qw, sw, qwT = weights(fq, E, N, K, 3160)
    e = lambda *s, dt=torch.uint8: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    fq.grouped_linear_fwd(e(0, K), e(1, 4, dt=torch.float32), qw, sw, o, e(0, N, dt=torch.bfloat16))
    fq.grouped_linear_dgrad(e(0, N), e(2, 4, dt=torch.float32), qwT, sw, o, e(0, K, dt=torch.bfloat16))
    q, s, qT, sT = fq.grouped_transpose_quant_bf16_alloc(e(0, N, dt=torch.bfloat16), o)
    xT, xs = fq.grouped_transpose_quant_fp8_alloc(e(0, K), e(1, 4, dt=torch.float32), o)
    dw = torch.full((E, N, K), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qT, sT, xT, xs, o, dw)
    torch.cuda.synchronize()
    assert torch.all(dw == 0) and fq.device_error() == fq.FP8Q_OK
