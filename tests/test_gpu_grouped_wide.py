"""The expert layer's products at sizes where the large tiles (pairs of CTAs) take the call:
many rows per expert, rows of nobody around and between the boxes, more than eight column
panels; against the oracle, the dense entry points and the same rows in calls of their own,
which strips of weight rows take. Which kernel a call takes is read from a captured graph."""
import re
import warnings

import numpy as np
import pytest
import torch

import workloads
from gpu_util import assert_gemm_close, bf16_values, np_f32, np_u8
from test_gpu_grouped import dev_offsets, fq, same_bits, weights  # noqa: F401  (fq: fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAIR, STRIP = "gemm_kernel", "grouped_strip_kernel"


def kernel_of(call, tmp_path):
    """The product kernel that `call` launches: the function names of a captured graph."""
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    path = str(tmp_path / "graph.dot")
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # torch announces the dump
        g.enable_debug_mode()
        g.debug_dump(path)
    with open(path, errors="replace") as f:
        text = f.read()
    names = set(re.findall(r"grouped_strip_kernel|(?<!skinny_)gemm_kernel", text))
    assert len(names) == 1, names
    return names.pop()


def rows_around(counts, lead, spare):
    off = (np.concatenate([[0], np.cumsum(counts)]) + lead).astype(np.int32)
    return off, int(off[-1]) + spare


COUNTS = [517, 600, 0, 701, 530, 1, 633, 699, 545, 610, 661, 578]


def poisoned(q, s, off):
    """The rows of nobody: NaN codes and scales."""
    q, s = q.clone(), s.clone()
    for a, b in ((0, int(off[0])), (int(off[-1]), q.shape[0])):
        q[a:b] = 0x7F
        s[:, a:b] = float("nan")
    return q, s


@pytest.mark.parametrize("lead,spare,wide", [(3, 70, 0), (0, 0, 0), (33, 1, 8), (256, 700, 136)])
@pytest.mark.parametrize("dgrad", [False, True])
def test_large_tiles(fq, oracle_mod, tmp_path, lead, spare, wide, dgrad):  # noqa: F811
    """Experts that start and end anywhere in a box of 32 rows; nothing else is written,
    beside the rows or (row stride over the width) beside the columns."""
    off, M = rows_around(COUNTS, lead, spare)
    E, red, out = len(COUNTS), 256 if dgrad else 384, 1152  # reduction, width of the output
    qw, sw, qwT = weights(fq, E, red, out, 3301) if dgrad else weights(fq, E, out, red, 3300)
    o = dev_offsets(off)
    a = (workloads.gradients_bf16((M, red), 1e-3, 0, 3302, DEV) if dgrad
         else workloads.activations_bf16((M, red), 0, 3302, DEV))
    qa, sa = fq.quant_act_1x128_alloc(a)
    qa, sa = poisoned(qa, sa, off)
    big = torch.full((M, out + wide), 7.5, dtype=torch.bfloat16, device=DEV)
    y = big[:, wide // 2:wide // 2 + out] if wide % 16 == 0 else big[:, wide:]
    product = fq.grouped_linear_dgrad if dgrad else fq.grouped_linear_fwd
    w = qwT if dgrad else qw
    product(qa, sa, w, sw, o, y)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    left = torch.ones_like(big, dtype=torch.bool)
    at = y.storage_offset()
    left[off[0]:off[-1], at:at + out] = False
    assert torch.all(big[left] == 7.5)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        qe, se = fq.quant_act_1x128_alloc(a[lo:hi].contiguous())
        we = qwT[:, e].contiguous() if dgrad else qw[e]
        dense = (fq.linear_dgrad_alloc if dgrad else fq.linear_fwd_alloc)(qe, se, we, sw[e].clone())
        assert same_bits(y[lo:hi].contiguous(), dense), e
        if e in (1, 5, 11):
            ref, ab = (oracle_mod.linear_dgrad if dgrad else oracle_mod.linear_fwd)(
                np_u8(qe), np_f32(se[:, :hi - lo]), np_u8(qw[e]), np_f32(sw[e]))
            assert_gemm_close(bf16_values(y[lo:hi]), ref, ab, "expert %d" % e)

    def alone(m):  # one row in a call of its own
        e = int(np.searchsorted(off, m, side="right")) - 1
        o1 = torch.tensor([0] * (e + 1) + [1] * (E - e), dtype=torch.int32, device=DEV)
        q1, s1 = fq.quant_act_1x128_alloc(a[m:m + 1].contiguous())
        y1 = torch.zeros((1, out), dtype=torch.bfloat16, device=DEV)
        return lambda: product(q1, s1, w, sw, o1, y1), y1

    for m in (int(off[0]), int(off[1]) - 1, int(off[1]), int(off[5]), int(off[-1]) - 1):
        call, y1 = alone(m)
        call()
        assert same_bits(y1, y[m:m + 1].contiguous()), m
    assert kernel_of(lambda: product(qa, sa, w, sw, o, y), tmp_path) == PAIR
    assert kernel_of(alone(int(off[1]))[0], tmp_path) == STRIP


@pytest.mark.parametrize("width", [2304, 2688])
def test_many_column_panels(fq, tmp_path, width):  # noqa: F811
    """Nine panels (the second group of panels holds one) and eleven, the last one half
    full: forward, DGrad and WGrad, bit for bit the dense products."""
    off, M = rows_around([300, 0, 411, 260], 5, 9)
    E, other = 4, 384
    o = dev_offsets(off)
    x = workloads.activations_bf16((M, other), 0, 3310, DEV)
    dy = workloads.gradients_bf16((M, other), 1e-3, 0, 3311, DEV)
    wide = workloads.activations_bf16((M, width), 0, 3312, DEV)
    qw, sw, _ = weights(fq, E, width, other, 3313)
    _, sv, qvT = weights(fq, E, other, width, 3314)
    qx, sx = fq.quant_act_1x128_alloc(x)
    q, s = fq.quant_act_1x128_alloc(dy)
    y = torch.full((M, width), 7.5, dtype=torch.bfloat16, device=DEV)
    dx = torch.full_like(y, 7.5)
    dw = torch.full((E, other, width), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qx, sx, qw, sw, o, y)
    fq.grouped_linear_dgrad(q, s, qvT, sv, o, dx)
    _, _, qdyT, sdy = fq.grouped_transpose_quant_bf16_alloc(dy, o, want_row=False)
    qT, sT = fq.grouped_transpose_quant_fp8_alloc(*fq.quant_act_1x128_alloc(wide), o)
    fq.grouped_linear_wgrad(qdyT, sdy, qT, sT, o, dw)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    rest = torch.ones(M, dtype=torch.bool, device=DEV)
    rest[off[0]:off[-1]] = False
    assert torch.all(y[rest] == 7.5) and torch.all(dx[rest] == 7.5)
    g = 0
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            assert torch.all(dw[e] == 0)
            continue
        qe, se = fq.quant_act_1x128_alloc(x[lo:hi].contiguous())
        assert same_bits(y[lo:hi], fq.linear_fwd_alloc(qe, se, qw[e], sw[e].clone())), e
        qe, se = fq.quant_act_1x128_alloc(dy[lo:hi].contiguous())
        assert same_bits(dx[lo:hi], fq.linear_dgrad_alloc(qe, se, qvT[:, e].contiguous(),
                                                          sv[e].clone())), e
        n = -(-(hi - lo) // 128)
        p = slice(128 * g, 128 * (g + n))
        assert same_bits(dw[e], fq.linear_wgrad_alloc(
            qdyT[:, p].contiguous(), sdy[g:g + n].contiguous(), qT[:, p].contiguous(),
            sT[g:g + n].contiguous())), e
        g += n
    assert kernel_of(lambda: fq.grouped_linear_fwd(qx, sx, qw, sw, o, y), tmp_path) == PAIR
    assert kernel_of(lambda: fq.grouped_linear_dgrad(q, s, qvT, sv, o, dx), tmp_path) == PAIR


def test_a_few_rows_in_buffers_of_many(fq, tmp_path):  # noqa: F811
    """Buffers that hold the worst case, most of their rows nobody's: the large tiles take
    the call (the choice goes by the buffers), with the bits of a call with exact buffers."""
    E, N, K, M = 4, 1280, 256, 4000
    qw, sw, _ = weights(fq, E, N, K, 3320)
    x = workloads.activations_bf16((M, K), 0, 3321, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)
    for counts in ([3, 0, 1, 7], [0, 0, 0, 0], [0, 33, 0, 0]):
        off, rows = rows_around(counts, 0, 0)
        o = dev_offsets(off)
        y = torch.full((M, N), 7.5, dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_fwd(qa, sa, qw, sw, o, y)
        assert torch.all(y[rows:] == 7.5)
        if rows:
            q1, s1 = fq.quant_act_1x128_alloc(x[:rows].contiguous())
            y1 = torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
            fq.grouped_linear_fwd(q1, s1, qw, sw, o, y1)
            assert same_bits(y[:rows], y1)
            assert kernel_of(lambda: fq.grouped_linear_fwd(q1, s1, qw, sw, o, y1), tmp_path) == STRIP
        assert kernel_of(lambda: fq.grouped_linear_fwd(qa, sa, qw, sw, o, y), tmp_path) == PAIR
    assert fq.device_error() == fq.FP8Q_OK


def test_calls_repeat_themselves(fq):  # noqa: F811
    """The same call again, with calls on other operands between: the same bits."""
    off, M = rows_around([700, 1, 0, 1300, 517], 2, 6)
    E, N, K = 5, 640, 512
    o, o2 = dev_offsets(off), dev_offsets(rows_around([1, 900, 700, 0, 900], 0, 0)[0])
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3330, DEV)
    x = workloads.activations_bf16((M, K), 0, 3331, DEV)
    qw, sw, qwT = weights(fq, E, N, K, 3332)

    def step(o, dy, x):
        qa, sa = fq.quant_act_1x128_alloc(x)
        y = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_fwd(qa, sa, qw, sw, o, y)
        qr, sr, qc, sc = fq.grouped_transpose_quant_bf16_alloc(dy, o)
        dx = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_dgrad(qr, sr, qwT, sw, o, dx)
        xT, xs = fq.grouped_transpose_quant_fp8_alloc(qa, sa, o)
        dw = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_wgrad(qc, sc, xT, xs, o, dw)
        return y, dx, dw

    first = step(o, dy, x)
    for _ in range(10):
        step(o2, dy.flip(0), x.flip(0))
        for a, b in zip(step(o, dy, x), first):
            assert same_bits(a, b)


def test_nan_scales_beside_an_expert(fq):  # noqa: F811
    """NaN or infinite scales (and codes) in the rows of other experts, of nobody and behind
    the last expert change nothing in an expert's requantized groups."""
    counts = [130, 61, 0, 1, 255, 128]
    off, M = rows_around(counts, 3, 70)
    K, o = 272, dev_offsets(off)
    q, s = fq.quant_act_1x128_alloc(workloads.activations_bf16((M, K), 0, 3340, DEV))
    qT, sT = fq.grouped_transpose_quant_fp8_alloc(q, s, o)
    g = 0
    for e, n in enumerate(counts):
        lo, hi, k = int(off[e]), int(off[e + 1]), -(-n // 128)
        for bad in (float("nan"), float("inf")):
            q2, s2 = torch.full_like(q, 0x7F), torch.full_like(s, bad)
            if bad == float("inf"):
                q2[:lo], q2[hi:] = q[:lo], q[hi:]
            q2[lo:hi], s2[:, lo:hi] = q[lo:hi], s[:, lo:hi]
            qT2, sT2 = fq.grouped_transpose_quant_fp8_alloc(q2, s2, o)
            assert torch.equal(qT2[:, 128 * g:128 * (g + k)], qT[:, 128 * g:128 * (g + k)]), (e, bad)
            assert torch.equal(sT2[g:g + k], sT[g:g + k]), (e, bad)
        g += k
    assert fq.device_error() == fq.FP8Q_OK


def test_outputs_on_another_stream_do_not_meet_a_freed_block(fq):  # noqa: F811
    """A block that the current stream still writes when it is freed is not what a call on
    another stream gets for its outputs."""
    M, H = 256, 1024
    x = workloads.activations_bf16((M, H), 0, 3350, DEV)
    res = workloads.activations_bf16((M, H), 0, 3351, DEV)
    gamma = workloads.gamma_bf16(H, 0, 3352, DEV)
    want = [t.clone() for t in fq.add_rmsnorm_quant_alloc(x, res, gamma, 1e-5)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(20_000_000)  # about 10 ms of the current stream
    for t in old:
        t.fill_(1)
    del old, t
    got = fq.add_rmsnorm_quant_alloc(x, res, gamma, 1e-5, stream=side)
    torch.cuda.synchronize()
    assert same_bits(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[2], want[2])


def test_weights_past_32_bits(fq):  # noqa: F811
    """More than 2^31 codes of stacked weights (and elements of dW): the last expert."""
    E, N, K, n = 132, 4096, 4096, 70
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w[e].normal_(std=0.02)
    qw, sw, qwT = fq.grouped_quant_weight_alloc(w)
    q1, s1, q1T = fq.quant_weight_alloc(w[-1])
    assert torch.equal(qw[-1], q1) and torch.equal(sw[-1], s1) and torch.equal(qwT[:, -1], q1T)
    del w
    o = torch.tensor([0] * E + [n], dtype=torch.int32, device=DEV)
    x = workloads.activations_bf16((n, K), 0, 3360, DEV)
    dy = workloads.gradients_bf16((n, N), 1e-3, 0, 3361, DEV)
    qa, sa = fq.quant_act_1x128_alloc(x)
    qr, sr, qc, sc = fq.grouped_transpose_quant_bf16_alloc(dy, o)
    xT, xs = fq.grouped_transpose_quant_fp8_alloc(qa, sa, o)
    y = torch.zeros((n, N), dtype=torch.bfloat16, device=DEV)
    dx = torch.zeros((n, K), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qa, sa, qw, sw, o, y)
    fq.grouped_linear_dgrad(qr, sr, qwT, sw, o, dx)
    dw = torch.full((E, N, K), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qc, sc, xT, xs, o, dw)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    assert same_bits(y, fq.linear_fwd_alloc(qa, sa, q1, s1))
    assert same_bits(dx, fq.linear_dgrad_alloc(qr, sr, q1T, s1))
    assert not torch.any(dw[:-1].view(torch.int16))
    p = slice(0, 128)
    assert same_bits(dw[-1], fq.linear_wgrad_alloc(qc[:, p].contiguous(), sc[:1].contiguous(),
                                                   xT[:, p].contiguous(), xs[:1].contiguous()))
    # many rows of the last expert: the large tiles
    M = 200 * E
    o = torch.tensor([0] * E + [M], dtype=torch.int32, device=DEV)
    q2, s2 = fq.quant_act_1x128_alloc(x.repeat(M // n + 1, 1)[:M].contiguous())
    y2 = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(q2, s2, qw, sw, o, y2)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    assert same_bits(y2[:n], y) and same_bits(y2[M - M % n:], y[:M % n])


def test_wgrad_checks_the_order_and_its_columns(fq):  # noqa: F811
    """What WGrad notices of wrong offsets, as documented: it does not know the rows, so
    entries beyond them pass where their groups fit the columns (the quantizers report them);
    without columns it reads no offsets."""
    N, K, E, M = 128, 256, 3, 100
    off = [0, 40, 60, 100]
    dy = workloads.gradients_bf16((M, N), 1e-3, 0, 3370, DEV)
    qa, sa = fq.quant_act_1x128_alloc(workloads.activations_bf16((M, K), 0, 3371, DEV))
    P = fq.grouped_padded_rows(M, E) + 256
    new = lambda *n, dt=torch.uint8: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
    qdyT, sdy, qxT, sx = new(N, P), new(P // 128, N, dt=torch.float32), new(K, P), new(P // 128, K, dt=torch.float32)

    def wgrad(off):
        dw = torch.full((E, N, K), 7.5, dtype=torch.bfloat16, device=DEV)
        fq.grouped_linear_wgrad(qdyT, sdy, qxT, sx, dev_offsets(np.array(off, np.int32)), dw)
        return dw

    o = dev_offsets(np.array(off, np.int32))
    fq.grouped_transpose_quant_bf16(dy, o, None, None, qdyT, sdy)
    fq.grouped_transpose_quant_fp8(qa, sa, o, qxT, sx)
    want = wgrad(off)
    assert fq.device_error() == fq.FP8Q_OK
    beyond = wgrad([0, 40, 60, 300])                        # past M, within P: zero columns here
    assert fq.device_error() == fq.FP8Q_OK and same_bits(beyond, want)
    fq.grouped_transpose_quant_fp8(qa, sa, dev_offsets(np.array([0, 40, 60, 300], np.int32)), qxT, sx)
    assert fq.device_error() == fq.FP8Q_ERR_OFFSETS
    for bad in ([0, 60, 40, 100], [-1, 40, 60, 100], [0, 40, 60, 60 + P]):
        wgrad(bad)
        assert fq.device_error() == fq.FP8Q_ERR_OFFSETS, bad
    dw = torch.full((E, N, K), 7.5, dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qdyT[:, :0], sdy[:0], qxT[:, :0], sx[:0], o, dw)
    assert fq.device_error() == fq.FP8Q_OK and torch.all(dw == 0)


def test_which_kernel_a_call_takes(fq, tmp_path):  # noqa: F811
    """Strips up to 128 rows per expert, the large tiles above, where one tile per SM does not
    hold the whole product."""
    E, N, K = 12, 1152, 256
    qw, sw, qwT = weights(fq, E, N, K, 3380)
    new = lambda *n, dt=torch.uint8: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
    for M, kernel in ((1, STRIP), (16 * E + 1, STRIP), (100 * E, STRIP), (128 * E, STRIP),
                      (128 * E + 1, PAIR), (160 * E, PAIR), (500 * E, PAIR)):
        o = torch.tensor([i * M // E for i in range(E + 1)], dtype=torch.int32, device=DEV)
        q, s, y = new(M, K), new(K // 128, fq.lds_for(M), dt=torch.float32), new(M, N, dt=torch.bfloat16)
        assert kernel_of(lambda: fq.grouped_linear_fwd(q, s, qw, sw, o, y), tmp_path) == kernel, M
