"""The expert layer as a program uses it: the norm's backward over a ragged number of rows, and
a whole routed step (norm, router, gather by expert, both products and SwiGLU, combination;
then the gradients of all of it)."""
import numpy as np
import pytest
import torch

import workloads
from test_gpu_grouped import dev_offsets, fq, same_bits  # noqa: F401  (fq: fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


def up128(n):
    return -(-n // 128) * 128


def norm_backward(fq, h, gamma, dy, dh):  # noqa: F811
    """The gradient of both addends, and of gamma, for buffers h, dy, dh of a multiple of 128
    rows, the ones behind the last token zero."""
    out, _, _, _, _, dgamma = fq.rmsnorm_bwd_quant_dual_alloc(h, gamma, dy, dh, EPS)
    return out, dgamma


def check_norm_gradient(h, gamma, dy, dh, out, dgamma):
    """Against 64-bit autograd of the formula at the stored stream."""
    t = h.double().requires_grad_()
    g = gamma.double().requires_grad_()
    y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * g
    ((y * dy.double()).sum() + (t * dh.double()).sum()).backward()
    dx = t.grad - dh.double()
    # two BF16 roundings (dx and out: half a step each) and the fp32 steps, whose terms
    # r gamma dy and k x can cancel: k = r^3 <gamma dy, x> / H
    r = torch.rsqrt(h.double().square().mean(1, keepdim=True) + EPS)
    k = r ** 3 * (gamma.double() * dy.double() * h.double()).abs().mean(1, keepdim=True)
    terms = (r * gamma.double() * dy.double()).abs() + (k * h.double()).abs()
    tol = 2.0 ** -8 * (dx.abs() + t.grad.abs()) + 2.0 ** -20 * (terms + dh.double().abs()) + 1e-30
    assert torch.all((out.double() - t.grad).abs() <= tol)
    # exact sum of products of three fp32 roundings (and r's), rounded once
    ab = (dy.double() * h.double() * r).abs().sum(0)
    assert torch.all((dgamma.double() - g.grad).abs() <= 2.0 ** -22 * ab + 1e-30)


@pytest.mark.parametrize("M", [1, 77, 200])
def test_norm_backward_of_ragged_rows(fq, M):  # noqa: F811
    H, P = 384, up128(M)
    x = workloads.activations_bf16((M, H), 0, 3400, DEV)
    res = workloads.activations_bf16((M, H), 0, 3401, DEV)
    gamma = workloads.gamma_bf16(H, 0, 3402, DEV)
    h = torch.zeros((P, H), dtype=torch.bfloat16, device=DEV)
    dy, dh = torch.zeros_like(h), torch.zeros_like(h)
    dy[:M] = workloads.gradients_bf16((M, H), 1.0, 0, 3403, DEV)
    dh[:M] = workloads.gradients_bf16((M, H), 1.0, 0, 3404, DEV)
    q = torch.empty((M, H), dtype=torch.uint8, device=DEV)
    s = torch.empty((H // 128, fq.lds_for(M)), device=DEV)
    fq.add_rmsnorm_quant(x, res, gamma, EPS, h[:M], q, s)
    assert same_bits(h[:M], (x.float() + res.float()).to(torch.bfloat16))
    out, dgamma = norm_backward(fq, h, gamma, dy, dh)
    torch.cuda.synchronize()
    assert torch.all(out[M:] == 0) and fq.device_error() == fq.FP8Q_OK
    check_norm_gradient(h[:M], gamma, dy[:M], dh[:M], out[:M], dgamma)
    # the rows do not depend on those behind them: the same rows below others
    if M < 128:
        more = torch.cat([h[:M], h[:128 - M]]) if 2 * M >= 128 else None
        if more is not None:
            full = norm_backward(fq, more, gamma, torch.cat([dy[:M], dy[:128 - M]]),
                                 torch.cat([dh[:M], dh[:128 - M]]))[0]
            assert same_bits(full[:M], out[:M])


def test_norm_backward_refuses_other_multiples(fq):  # noqa: F811
    e = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    assert fq.rmsnorm_bwd_workspace_bytes(77, 256) == -1
    for M, H in ((77, 256), (128, 272)):
        with pytest.raises(fq.Fp8qError, match="FP8Q_ERR_SHAPE"):
            fq.rmsnorm_bwd_quant_dual_alloc(e(M, H), e(H), e(M, H), None, EPS)


def test_a_rank_without_tokens(fq):  # noqa: F811
    """No rows: the norm returns, as the grouped calls do, and its checks stay."""
    e = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    h, q, s = fq.add_rmsnorm_quant_alloc(e(0, 256), e(0, 256), e(256), EPS)
    assert h.shape == q.shape == (0, 256) and s.shape == (2, 4)
    with pytest.raises(ValueError, match="gamma"):
        fq.add_rmsnorm_quant_alloc(e(0, 256), e(0, 256), e(128), EPS)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK


# ---------------------------------------------------------------- a routed step

def route_top2(logits, E):
    """Two experts of each token: (row -> token, weight of the row, offsets), rows sorted by
    expert."""
    weight, expert = torch.softmax(logits.float(), 1).topk(2, dim=1)
    order = expert.flatten().sort(stable=True).indices
    counts = torch.bincount(expert.flatten(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return order // 2, weight.flatten()[order], offsets


def gather_rows(fq, q, s, token):  # noqa: F811
    """Codes and 1x128 scales of the rows `token`: a token sent to two experts comes twice."""
    R = token.numel()
    sg = torch.zeros((s.shape[0], fq.lds_for(R)), device=DEV)
    sg[:, :R] = s[:, token]
    return q[token], sg


def add_by_token(rows, token, T):
    """Sum of each token's rows in fp32, rounded once."""
    return torch.zeros((T, rows.shape[1]), device=DEV).index_add_(0, token, rows.float()).to(torch.bfloat16)


def routed_step(fq, x, res, gamma, wr, wgu, wd, dout):  # noqa: F811
    """Forward and backward of a layer of E experts, two per token; dout is the gradient of
    the layer's output, res + ... + experts. Returns everything a training step keeps."""
    (T, H), (E, _, I) = x.shape, wd.shape
    P = up128(T)
    qgu, sgu, qguT = fq.grouped_quant_weight_alloc(wgu)
    qd, sd, qdT = fq.grouped_quant_weight_alloc(wd)
    h = torch.zeros((P, H), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((T, H), dtype=torch.uint8, device=DEV)
    s = torch.empty((H // 128, fq.lds_for(T)), device=DEV)
    fq.add_rmsnorm_quant(x, res, gamma, EPS, h[:T], q, s)
    normed = q.view(torch.float8_e4m3fn).float() * s[:, :T].t().repeat_interleave(128, 1)
    token, weight, o = route_top2(normed @ wr, E)
    R = token.numel()
    qg, sg = gather_rows(fq, q, s, token)
    gu = torch.zeros((up128(R), 2 * I), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qg, sg, qgu, sgu, o, gu[:R])
    qh, sh = fq.swiglu_quant_alloc(gu[:R])
    y = torch.zeros((R, H), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_fwd(qh, sh, qd, sd, o, y)
    out = add_by_token(y * weight[:, None].to(torch.bfloat16), token, T)
    # backward: down projection
    dy = dout[token] * weight[:, None].to(torch.bfloat16)
    qr, sr, qc, sc = fq.grouped_transpose_quant_bf16_alloc(dy, o)
    dh = torch.zeros((up128(R), I), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_dgrad(qr, sr, qdT, sd, o, dh[:R])
    dwd = torch.empty((E, H, I), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qc, sc, *fq.grouped_transpose_quant_fp8_alloc(qh, sh, o), o, dwd)
    # SwiGLU (rows behind R are zero), gate and up projections
    dgu = fq.swiglu_bwd_quant_dual_alloc(gu, dh, want_dgu=True)[4]
    qr, sr, qc, sc = fq.grouped_transpose_quant_bf16_alloc(dgu[:R], o)
    dx = torch.zeros((R, H), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_dgrad(qr, sr, qguT, sgu, o, dx)
    dwgu = torch.empty((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
    fq.grouped_linear_wgrad(qc, sc, *fq.grouped_transpose_quant_fp8_alloc(qg, sg, o), o, dwgu)
    # the norm
    dn, dres = torch.zeros_like(h), torch.zeros_like(h)
    dn[:T] = add_by_token(dx, token, T)
    dres[:T] = dout
    grad, dgamma = norm_backward(fq, h, gamma, dn, dres)
    return dict(h=h[:T], q=q, s=s, token=token, weight=weight, o=o, gu=gu[:R], qh=qh, sh=sh, y=y,
                out=out, dy=dy, dh=dh[:R], dwd=dwd, dgu=dgu[:R], dx=dx, dwgu=dwgu, dn=dn[:T],
                grad=grad[:T], dgamma=dgamma)


def step_inputs(T, H, I, E):
    return (workloads.activations_bf16((T, H), 0, 3410, DEV),
            workloads.activations_bf16((T, H), 0, 3411, DEV), workloads.gamma_bf16(H, 0, 3412, DEV),
            torch.randn(H, E, generator=torch.Generator(DEV).manual_seed(9), device=DEV) * 0.1,
            workloads.normal_bf16((E, 2 * I, H), 0.02, 0, 3413, DEV),
            workloads.normal_bf16((E, H, I), 0.02, 0, 3414, DEV),
            workloads.gradients_bf16((T, H), 1e-2, 0, 3415, DEV))


@pytest.mark.parametrize("T,E", [(1, 8), (5, 16), (203, 6), (1500, 12)])
def test_routed_step(fq, T, E):  # noqa: F811
    """Every product and quantizer equals the dense one over the expert's rows alone, the
    gradients of the weights and of the norm are those of the formulas."""
    H, I = 384, 256
    inputs = step_inputs(T, H, I, E)
    x, res, gamma, _, wgu, wd, dout = inputs
    r = routed_step(fq, *inputs)
    torch.cuda.synchronize()
    assert fq.device_error() == fq.FP8Q_OK
    off = r["o"].tolist()
    assert off[-1] == 2 * T
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            assert torch.all(r["dwd"][e] == 0) and torch.all(r["dwgu"][e] == 0)
            continue
        n, rows = hi - lo, r["token"][lo:hi]
        assert torch.equal(rows, rows.unique())           # two different experts of a token
        qgu, sgu, qguT = fq.quant_weight_alloc(wgu[e])
        qd, sd, qdT = fq.quant_weight_alloc(wd[e])
        qe, se = fq.rmsnorm_quant_alloc(r["h"][rows], gamma, EPS)
        gu = fq.linear_fwd_alloc(qe, se, qgu, sgu)
        assert same_bits(gu, r["gu"][lo:hi])
        qh, sh = fq.swiglu_quant_alloc(gu)
        assert same_bits(fq.linear_fwd_alloc(qh, sh, qd, sd), r["y"][lo:hi])
        q1, s1 = fq.quant_act_1x128_alloc(r["dy"][lo:hi].contiguous())
        assert same_bits(fq.linear_dgrad_alloc(q1, s1, qdT, sd), r["dh"][lo:hi])
        q1, s1 = fq.quant_act_1x128_alloc(r["dgu"][lo:hi].contiguous())
        assert same_bits(fq.linear_dgrad_alloc(q1, s1, qguT, sgu), r["dx"][lo:hi])
        # WGrad against 64 bits of what was quantized: codes are off by half a step at most
        # (2^-4 of the value, or half the smallest step, 2^-10 of 448 steps to the amax); the
        # saved activations were FP8 already
        for dw, g, qa, sa in ((r["dwd"][e], r["dy"][lo:hi], qh, sh), (r["dwgu"][e], r["dgu"][lo:hi], qe, se)):
            a = qa.view(torch.float8_e4m3fn).double() * sa[:, :n].double().t().repeat_interleave(128, 1)
            g = g.double()
            off_by = []
            for v in (g, a):
                amax = torch.cat([c.abs().amax(0, keepdim=True).expand_as(c) for c in v.split(128)])
                off_by.append(torch.maximum(2.0 ** -4 * v.abs(), amax / 448 * 2.0 ** -10))
            want, ab = g.t() @ a, g.abs().t() @ a.abs()
            err = off_by[0].t() @ a.abs() + g.abs().t() @ off_by[1] + off_by[0].t() @ off_by[1]
            tol = err + 2.0 ** -8 * (want.abs() + err) + 1e-5 * ab
            assert torch.all((dw.double() - want).abs() <= tol * (1 + 1e-6))
    check_norm_gradient(r["h"], gamma, r["dn"], dout, r["grad"], r["dgamma"])
    # SwiGLU's gradient in 64 bits, at the stored gate, up and incoming gradient: four
    # BF16-sized roundings at most (the output's own half step, fp32 steps far below)
    g, u = r["gu"].double().split(I, 1)
    sg = torch.sigmoid(g)
    want = torch.cat([r["dh"].double() * u * sg * (1 + g * (1 - sg)), r["dh"].double() * g * sg], 1)
    big = torch.cat([(r["dh"].double() * u).abs() * (1 + g.abs()), (r["dh"].double() * g).abs()], 1)
    assert torch.all((r["dgu"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * big + 1e-30)
    # a token's output is the sum of its rows
    w = r["weight"][:, None].to(torch.bfloat16)
    parts = (r["y"] * w).double()
    total = torch.zeros((T, H), dtype=torch.float64, device=DEV).index_add_(0, r["token"], parts)
    assert torch.all((r["out"].double() - total).abs() <= 2.0 ** -8 * total.abs() + 2.0 ** -22 *
                     torch.zeros_like(total).index_add_(0, r["token"], parts.abs()))


def test_routed_step_repeats_itself(fq):  # noqa: F811
    """The same bits again, with a step of another routing between; rows come in two sums of
    two terms, whose order does not matter."""
    a, b = step_inputs(203, 384, 256, 6), step_inputs(130, 384, 256, 6)
    first = routed_step(fq, *a)
    for _ in range(3):
        routed_step(fq, *b)
        again = routed_step(fq, *a)
        for name, t in first.items():
            if name not in ("s", "sh"):
                assert torch.equal(t, again[name]), name
