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
