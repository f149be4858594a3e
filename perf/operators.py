"""Cases and plain forms of the expert-layer operators: the RMSNorm that adds the residual
stream and quantizes, and the block-scaled FP8 linear layer with one weight per expert
over ragged groups of token rows (forward, DGrad, WGrad and the two quantizers that make
WGrad's operands).

Tokens are sorted by expert: expert e owns rows offsets[e] .. offsets[e + 1] - 1 of every
[M, ...] tensor (int32, on the device, so a program never waits for the host to learn the
routing); rows from offsets[E] on belong to nobody and stay as they are. Column-wise
(128x1) groups restart at each expert: expert e's groups start at column 128 * (the
number of groups of the experts before it) of the transposed arrays, and a last partial
group is filled up with zero codes.

`own` selects the library's kernels; otherwise `run` computes the same in elementary
torch operations, with the roundings that define the FP8 operators (fp32 scale = amax /
448, code = nearest E4M3 value to the fp32 quotient, BF16 between the norm and its
quantizer).
"""
import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
LARGEST_FLOPS = 2.0 * 16384 * 4096 * 4096


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 16 sequences through the norm in front of the experts
        dict(name="norm_decode", op="norm", M=16, H=4096, pad=0),
        # the norm of a training micro-batch of 8192 tokens
        dict(name="norm_train", op="norm", M=8192, H=4096, pad=0),
        # decoding: 16 sequences, each to 8 of 64 experts; a buffer with a few free rows
        dict(name="fwd_decode", op="fwd", E=64, M=136, spare=8, N=4096, K=4096, skew=0.3),
        # prefill or training: 8192 tokens, each to 2 of 8 experts, gate and up projection
        dict(name="fwd_train", op="fwd", E=8, M=16384, spare=0, N=4096, K=4096, skew=0.3),
        # the down projection's input gradient of a small ragged micro-batch
        dict(name="dgrad_small", op="dgrad", E=16, M=1023, spare=0, N=3584, K=1024, skew=0.5),
        # the same over 16 experts at training size
        dict(name="dgrad_train", op="dgrad", E=16, M=16384, spare=100, N=4096, K=2048, skew=0.3),
        # weight gradients of many experts with few tokens each, some of them without any
        dict(name="wgrad_small", op="wgrad", E=32, M=777, spare=9, N=2048, K=1024, skew=0.5),
        # weight gradients at training size
        dict(name="wgrad_train", op="wgrad", E=8, M=16384, spare=0, N=4096, K=2048, skew=0.3),
        # the gradient quantizer of a small ragged micro-batch
        dict(name="tq_bf16_small", op="tq_bf16", E=16, M=301, spare=0, N=3584, skew=0.5),
        # the gradient quantizer at training size
        dict(name="tq_bf16_train", op="tq_bf16", E=8, M=16384, spare=0, N=4096, skew=0.3),
        # the saved activation's requantizer of a small ragged micro-batch
        dict(name="tq_fp8_small", op="tq_fp8", E=64, M=1001, spare=1, N=1024, skew=0.3),
        # the saved activation's requantizer at training size
        dict(name="tq_fp8_train", op="tq_fp8", E=8, M=16384, spare=0, N=4096, skew=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    """A case of the same ranges: 1 to 16384 rows, 1 to 64 experts, 512 to 5120 features."""
    op = rng.choice(["norm", "fwd", "dgrad", "wgrad", "tq_bf16", "tq_fp8"])
    M = _log(rng, 1, 16384)
    if op == "norm":
        return dict(op=op, M=M, H=16 * _log(rng, 32, 512), pad=rng.choice([0, 0, 64]))
    E = _log(rng, 1, 64)
    spare = rng.choice([0, rng.randrange(0, max(1, M // 8))])
    N, K = 128 * _log(rng, 4, 40), 128 * _log(rng, 4, 40)
    skew = rng.choice([0.0, 0.3, 0.5])
    if op in ("fwd", "dgrad", "wgrad"):
        while E > 1 and E * N * K > 64 * 4096 * 4096:
            E -= 1
        while 2.0 * M * N * K > LARGEST_FLOPS:
            M -= M // 8
        return dict(op=op, E=E, M=M, spare=min(spare, M - 1), N=N, K=K, skew=skew)
    return dict(op=op, E=E, M=M, spare=spare, N=N, skew=skew)


def _counts(c):
    """Rows of each expert, before the seed gives them to experts in some order: a share
    that falls off with the rank and is uneven besides (some experts get none)."""
    E, rows = c["E"], c["M"] - c["spare"]
    i = np.arange(1, E + 1)
    w = i ** -float(c["skew"]) * (0.75 + 0.5 * np.modf(0.6180339887 * i)[0])
    n = np.floor(rows * w / w.sum()).astype(np.int64)
    n[: rows - n.sum()] += 1
    return n


def _padded(M, E):
    """Columns of the transposed arrays: every expert's rows rounded up to 128, at most."""
    return 128 * ((M + 127 * min(E, M)) // 128)


def work(c):
    if c["op"] == "norm":
        M, H = c["M"], c["H"]
        return {"bytes": 7 * M * H + 4 * M * -(-H // 128) + 2 * H, "flops": 10 * M * H}
    n = _counts(c)
    rows, used, groups = int(n.sum()), int((n > 0).sum()), int((-(-n // 128)).sum())
    N, K, off = c["N"], c.get("K", 0), 4 * (c["E"] + 1)
    if c["op"] in ("fwd", "dgrad"):
        k, m = (K, N) if c["op"] == "fwd" else (N, K)
        scales = 4 * rows * (k // 128) + 4 * used * (N // 128) * (K // 128)
        return {"bytes": rows * k + used * N * K + scales + 2 * rows * m + off,
                "flops": 2 * rows * N * K}
    if c["op"] == "wgrad":
        return {"bytes": (rows + 4 * groups) * (N + K) + 2 * c["E"] * N * K + off,
                "flops": 2 * rows * N * K}
    row = rows * N + 4 * rows * (N // 128)          # codes and scales of 1x128 groups
    col = 128 * groups * N + 4 * groups * N         # codes and scales of 128x1 groups
    read = 2 * rows * N + row if c["op"] == "tq_bf16" else row
    return {"bytes": read + col + off, "flops": 6 * rows * N}


# ---------------------------------------------------------------------------- plain forms

def _lds(m):
    return (m + 3) // 4 * 4


def _scale(amax):
    return torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))


def _code(t):
    return t.clamp(-448.0, 448.0).to(F8)


def _decode(q):
    return q.view(F8).float()


def _rows_1x128(y):
    """1x128 groups of fp32 y [M, H]: codes [M, H], scales [G, lds]."""
    M, H = y.shape
    G = -(-H // 128)
    g = torch.nn.functional.pad(y, (0, 128 * G - H)).view(M, G, 128)
    s = _scale(g.abs().amax(-1))
    q = _code(g / s[..., None]).view(M, 128 * G)[:, :H].contiguous()
    out = torch.zeros(G, _lds(M), device=y.device)
    out[:, :M] = s.t()
    return q, out


def _blocks_128x128(w):
    """128x128 blocks of fp32 w [E, N, K]: codes [E, N, K], scales [E, N/128, K/128]."""
    E, N, K = w.shape
    b = w.view(E, N // 128, 128, K // 128, 128)
    s = _scale(b.abs().amax((2, 4)))
    return _code(b / s[:, :, None, :, None]).view(E, N, K), s


def _row_values(q, s):
    """fp32 values of codes [M, H] with 1x128 scales [G, lds], H a multiple of 128."""
    M, H = q.shape
    return (_decode(q).view(M, H // 128, 128) * s[:, :M].t()[..., None]).view(M, H)


def _weight_values(q, s):
    E, N, K = q.shape
    b = _decode(q).view(E, N // 128, 128, K // 128, 128)
    return (b * s[:, :, None, :, None]).view(E, N, K)


def _grouped_product(a, w, offsets, cap):
    """a [M, K] rows of expert e times w[e] [K, N], BF16, zero in rows of nobody."""
    M = a.shape[0]
    idx = offsets[:-1, None].long() + torch.arange(cap, device=a.device)
    ok = idx < offsets[1:, None]
    rows = a[idx.clamp(max=M - 1)]
    y = torch.bmm(rows, w).to(torch.bfloat16)
    out = torch.zeros(M + 1, y.shape[2], dtype=torch.bfloat16, device=a.device)
    out[torch.where(ok, idx, M).flatten()] = y.flatten(0, 1)
    return out[:M]


def _padded_rows(offsets, P):
    """For each column of the transposed arrays: its row, whether a row is there, and
    whether its group belongs to an expert."""
    n = offsets[1:].long() - offsets[:-1]
    ends = ((n + 127) // 128 * 128).cumsum(0)
    p = torch.arange(P, device=offsets.device)
    e = torch.searchsorted(ends, p, right=True).clamp(max=n.numel() - 1)
    within = p - (ends[e] - (n[e] + 127) // 128 * 128)
    return offsets[e].long() + within, (p < ends[-1]) & (within < n[e]), p < ends[-1]


def _columns_128x1(x, offsets, P):
    """128x1 groups of fp32 x [M, N] that restart at each expert: transposed codes [N, P]
    and scales [P/128, N]; zero where no expert's group is."""
    row, ok, group = _padded_rows(offsets, P)
    v = torch.where(ok[:, None], x[row.clamp(max=x.shape[0] - 1)], 0.0)
    v = v.view(P // 128, 128, -1)
    s = _scale(v.abs().amax(1))
    q = _code(v / s[:, None]).view(P, -1).t().contiguous()
    return q, torch.where(group[::128, None], s, 0.0)


def _column_values(q, s):
    """fp32 values [P, N] of transposed codes [N, P] with 128x1 scales [P/128, N]."""
    N, P = q.shape
    return (_decode(q).t().reshape(P // 128, 128, N) * s[:, None]).view(P, N)


def _rows_of_nobody(t, offsets, dim):
    i = torch.arange(t.shape[dim], device=t.device)
    keep = (i >= offsets[0]) & (i < offsets[-1])
    keep = keep[:, None] if dim == 0 else keep
    return torch.where(keep, t.float(), 0.0).to(t.dtype)


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
        ss = h.double().square().sum(1, keepdim=True)
        r = (1.0 / torch.sqrt(ss / h.shape[1] + s["eps"])).float()
        y = (h.float() * r * s["gamma"].float()).to(torch.bfloat16)
        return (h,) + _rows_1x128(y.float())
    off = s["offsets"]
    if op == "fwd":
        w = _weight_values(s["qw"], s["sw"])
        return _grouped_product(_row_values(s["qa"], s["sa"]), w.transpose(1, 2), off, s["cap"])
    if op == "dgrad":
        w = _weight_values(s["qwT"].permute(1, 2, 0).contiguous(), s["sw"])
        return _grouped_product(_row_values(s["qa"], s["sa"]), w, off, s["cap"])
    if op == "wgrad":
        n = off[1:].long() - off[:-1]
        pad = (n + 127) // 128 * 128
        start = pad.cumsum(0) - pad
        idx = start[:, None] + torch.arange(s["cap"], device=off.device)
        ok = (torch.arange(s["cap"], device=off.device) < n[:, None])[..., None]
        idx = idx.clamp(max=s["qdyT"].shape[1] - 1)
        dy = torch.where(ok, _column_values(s["qdyT"], s["sdy"])[idx], 0.0)
        x = torch.where(ok, _column_values(s["qxT"], s["sx"])[idx], 0.0)
        return torch.bmm(dy.transpose(1, 2), x).to(torch.bfloat16)
    if op == "tq_bf16":
        q, sr = _rows_1x128(s["dy"].float())
        return ((_rows_of_nobody(q, off, 0), _rows_of_nobody(sr, off, 1))
                + _columns_128x1(s["dy"].float(), off, s["qT"].shape[1]))
    return _columns_128x1(_row_values(s["q"], s["s"]), off, s["qT"].shape[1])


# ---------------------------------------------------------------------------- inputs

def _activations(g, M, H):
    """N(0,1) with 0.5 % outlier channels, BF16."""
    x = torch.randn(M, H, generator=g, device=DEV)
    return (x * torch.where(torch.rand(H, generator=g, device=DEV) < 0.005, 50.0, 1.0)).to(torch.bfloat16)


def _gradients(g, M, H):
    return (1e-3 * torch.randn(M, H, generator=g, device=DEV)).to(torch.bfloat16)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"op": c["op"]}

    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device=DEV)

    def f32(*shape):
        return torch.zeros(shape, device=DEV)

    if c["op"] == "norm":
        M, H = c["M"], c["H"]
        s["x"] = _activations(g, M, H + c["pad"])[:, :H]
        s["res"] = _activations(g, M, H + c["pad"])[:, :H]
        s["gamma"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
        s["eps"] = 1e-5
        s["h"] = torch.zeros(M, H, dtype=torch.bfloat16, device=DEV)
        s["q"], s["s"] = u8(M, H), f32(-(-H // 128), _lds(M))
        return s
    E, M, N, K = c["E"], c["M"], c["N"], c.get("K")
    n = np.random.RandomState(seed % (1 << 31)).permutation(_counts(c))
    s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    s["cap"] = max(int(n.max()), 1)  # the plain forms' batch capacity
    P = _padded(M, E)
    if c["op"] in ("fwd", "dgrad"):
        w = (0.02 * torch.randn(E, N, K, generator=g, device=DEV)).to(torch.bfloat16).float()
        qw, s["sw"] = _blocks_128x128(w)
        del w
        if c["op"] == "fwd":
            s["qw"] = qw.view(torch.uint8)
            a, out = _activations(g, M, K), N
        else:
            s["qwT"] = qw.view(torch.uint8).permute(2, 0, 1).contiguous()
            a, out = _gradients(g, M, N), K
        q, s["sa"] = _rows_1x128(a.float())
        s["qa"] = q.view(torch.uint8)
        s["y"] = torch.zeros(M, out, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "wgrad":
        q, s["sdy"] = _columns_128x1(_gradients(g, M, N).float(), s["offsets"], P)
        s["qdyT"] = q.view(torch.uint8)
        q, s["sx"] = _columns_128x1(_activations(g, M, K).float(), s["offsets"], P)
        s["qxT"] = q.view(torch.uint8)
        s["dw"] = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "tq_bf16":
        s["dy"] = _gradients(g, M, N)
        s["q"], s["s"] = u8(M, N), f32(N // 128, _lds(M))
        s["qT"], s["sT"] = u8(N, P), f32(P // 128, N)
    else:
        q, s["s"] = _rows_1x128(_activations(g, M, N).float())
        s["q"] = q.view(torch.uint8)
        s["qT"], s["sT"] = u8(N, P), f32(P // 128, N)
    return s


def run(s):
    if not own:
        return _plain(s)
    import fp8_block_scaled_08_b200 as fq
    op = s["op"]
    if op == "norm":
        fq.add_rmsnorm_quant(s["x"], s["res"], s["gamma"], s["eps"], s["h"], s["q"], s["s"])
        return s["h"], s["q"].view(F8), s["s"]
    if op == "fwd":
        fq.grouped_linear_fwd(s["qa"], s["sa"], s["qw"], s["sw"], s["offsets"], s["y"])
        return s["y"]
    if op == "dgrad":
        fq.grouped_linear_dgrad(s["qa"], s["sa"], s["qwT"], s["sw"], s["offsets"], s["y"])
        return s["y"]
    if op == "wgrad":
        fq.grouped_linear_wgrad(s["qdyT"], s["sdy"], s["qxT"], s["sx"], s["offsets"], s["dw"])
        return s["dw"]
    if op == "tq_bf16":
        fq.grouped_transpose_quant_bf16(s["dy"], s["offsets"], s["q"], s["s"], s["qT"], s["sT"])
        return s["q"].view(F8), s["s"], s["qT"].view(F8), s["sT"]
    fq.grouped_transpose_quant_fp8(s["q"], s["s"], s["offsets"], s["qT"], s["sT"])
    return s["qT"].view(F8), s["sT"]


# ---------------------------------------------------------------------------- exact values

def exact(c, seed):
    """The definitions in 64 bits, expert by expert. Codes are the quotients that they
    stand for; the norm keeps the roundings that are part of its definition (the stored
    residual stream, r, the two fp32 products and the BF16 that is quantized)."""
    s = prepare(c, seed)
    f64 = torch.float64

    def groups(v):  # v [..., 128] -> (quotients, scales)
        a = v.abs().amax(-1, keepdim=True)
        sc = torch.where(a > 0, a / 448.0, torch.ones_like(a))
        return v / sc, sc[..., 0]

    if c["op"] == "norm":
        M, H = c["M"], c["H"]
        h = (s["x"].to(f64) + s["res"].to(f64)).to(torch.bfloat16).to(f64)
        r = (h.pow(2).mean(1) + s["eps"]).rsqrt().to(torch.float32).to(f64)
        y = (h * r[:, None]).to(torch.float32).to(f64) * s["gamma"].to(f64)[None]
        y = y.to(torch.float32).to(torch.bfloat16).to(f64)
        q = torch.zeros(M, H, dtype=f64, device=DEV)
        sc = torch.zeros(s["s"].shape, dtype=f64, device=DEV)
        for j in range(sc.shape[0]):
            q[:, 128 * j:128 * j + 128], sc[j, :M] = groups(y[:, 128 * j:128 * j + 128])
        return h, q, sc
    off = s["offsets"].tolist()
    if c["op"] in ("fwd", "dgrad"):
        fwd = c["op"] == "fwd"
        a = s["qa"].view(F8).to(f64) * s["sa"][:, :c["M"]].to(f64).t().repeat_interleave(128, 1)
        y = torch.zeros(s["y"].shape, dtype=f64, device=DEV)
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            sw = s["sw"][e].to(f64).repeat_interleave(128, 0).repeat_interleave(128, 1)
            if fwd:
                y[lo:hi] = a[lo:hi] @ (s["qw"][e].view(F8).to(f64) * sw).t()
            else:
                y[lo:hi] = a[lo:hi] @ (s["qwT"][:, e].view(F8).to(f64) * sw.t()).t()
        return y
    if c["op"] == "wgrad":
        dw = torch.zeros(s["dw"].shape, dtype=f64, device=DEV)
        b = 0
        for e in range(c["E"]):
            n = off[e + 1] - off[e]
            k = -(-n // 128)
            p = slice(128 * b, 128 * b + n)
            sdy = s["sdy"][b:b + k].to(f64).repeat_interleave(128, 0)[:n]
            sx = s["sx"][b:b + k].to(f64).repeat_interleave(128, 0)[:n]
            dw[e] = ((s["qdyT"][:, p].view(F8).to(f64) * sdy.t())
                     @ (s["qxT"][:, p].view(F8).to(f64).t() * sx))
            b += k
        return dw
    M, N = c["M"], c["N"]
    qT = torch.zeros(s["qT"].shape, dtype=f64, device=DEV)
    sT = torch.zeros(s["sT"].shape, dtype=f64, device=DEV)
    if c["op"] == "tq_bf16":
        x = s["dy"].to(f64)
    else:
        x = s["q"].view(F8).to(f64) * s["s"][:, :M].to(f64).t().repeat_interleave(128, 1)
    b = 0
    for e in range(c["E"]):
        for lo in range(off[e], off[e + 1], 128):
            n = min(128, off[e + 1] - lo)
            qT[:, 128 * b:128 * b + n], sT[b] = groups(x[lo:lo + n].t())
            b += 1
    if c["op"] == "tq_fp8":
        return qT, sT
    q = torch.zeros(M, N, dtype=f64, device=DEV)
    sr = torch.zeros(s["s"].shape, dtype=f64, device=DEV)
    lo, hi = off[0], off[-1]
    for j in range(N // 128):
        q[lo:hi, 128 * j:128 * j + 128], sr[j, lo:hi] = groups(x[lo:hi, 128 * j:128 * j + 128])
    return q, sr, qT, sT
