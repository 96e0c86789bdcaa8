"""Plain 64-bit implementations of the FP8 serving operators for the parity tests, on the CPU, and the
error bounds the GPU results are held to."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def values(codes: torch.Tensor) -> torch.Tensor:
    """e4m3 codes -> 64-bit values, from the format: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = codes.cpu().view(torch.uint8).to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).to(F64)
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2((e - 10).to(F64)))
    v = torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where((c & 128) != 0, -v, v)


def finite_codes(shape, gen) -> torch.Tensor:
    """Uniform e4m3 codes without NaN."""
    c = torch.randint(0, 254, shape, generator=gen, dtype=torch.int64)
    return torch.where(c >= 127, c + 1, c).to(torch.uint8)


def matmul(a, sa, b, sb):
    """(out, bound without the output rounding) of the block-scaled product in 64 bits.

    The bound: fp32 products and sums within a block of 128 (at most 128 roundings of at most 2^-24 of the
    sum of magnitudes: a serial sum; the tensor cores round less often), the product of the two scales (one)
    and one FMA per block: (128 + 2 + blocks) * 2^-24 * sum |a b| scales. Doubled because a tensor core
    truncates where the FMA rounds (2^-23 per step).
    """
    K = a.shape[1]
    g = torch.arange(K) // 128
    rows = torch.arange(b.shape[0]) // 128
    av = values(a) * sa.cpu().to(F64)[:, g]
    bv = values(b) * sb.cpu().to(F64)[rows][:, g]
    bound = (130 + int(sa.shape[1])) * 2.0 ** -23 * (av.abs() @ bv.abs().T)
    return av @ bv.T, bound


def assert_matmul(out, a, sa, b, sb):
    ref, bound = matmul(a, sa, b, sb)
    got = out.cpu().to(F64)
    tol = HALF_STEP[out.dtype] * ref.abs() + bound * (1 + HALF_STEP[out.dtype])
    if out.dtype == torch.float16:  # subnormal outputs: half a step is 2^-25
        tol = tol + 2.0 ** -25
    bad = (got - ref).abs() > tol
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} outside; worst "
                                 f"{float(((got - ref).abs() / tol.clamp(min=1e-300)).max()):.3g} of the tolerance")


def attention(q, qs, k, v, ks, vs, table, lens, scale, max_len=None):
    """(out, lse, out bound, lse bound) in 64 bits; k, v [P, Hk, page, D], table and lens as given.

    Bounds, without the output rounding: a score is a sum of D exact products in fp32 (D * 2^-23 of the sum
    of magnitudes) times factors rounded a few times (8 * 2^-24 of the score); an error e of a score moves
    its weight by a factor exp(e), and the weights' sum by no more. exp2 and log2 approximations: 2^-21.
    Each weight times its V scale is rounded to fp16 relative to the row's largest (2^-11, or 2^-25 of the
    largest absolutely); sums of n terms in fp32: n * 2^-23, n being at most the length, in practice
    spread over many partial sums.
    """
    q, k, v = values(q), values(k), values(v)
    qs, ks, vs = (t.cpu().to(F64) for t in (qs, ks, vs))
    table, lens = table.cpu().long(), lens.cpu().long()
    B, Hq, D = q.shape
    P, Hk, page, _ = k.shape
    G = Hq // Hk
    out, ob = torch.zeros(B, Hq, D, dtype=F64), torch.zeros(B, Hq, D, dtype=F64)
    lse, lb = torch.full((B, Hq), -math.inf, dtype=F64), torch.zeros(B, Hq, dtype=F64)
    most = table.shape[1] * page if max_len is None else min(max_len, table.shape[1] * page)
    for b in range(B):
        n = max(0, min(int(lens[b]), most))
        pos = torch.arange(n)
        ids = table[b, pos // page] if n else pos
        live = (ids >= 0) & (ids < P)
        ids, off = ids[live], (pos % page)[live]
        n = int(live.sum())
        if n == 0:
            continue
        for h in range(Hk):
            rows = slice(h * G, (h + 1) * G)
            kk, vv = k[ids, h, off], v[ids, h, off]
            f = qs[b, rows][:, None] * ks[ids, h, off][None] * scale
            x = (q[b, rows] @ kk.T) * f
            mag = (q[b, rows].abs() @ kk.abs().T) * f.abs()
            e = (D * 2.0 ** -23 * mag + 8 * 2.0 ** -24 * x.abs()).amax(1, keepdim=True)
            lse[b, rows] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1)
            w = p * vs[ids, h, off][None]
            out[b, rows] = w @ vv
            rel = 2 * e + 2.0 ** -21 + n * 2.0 ** -23
            lb[b, rows] = (e + 2.0 ** -20 + n * 2.0 ** -23).squeeze(1) + lse[b, rows].abs() * 2.0 ** -22
            ob[b, rows] = (rel + 2.0 ** -11 * (1 + rel)) * (w.abs() @ vv.abs()) + \
                2.0 ** -25 * w.abs().amax(1, keepdim=True) * vv.abs().sum(0)[None]
    return out, lse, ob, lb


def assert_attention(out, lse, *args, max_len=None):
    ref, ref_lse, ob, lb = attention(*args, max_len=max_len)
    got = out.cpu().to(F64)
    half = HALF_STEP[out.dtype]
    tol = half * ref.abs() + ob * (1 + half) + (2.0 ** -25 if out.dtype == torch.float16 else 0.0)
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"out: {int(bad.sum())} of {bad.numel()} outside; worst "
                                 f"{float((err / tol.clamp(min=1e-300)).max()):.3g} of the tolerance")
    if lse is not None:
        g = lse.cpu().to(F64)
        same = (g == ref_lse) | ((g - ref_lse).abs() <= lb)
        assert bool(same.all()), f"lse: worst {float((g - ref_lse).abs().nan_to_num(0).max()):.3g}"


def append(qkv, wq, wk, cos, sin, Hq, Hk, D, R, eps=1e-6, fp8_max=448.0):
    """64-bit rows after norm and rotation: (values [T, Hq+2Hk, D], scale [T, Hq+2Hk])."""
    T = qkv.shape[0]
    x = qkv.cpu()[:, :(Hq + 2 * Hk) * D].to(F64).view(T, Hq + 2 * Hk, D)
    w = torch.cat([wq.cpu().to(F64).expand(Hq, D), wk.cpu().to(F64).expand(Hk, D)])
    y = x[:, :Hq + Hk]
    y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w
    lo, hi = y[..., D - R:D - R // 2], y[..., D - R // 2:]
    c, s = cos.cpu().to(F64)[:, None], sin.cpu().to(F64)[:, None]
    y = torch.cat([y[..., :D - R], lo * c - hi * s, hi * c + lo * s, ], -1)
    y = torch.cat([y, x[:, Hq + Hk:]], 1)
    return y, y.abs().amax(-1).clamp(min=1e-4) / fp8_max


def e4m3_codes(y):
    """Nearest e4m3 codes (ties to even) of 64-bit values, saturating at 448; the sign of zero kept."""
    grid = values(torch.arange(127, dtype=torch.uint8))
    mag = y.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, mag.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - mag, mag - grid[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + 128 * torch.signbit(y).long()).to(torch.uint8)
