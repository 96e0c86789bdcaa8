"""Plain implementations, in 64 bits or whole numbers on the CPU, of the serving loop's other operators: block tables and
slot maps, attention of a window with sinks, the matrix product with an epilogue, sampling."""
from __future__ import annotations

import math

import torch

import serving_ref as ref

F64 = torch.float64
MAX32 = 2 ** 31 - 1


def ceil(a, b):
    return -(-a // b)


def extend(table, lens, new, ring, pool, page, T):
    """One sequence after the other; lists in, a dict of lists out. `table` and `ring` are updated copies."""
    table, ring = [list(r) for r in table], list(ring)
    B, F = len(lens), len(ring)
    W = len(table[0]) if B else 0
    head, count = pool[0] % F, min(max(pool[1], 0), F)
    used, asked, back, missing = 0, 0, [], 0
    slots, positions, starts, out = [-1] * T, [0] * T, [0], []
    for b in range(B):
        n, m = max(lens[b], 0), new[b]
        start = starts[-1]
        starts.append(start + max(m, 0))
        held = ceil(n, page)
        if m < 0:
            back += table[b][:min(held, W)]
            out.append(0)
            continue
        fits = ceil(n + m, page) <= W and start + m <= T
        need = ceil(n + m, page) - held if fits else 0
        asked += need
        granted = fits and (need == 0 or asked <= count)
        if granted:
            for i in range(need):
                table[b][held + i] = ring[(head + used) % F]
                used += 1
        else:
            missing += need
        out.append(n + m if granted else n)
        for i in range(min(m, max(T - start, 0))):
            positions[start + i] = min(n + i, MAX32)
            if granted:
                id = table[b][(n + i) // page]
                slots[start + i] = id * page + (n + i) % page if id >= 0 else -1
    back = back[:F - count]
    for j, id in enumerate(back):
        ring[(head + count + j) % F] = id
    return dict(slots=slots, positions=positions, starts=[min(s, MAX32) for s in starts], seq_lens=out,
                pool=[(head + used) % F, count - used + len(back), min(missing, MAX32)], table=table, ring=ring)


def windowed(q, qs, k, v, ks, vs, table, lens, window, sinks, max_len=None):
    """The same attention over the visible tokens alone: each becomes a page of one token, in a table of its own."""
    k, v, ks, vs, table, lens = (t.cpu() for t in (k, v, ks, vs, table, lens))
    P, Hk, page, D = k.shape
    most = table.shape[1] * page if max_len is None else min(max_len, table.shape[1] * page)
    rows, picked, short = [], [], []
    for b in range(table.shape[0]):
        n = max(0, min(int(lens[b]), most))
        j = torch.arange(n)
        j = j[(j < sinks) | (j >= n - window)]
        ids = table[b].long()[j // page] if n else j
        j, ids = j[(ids >= 0) & (ids < P)], ids[(ids >= 0) & (ids < P)]
        rows.append(torch.arange(len(j)) + sum(short))
        short.append(len(j))
        picked.append(torch.stack([ids, j % page]) if len(j) else torch.zeros(2, 0, dtype=torch.int64))
    at = torch.cat(picked, 1)
    width = max(max(short), 1)
    small = torch.zeros(table.shape[0], width, dtype=torch.int32)
    for b, r in enumerate(rows):
        small[b, :len(r)] = r.int()

    def pages(t):
        return t[at[0], :, at[1]].unsqueeze(2) if at.shape[1] else t.new_zeros((1, Hk, 1, *t.shape[3:]))
    return q, qs, pages(k), pages(v), pages(ks), pages(vs), small, torch.tensor(short, dtype=torch.int32)


ACTIVATIONS = {
    None: lambda y: y,
    "relu": lambda y: torch.where(y > 0, y, torch.zeros_like(y)),
    "gelu": lambda y: y * torch.special.erfc(-y / math.sqrt(2)) / 2,
    "gelu_tanh": lambda y: y * torch.sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3)),
    "silu": lambda y: y * torch.sigmoid(y),
}


def assert_epilogue(out, a, sa, b, sb, bias, act, residual):
    """Bounds: the product's (serving_ref.matmul); the bias added in fp32 (2^-24 of the sum); an activation's slope is
    at most 1.13 (gelu; silu 1.1, relu 1), so it passes on 1.13 of that error, and adds 2^-19 of its value (the
    approximations of the logistic function 2^-21, its exponent rounded to 2^-24 of up to 2^5; erfc of a rounded
    argument, 2 x^2 2^-24 for x up to 2.8, 4 ulp) or, further out, less than 2^-24 of the argument; the residual added
    in fp32; half a step of the output."""
    y, e = ref.matmul(a, sa, b, sb)
    if bias is not None:
        y = y + bias.cpu().to(F64)
        e = e + 2.0 ** -24 * (y.abs() + e)
    if act is not None:
        z = ACTIVATIONS[act](y)
        e = 1.13 * e + 2.0 ** -19 * z.abs() + 2.0 ** -24 * y.abs()
        y = z
    if residual is not None:
        y = y + residual.cpu().to(F64)
        e = e + 2.0 ** -24 * (y.abs() + e)
    half = ref.HALF_STEP[out.dtype]
    tol = half * y.abs() + e * (1 + half) + (2.0 ** -25 if out.dtype == torch.float16 else 0.0)
    err = (out.cpu().to(F64) - y).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside; worst {float((err / tol.clamp(min=1e-300)).max()):.3g} of the tolerance"


def sample(x, u, heat=1.0, k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, margin) of one row of 64-bit logits: sorted, then running sums. margin: how far, relative to its
    sum, a border is from the nearest running sum it is compared with; 1 where weights are 0 or 1 alone: sums and borders
    are exact then (whole numbers below 2^29 times 24-bit ones), and so are comparisons of a weight of 0 or 1."""
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    some = x > -math.inf
    if not bool(some.any()):
        return -1, -math.inf, 1.0
    if not heat >= 2.0 ** -126 or k == 1:
        return int((x == x.max()).nonzero()[0]), 0.0, 1.0
    order = torch.sort(-x, stable=True).indices[:int(some.sum())]
    s = x[order]
    w = torch.where(s == s[0], torch.ones_like(s), torch.exp((s - s[0]) / heat)) if math.isfinite(heat) else torch.where(
        s.isinf() != s[0].isinf(), torch.zeros_like(s), torch.ones_like(s))
    if k > 0:
        w = w[:k]
    exact = bool(((w == 0) | (w == 1)).all())
    margin = 1.0
    run = w.cumsum(0)
    if top_p < 1:
        border = max(top_p, 0.0) * run[-1]
        before = torch.cat([run.new_zeros(1), run[:-1]])
        keep = before < border
        keep[0] = True
        if len(before) > 1:
            margin = min(margin, float((before[1:] - border).abs().min() / run[-1]))
        w = w[:int(keep.sum())]
    if min_p > 0:
        keep = w >= min(min_p, 1.0)
        some = w[(w != 0) & (w != 1)]
        margin = min(margin, float((some - min_p).abs().min()) if len(some) else 1.0)
        keep[0] = True
        w = w[:int(keep.sum())]
    run = w.cumsum(0)
    aim = min(max(u, 0.0), 1 - 2.0 ** -24) * run[-1] if u == u else 0.0 * run[-1]
    at = min(int((run <= aim).sum()), len(run) - 1)
    margin = min(margin, float((run - aim).abs().min() / run[-1]))
    return int(order[at]), float(torch.log(w[at] / run[-1])), 1.0 if exact else margin
