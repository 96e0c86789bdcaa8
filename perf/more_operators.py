"""Measured calls of a serving loop's other operators: block tables and slot maps from request lengths, paged
attention with a sliding window and sinks, the FP8 matrix product with bias, activation and residual, and sampling.

Each case is one pass through one operator. With ``own`` false, ``run`` computes the operator in elementary
torch operations; with ``own`` true it makes the library call. ``exact`` computes the same outputs in 64 bits
from the definitions, written apart from the plain form.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 128
AMAX_FLOOR = 1e-4
FP8_MAX = 448.0


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # A decoding batch: one new token each, some sequences end and return their pages (latency).
        dict(name="extend_batch", op="extend", B=64, L=8192, T=64, page=64, ends=4),
        # Prompts of ragged lengths and running sequences in one step.
        dict(name="extend_prompts", op="extend", B=1000, L=8192, T=65536, page=16, ends=100),
        # One long conversation that only sees its last 4096 tokens and the first page.
        dict(name="window_long", op="attend", B=1, L=131072, window=4096, sinks=64, Hq=64, Hk=8, D=128, page=64, dtype="bf16"),
        # A decoding batch whose lengths run from 0 to 32768.
        dict(name="window_batch", op="attend", B=64, L=32768, window=2048, sinks=4, Hq=32, Hk=8, D=128, page=64, dtype="bf16"),
        # Heads of 64 without sharing, pages that are no power of two, a window that starts inside a page, fp16 output.
        dict(name="window_heads", op="attend", B=17, L=2500, window=777, sinks=5, Hq=16, Hk=16, D=64, page=24, dtype="fp16"),
        # One token through the first projection of a feed-forward block.
        dict(name="linear_token", op="linear", M=1, N=8192, K=4096, bias=True, act="silu", residual=False, dtype="bf16"),
        # A decoding batch through the projection that leads back to the residual stream.
        dict(name="linear_batch", op="linear", M=64, N=4096, K=8192, bias=True, act="none", residual=True, dtype="bf16"),
        # A ragged chunk: no size is a multiple of a tile, the last scale block is partial.
        dict(name="linear_ragged", op="linear", M=333, N=1111, K=1968, bias=True, act="gelu", residual=True, dtype="fp16"),
        # A 4096-token prompt through a feed-forward projection.
        dict(name="linear_prompt", op="linear", M=4096, N=8192, K=4096, bias=True, act="gelu_tanh", residual=True, dtype="bf16"),
        # The next token of one conversation (latency).
        dict(name="sample_token", op="sample", B=1, V=32000, cuts="both", masked=0.0, dtype="bf16"),
        # A small batch with a grammar's masks, an odd vocabulary.
        dict(name="sample_masked", op="sample", B=17, V=50001, cuts="mixed", masked=0.9, dtype="fp16"),
        # A large batch, each row with its own settings.
        dict(name="sample_batch", op="sample", B=256, V=151936, cuts="mixed", masked=0.0, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "attend", "attend", "linear", "linear", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 64, 128])
    if op == "extend":
        B = _spread(rng, 1, 1000)
        return dict(op=op, B=B, L=_spread(rng, 1, 8192), T=max(B, _spread(rng, 1, 65536)), page=page, ends=B // rng.choice([3, 10, 50]))
    if op == "linear":
        M, N = _spread(rng, 1, 4096), _spread(rng, 64, 8192)
        K = 128 * _spread(rng, 1, 32) if rng.random() < 0.7 else 16 * _spread(rng, 1, 256)
        return dict(op=op, M=M, N=N, K=K, bias=rng.random() < 0.7, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                    residual=rng.random() < 0.6, dtype=dtype)
    if op == "sample":
        return dict(op=op, B=_spread(rng, 1, 256), V=_spread(rng, 500, 151936), cuts=rng.choice(["mixed", "both", "top_k", "top_p", "none"]),
                    masked=rng.choice([0.0, 0.0, 0.5, 0.99]), dtype=dtype)
    D = rng.choice([64, 96, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 4, 5, 8, 16])
    B = _spread(rng, 1, 64)
    window = _spread(rng, 1, min(4096, (64 * 2048 * 8 * 128) // (B * max(Hk, Hq // 8) * max(D, 128))))
    return dict(op=op, B=B, L=_spread(rng, 1, min(131072, (1 << 20) // B)), window=window, sinks=rng.choice([0, 1, 4, 16, 64]),
                Hq=Hq, Hk=Hk, D=D, page=page, dtype=dtype)


def _lengths(case):
    """The batch's lengths, evenly spread over [0, L], the longest of them L; one sequence has length L."""
    B, L = case["B"], case["L"]
    return [L] if B == 1 else [(L * i) // (B - 1) for i in range(B)]


def _step(case):
    """(lengths, new lengths) of an extend case: `ends` sequences end, a tenth wait, the T tokens go to the others,
    one each and the rest of them to one in eight."""
    B, T = case["B"], case["T"]
    rng = random.Random(B + 7 * T)
    lens = _lengths(case)
    rng.shuffle(lens)
    kind = ["end"] * min(case["ends"], B - 1)
    kind += ["wait"] * ((B - len(kind)) // 10)
    kind += ["run"] * (B - len(kind))
    rng.shuffle(kind)
    new = [{"end": -1, "wait": 0, "run": 1}[k] for k in kind]
    left = T - sum(n for n in new if n > 0)
    prompts = [b for b in range(B) if new[b] == 1][::8]
    for i, b in enumerate(prompts):
        part = left if i == len(prompts) - 1 else min(left, rng.randrange(2 * left // (len(prompts) - i) + 1))
        new[b] += part
        left -= part
    return lens, new


def _ceil(a, b):
    return -(-a // b)


def _visible(case):
    """(visible tokens, their pages) over the batch."""
    page, tokens, pages = case["page"], 0, 0
    for n in _lengths(case):
        start = max(n - case["window"], min(case["sinks"], n))
        first = min(case["sinks"], n)
        tokens += n - start + first
        at, sunk = start // page, _ceil(first, page)
        pages += sunk + max(0, _ceil(n, page) - max(at, sunk))
    return tokens, pages


def work(case):
    op = case["op"]
    if op == "extend":
        B, T, page = case["B"], case["T"], case["page"]
        lens, new = _step(case)
        got = sum(_ceil(n + m, page) - _ceil(n, page) for n, m in zip(lens, new) if m > 0)
        back = sum(_ceil(n, page) for n, m in zip(lens, new) if m < 0)
        part = sum(1 for n, m in zip(lens, new) if m > 0 and n % page)
        return {"bytes": 16 * B + 12 * T + 8 * (got + back) + 4 * part, "flops": 8 * (B + T)}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        g = _ceil(K, GROUP)
        return {"bytes": M * K + N * K + 4 * g * (M + _ceil(N, GROUP)) + 2 * M * N * (2 if case["residual"] else 1) + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if op == "sample":
        B, V = case["B"], case["V"]
        return {"bytes": 2 * B * V + 32 * B, "flops": 2 * B * V}
    B, Hq, Hk, D = (case[k] for k in ("B", "Hq", "Hk", "D"))
    tokens, pages = _visible(case)
    return {"bytes": tokens * Hk * (2 * D + 8) + B * Hq * (D + 4 + 2 * D + 4) + 4 * B + 4 * pages, "flops": 4 * tokens * Hq * D}


# ------------------------------------------------------------------------------------------ inputs
def _codes(x, groups=None):
    """e4m3 codes (uint8) and 32-bit scales of the rows of x, or of its groups of columns."""
    if groups is None:
        s = x.abs().amax(-1, keepdim=True).clamp(min=AMAX_FLOOR) / FP8_MAX
        return (x / s).to(torch.float8_e4m3fn).view(torch.uint8), s.squeeze(-1)
    rows, K = x.shape
    n = _ceil(K, groups)
    y = torch.nn.functional.pad(x, (0, n * groups - K)).view(rows, n, groups)
    s = y.abs().amax(-1).clamp(min=AMAX_FLOOR) / FP8_MAX
    q = (y / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, n * groups)
    return q[:, :K].contiguous(), s


def _cache(shape, gen):
    """A cache's codes [pages, heads, page, D] and scales [pages, heads, page], of normal values."""
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for p in range(0, shape[0], step):
        n = min(step, shape[0] - p)
        codes[p:p + n], scale[p:p + n] = _codes(torch.randn((n, *shape[1:]), device="cuda", generator=gen))
    return codes, scale


def _prepare_extend(s, gen, rng):
    B, page = s["B"], s["page"]
    lens, new = _step(s)
    owned = [_ceil(n, page) for n in lens]
    need = sum(_ceil(n + max(m, 0), page) for n, m in zip(lens, new)) - sum(owned)
    width = max(_ceil(n + max(m, 0), page) for n, m in zip(lens, new)) + 2
    pages = sum(owned) + need + 17
    order = torch.randperm(pages, device="cuda", generator=gen).int()
    # Every page is a sequence's or free; the free ones lie in a ring of as many places as there are pages.
    first = torch.tensor([sum(owned[:i]) for i in range(B)], device="cuda")
    col = torch.arange(width, device="cuda")
    used = col[None, :] < torch.tensor(owned, device="cuda")[:, None]
    s["page_table"] = torch.where(used, order[(first[:, None] + col).clamp(max=pages - 1)], -1).int()
    head, count = rng.randrange(pages), pages - sum(owned)
    s["free_pages"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free_pages"][(head + torch.arange(count, device="cuda")) % pages] = order[sum(owned):]
    s["pool"] = torch.tensor([head, count, 0], dtype=torch.int32, device="cuda")
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")


def _prepare_attend(s, gen, rng):
    B, Hq, Hk, D, page = (s[k] for k in ("B", "Hq", "Hk", "D", "page"))
    lens = _lengths(s)
    rng.shuffle(lens)
    s["q"], s["q_scale"] = _codes(1.5 * torch.randn(B, Hq, D, device="cuda", generator=gen))
    need = [_ceil(n, page) for n in lens]
    pages = sum(need) + 1
    s["k_cache"], s["k_scale"] = _cache((pages, Hk, page, D), gen)
    s["v_cache"], s["v_scale"] = _cache((pages, Hk, page, D), gen)
    order = torch.randperm(pages, device="cuda", generator=gen).int()
    first = torch.tensor([sum(need[:i]) for i in range(B)], device="cuda")
    col = torch.arange(max(need), device="cuda")
    used = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    s["page_table"] = torch.where(used, order[(first[:, None] + col).clamp(max=pages - 1)], -1).int()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")


def _prepare_linear(s, gen, rng):
    M, N, K, dtype = s["M"], s["N"], s["K"], DTYPES[s["dtype"]]
    # Activations after a norm, one scale per token and 128 columns; a projection's weights, one scale
    # per 128 x 128 block.
    s["a"], s["a_scale"] = _codes(torch.randn(M, K, device="cuda", generator=gen), GROUP)
    n, g = _ceil(N, GROUP), _ceil(K, GROUP)
    w = torch.randn(n * GROUP, g * GROUP, device="cuda", generator=gen) * (K ** -0.5)
    w[N:], w[:, K:] = 0.0, 0.0
    blocks = w.view(n, GROUP, g, GROUP)
    bs = blocks.abs().amax((1, 3)).clamp(min=AMAX_FLOOR) / FP8_MAX
    q = (blocks / bs[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n * GROUP, g * GROUP)
    s["b"], s["b_scale"] = q[:N, :K].contiguous(), bs
    s["bias_row"] = (0.5 * torch.randn(N, device="cuda", generator=gen)).to(dtype) if s["bias"] else None
    s["stream"] = (2.0 * torch.randn(M, N, device="cuda", generator=gen)).to(dtype) if s["residual"] else None


def _prepare_sample(s, gen, rng):
    B, V = s["B"], s["V"]
    # A broad bulk and some tens of likely tokens in each row.
    x = 2.0 * torch.randn(B, V, device="cuda", generator=gen)
    x += 9.0 * torch.rand(B, V, device="cuda", generator=gen) ** (V / 64)
    if s["masked"] > 0.0:
        x.masked_fill_(torch.rand(B, V, device="cuda", generator=gen) < s["masked"], -math.inf)
        if B > 4:
            x[rng.randrange(B)] = -math.inf  # a row whose mask leaves nothing
    s["logits"] = x.to(DTYPES[s["dtype"]])
    s["u"] = torch.rand(B, device="cuda", generator=gen)
    cuts, rows = s["cuts"], []
    for _ in range(B):
        kind = cuts if cuts != "mixed" else rng.choice(["both", "both", "top_k", "top_p", "none", "greedy"])
        rows.append((0.0 if kind == "greedy" else rng.choice([0.6, 0.8, 1.0, 1.0, 1.3]),
                     rng.choice([20, 40, 50, 200]) if kind in ("both", "top_k") else 0,
                     rng.choice([0.8, 0.9, 0.95]) if kind in ("both", "top_p") else 1.0,
                     rng.choice([0.0, 0.02, 0.1]) if cuts == "mixed" else 0.0))
    for i, (name, t) in enumerate((("temperature", torch.float32), ("top_k", torch.int32), ("top_p", torch.float32), ("min_p", torch.float32))):
        s[name] = torch.tensor([r[i] for r in rows], dtype=t, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    {"extend": _prepare_extend, "attend": _prepare_attend, "linear": _prepare_linear,
     "sample": _prepare_sample}[case["op"]](s, gen, random.Random(seed))
    return s


# ------------------------------------------------------------------------------------- plain forms
def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_extend(s):
    page, T = s["page"], s["T"]
    table, ring = s["page_table"], s["free_pages"]
    B, W = table.shape
    F = ring.numel()
    head, count = s["pool"][0].long(), s["pool"][1].long()
    lens, new = s["seq_lens"].long().clamp(min=0), s["new_lens"].long()
    n = new.clamp(min=0)
    starts = torch.nn.functional.pad(n.cumsum(0), (1, 0))
    had = (lens + page - 1) // page
    want = (lens + n + page - 1) // page - had
    fits = (new >= 0) & (had + want <= W) & (starts[:-1] + n <= T)
    need = torch.where(fits, want, 0)
    off = need.cumsum(0) - need
    granted = fits & ((need == 0) | (off + need <= count))
    taken = torch.where(granted, need, 0).sum()
    # The pages of sequences that end go behind the ring's last, then new ones come from its front.
    col = torch.arange(W, device=table.device)
    back = ((new < 0)[:, None] & (col < had[:, None])).flatten()
    place = torch.where(back, (head + count + back.cumsum(0) - 1) % F, F)
    fresh = ring[(head + off[:, None] + col - had[:, None]) % F]
    ring_out = torch.cat([ring, ring[:1]]).scatter(0, place, table.flatten())[:F]
    ring.copy_(ring_out)
    table.copy_(torch.where(granted[:, None] & (col >= had[:, None]) & (col < (had + want)[:, None]), fresh, table))
    t = torch.arange(T, device=table.device)
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=B - 1)
    inside = t < starts[-1]
    pos = torch.where(inside, lens[b] + t - starts[b], 0)
    id = table[b, (pos // page).clamp(max=W - 1)].long()
    slots = torch.where(inside & granted[b] & (id >= 0), id * page + pos % page, -1)
    pool = torch.stack([(head + taken) % F, (count - taken + back.sum()).clamp(max=F), torch.where(granted, 0, need).sum()]).int()
    return {"slots": slots, "positions": pos.int(), "starts": starts.int(),
            "seq_lens": torch.where(granted, lens + n, torch.where(new < 0, 0, lens)).int(), "pool": pool,
            "page_table": table, "free_pages": ring}


def _plain_attend(s):
    B, Hq, Hk, D, page = (s[k] for k in ("B", "Hq", "Hk", "D", "page"))
    # The visible places: the first tokens, then the last ones that are not among them.
    sinks, window, lens = min(s["sinks"], s["L"]), min(s["window"], s["L"]), s["seq_lens"].long()[:, None]
    start = torch.maximum(lens - window, lens.clamp(max=sinks))
    pos = torch.cat([torch.arange(sinks, device="cuda").expand(B, sinks), start + torch.arange(window, device="cuda")], 1)
    seen = pos < lens
    seen[:, :sinks] &= torch.arange(sinks, device="cuda") < start
    pos = torch.where(seen, pos, 0)
    at, off = s["page_table"].clamp(min=0).long().gather(1, pos // page), pos % page
    k = _values(s["k_cache"][at, :, off]) * s["k_scale"][at, :, off].unsqueeze(-1)  # [B, seen, Hk, D]
    q = (_values(s["q"]) * s["q_scale"].unsqueeze(-1)).view(B, Hk, Hq // Hk, D)
    score = torch.einsum("bhgd,blhd->bhgl", q, k) * D ** -0.5
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    v = _values(s["v_cache"][at, :, off]) * s["v_scale"][at, :, off].unsqueeze(-1)
    out = torch.einsum("bhgl,blhd->bhgd", p / total.clamp(min=1e-30), v)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return {"out": out.reshape(B, Hq, D).to(DTYPES[s["dtype"]]), "lse": lse.view(B, Hq)}


def _plain_linear(s):
    N, K = s["b"].shape
    a = _values(s["a"]) * s["a_scale"].repeat_interleave(GROUP, 1)[:, :K]
    b = _values(s["b"]) * s["b_scale"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
    y = a @ b.t()
    if s["bias"]:
        y = y + s["bias_row"].float()
    act = s["act"]
    if act == "relu":
        y = y.clamp(min=0.0)
    elif act == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    elif act == "silu":
        y = y / (1.0 + (-y).exp())
    if s["residual"]:
        y = y + s["stream"].float()
    return {"out": y.to(DTYPES[s["dtype"]])}


def _plain_sample(s):
    # The running sums of a row are compared with borders: in 64 bits.
    B, V = s["B"], s["V"]
    x, order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
    rank = torch.arange(V, device="cuda")
    greedy = s["temperature"] <= 0
    heat = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    k = torch.where(greedy, 1, torch.where(s["top_k"] <= 0, V, s["top_k"]).clamp(max=V)).long()[:, None]
    top = x[:, :1].double()
    w = torch.where(torch.isinf(x), 0.0, ((x.double() - top) / heat).exp())
    run = torch.where(rank < k, w, 0.0).cumsum(1)
    total = run[:, -1:]
    before = torch.nn.functional.pad(run[:, :-1], (1, 0))
    kept = (rank < k) & ((before < s["top_p"].double()[:, None] * total) | (rank == 0)) & (w >= s["min_p"].double()[:, None])
    kept_sum = (w * kept).sum(1, keepdim=True)
    run = run.masked_fill(~kept, math.inf)
    pick = torch.searchsorted(run, s["u"].double()[:, None] * kept_sum, right=True)
    pick = torch.minimum(pick, kept.sum(1, keepdim=True).clamp(min=1) - 1)
    some = kept_sum[:, 0] > 0
    token = torch.where(some, order.gather(1, pick)[:, 0], -1)
    logprob = torch.where(some, (w.gather(1, pick) / kept_sum)[:, 0].log(), -math.inf)
    return {"token": token, "logprob": logprob.float()}


def run(s):
    op = s["op"]
    if not own:
        return {"extend": _plain_extend, "attend": _plain_attend, "linear": _plain_linear, "sample": _plain_sample}[op](s)
    import fp8_quant_memory_gb300 as fq
    if op == "extend":
        slots, positions, starts, lens, pool = fq.paged_extend(s["page_table"], s["seq_lens"], s["new_lens"], s["free_pages"],
                                                               s["pool"], s["page"], s["T"])
        return {"slots": slots, "positions": positions, "starts": starts, "seq_lens": lens, "pool": pool,
                "page_table": s["page_table"], "free_pages": s["free_pages"]}
    if op == "attend":
        out, lse = fq.paged_attention(s["q"], s["q_scale"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                      s["page_table"], s["seq_lens"], out_dtype=DTYPES[s["dtype"]], max_seq_len=s["L"],
                                      want_lse=True, window=s["window"], sinks=s["sinks"])
        return {"out": out, "lse": lse}
    if op == "linear":
        return {"out": fq.fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=DTYPES[s["dtype"]], bias=s["bias_row"],
                                     activation=None if s["act"] == "none" else s["act"], residual=s["stream"])}
    token, logprob = fq.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"], want_logprob=True)
    return {"token": token, "logprob": logprob}


# ------------------------------------------------------------------------------- 64-bit definitions
def _table64():
    """The value of each e4m3 code: sign, 4 exponent bits (bias 7), 3 fraction bits, no infinities."""
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        m = math.nan if (c & 127) == 127 else math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        v.append(-m if c & 128 else m)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _exact_extend(s):
    """One sequence after the other, on the host."""
    page, T = s["page"], s["T"]
    table, ring = s["page_table"].tolist(), s["free_pages"].tolist()
    head, count, _ = s["pool"].tolist()
    F, W = len(ring), len(table[0])
    free = [ring[(head + i) % F] for i in range(count)]
    given, back, asked, missing, full = [], [], 0, 0, False
    slots, positions, starts, out_lens = [-1] * T, [0] * T, [0], []
    for b, (n, m) in enumerate(zip(s["seq_lens"].tolist(), s["new_lens"].tolist())):
        start = starts[-1]
        starts.append(start + max(m, 0))
        owned = _ceil(n, page)
        if m < 0:
            back += table[b][:owned]
            out_lens.append(0)
            continue
        ok = _ceil(n + m, page) <= W and start + m <= T
        need = _ceil(n + m, page) - owned if ok else 0
        asked += need
        if ok and (need == 0 or asked <= count):
            table[b][owned:owned + need] = free[len(given):len(given) + need]
            given += free[len(given):len(given) + need]
            out_lens.append(n + m)
        else:
            missing += need
            out_lens.append(n)
            ok = False
        for i in range(m):
            if start + i < T:
                positions[start + i] = n + i
                if ok:
                    slots[start + i] = table[b][(n + i) // page] * page + (n + i) % page
    for j, id in enumerate(back):
        ring[(head + count + j) % F] = id
    pool = [(head + len(given)) % F, min(F, count - len(given) + len(back)), missing]

    def whole(v, t=torch.int32):
        return torch.tensor(v, dtype=t, device="cuda")
    return {"slots": whole(slots, torch.int64), "positions": whole(positions), "starts": whole(starts), "seq_lens": whole(out_lens),
            "pool": whole(pool), "page_table": whole(table), "free_pages": whole(ring)}


def _exact_attend(s):
    t = _table64()
    B, Hq, Hk, D, page = (s[k] for k in ("B", "Hq", "Hk", "D", "page"))
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        j = torch.arange(n, device="cuda")
        j = j[(j < s["sinks"]) | (j >= n - s["window"])]
        if n == 0:
            continue
        ids, off = s["page_table"][b].long()[j // page], j % page
        for h in range(Hk):
            rows = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k, v = (t[s[c + "_cache"][ids, h, off].int()] * s[c + "_scale"][ids, h, off].double()[:, None] for c in "kv")
            x = (t[s["q"][b, rows].int()] * s["q_scale"][b, rows].double()[:, None]) @ k.T / math.sqrt(D)
            lse[b, rows] = torch.logsumexp(x, 1)
            out[b, rows] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}


def _exact_linear(s):
    t = _table64()
    M, K = s["a"].shape
    N = s["b"].shape[0]
    rows = torch.arange(N, device="cuda") // GROUP
    cols = torch.arange(K, device="cuda") // GROUP
    a = t[s["a"].int()] * s["a_scale"].double()[:, cols]
    b = t[s["b"].int()] * s["b_scale"].double()[rows][:, cols]
    y = torch.matmul(a, b.T)
    if s["bias_row"] is not None:
        y += s["bias_row"].double()
    if s["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif s["act"] == "gelu":
        y *= torch.special.erfc(-y / math.sqrt(2)) / 2
    elif s["act"] == "gelu_tanh":
        y *= torch.sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3))
    elif s["act"] == "silu":
        y *= torch.sigmoid(y)
    if s["stream"] is not None:
        y += s["stream"].double()
    return {"out": y}


def _exact_sample(s):
    """Row by row, over the distinct values and how often each occurs."""
    token, logprob = [], []
    for b in range(s["B"]):
        x = s["logits"][b].double()
        heat, k, top_p, min_p = (s[n][b].item() for n in ("temperature", "top_k", "top_p", "min_p"))
        val, times = torch.unique(x[x > -math.inf], return_counts=True)
        if val.numel() == 0:
            token.append(-1)
            logprob.append(-math.inf)
            continue
        val, times = val.flip(0), times.flip(0)
        if heat <= 0:
            token.append(int((x == val[0]).nonzero()[0]))
            logprob.append(0.0)
            continue
        w = torch.exp((val - val[0]) / heat)
        if k > 0:
            times = torch.minimum(times, (k - (times.cumsum(0) - times)).clamp(min=0))
        run = (w * times).cumsum(0)
        border = top_p * run[-1]
        at = int((run < border).sum().clamp(max=len(w) - 1))  # the value at which the running sum reaches the border
        ahead = run[at] - w[at] * times[at]
        times[at + 1:] = 0
        times[at] = min(int(times[at]), max(1, math.ceil((border - ahead) / w[at]))) if top_p < 1 else times[at]
        times = torch.where(w >= min_p, times, 0)
        run = (w * times).cumsum(0)
        aim = s["u"][b].double() * run[-1]
        at = int((run <= aim).sum().clamp(max=int((times > 0).sum()) - 1))
        nth = min(int(times[at]) - 1, int((aim - (run[at] - w[at] * times[at])) / w[at]))
        token.append(int((x == val[at]).nonzero()[max(nth, 0)]))
        logprob.append(float(torch.log(w[at] / run[-1])))
    return {"token": torch.tensor(token, device="cuda"), "logprob": torch.tensor(logprob, dtype=torch.float64, device="cuda")}


def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": _exact_extend, "attend": _exact_attend, "linear": _exact_linear, "sample": _exact_sample}[case["op"]](s)
