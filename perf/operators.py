"""Measured calls of the FP8 serving operators: the block-scaled FP8 matrix product, the QKV prologue
that appends to a paged FP8 key-value cache, and the attention of one new token over that cache.

Each case is one pass through one operator. With ``own`` false, ``run`` computes the operator in plain
32-bit torch operations; with ``own`` true it makes the library call. ``exact`` computes the same
outputs in 64 bits from the definitions, written apart from the plain form.

e4m3 codes are returned as float8_e4m3fn tensors, the values the codes stand for.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 128
AMAX_FLOOR = 1e-4
FP8_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # One token through the QKV projection of a 4096-wide block with 32 + 8 + 8 heads of 128.
        dict(name="matmul_token", op="matmul", M=1, N=6144, K=4096, dtype="bf16"),
        # A decoding batch through a wide projection.
        dict(name="matmul_batch", op="matmul", M=64, N=8192, K=4096, dtype="bf16"),
        # A ragged chunk: no size is a multiple of a tile, the last scale block is partial.
        dict(name="matmul_ragged", op="matmul", M=333, N=1111, K=1968, dtype="fp16"),
        # A 4096-token prompt through the QKV projection.
        dict(name="matmul_prompt", op="matmul", M=4096, N=6144, K=4096, dtype="bf16"),
        # A long prompt through a square projection of a wide model.
        dict(name="matmul_large", op="matmul", M=8192, N=8192, K=8192, dtype="bf16"),
        # A decoding batch's new rows go into the cache (latency).
        dict(name="append_batch", op="append", T=64, Hq=32, Hk=8, D=128, R=128, page=64, dtype="bf16", table="fp32"),
        # A 4096-token prompt's rows go into the cache, as many of them as the prologue benchmark has.
        dict(name="append_prompt", op="append", T=4096, Hq=32, Hk=8, D=128, R=128, page=64, dtype="bf16", table="fp32"),
        # The first tokens of one conversation (latency).
        dict(name="attend_short", op="attend", B=1, L=100, Hq=32, Hk=8, D=128, page=16, dtype="bf16"),
        # One conversation of 131072 tokens: the length has to be split to fill the GPU.
        dict(name="attend_long", op="attend", B=1, L=131072, Hq=64, Hk=8, D=128, page=64, dtype="bf16"),
        # A decoding batch whose lengths run from 0 to 8192.
        dict(name="attend_batch", op="attend", B=64, L=8192, Hq=32, Hk=8, D=128, page=64, dtype="bf16"),
        # Heads of 64 without sharing, pages that are no power of two, fp16 output.
        dict(name="attend_heads", op="attend", B=17, L=2500, Hq=16, Hk=16, D=64, page=24, dtype="fp16"),
        # Heads of 256, sixteen query heads on one key head.
        dict(name="attend_wide", op="attend", B=40, L=4096, Hq=32, Hk=2, D=256, page=32, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "matmul":
        M, N = _spread(rng, 1, 8192), _spread(rng, 64, 8192)
        K = 128 * _spread(rng, 1, 64) if rng.random() < 0.7 else 16 * _spread(rng, 1, 512)
        return dict(op=op, M=M, N=N, K=K, dtype=dtype)
    D = rng.choice([64, 96, 128, 128, 192, 256])
    page = rng.choice([8, 16, 16, 24, 32, 64, 64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    if op == "append":
        T = _spread(rng, 1, 4096)
        Hq = Hk * rng.choice([1, 2, 3, 4])
        if D > 128:
            T = max(1, T // 2)
        return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D, D // 2]), page=page, dtype=dtype,
                    table=rng.choice(["fp32", "fp32", dtype]))
    Hq = Hk * rng.choice([1, 2, 4, 4, 5, 8, 16])
    B = _spread(rng, 1, 128)
    most = min(131072, (64 * 8192 * 8 * 128) // (B * max(Hk, Hq // 8) * max(D, 128)))
    return dict(op=op, B=B, L=_spread(rng, 1, most), Hq=Hq, Hk=Hk, D=D, page=page, dtype=dtype)


def _lengths(case):
    """The batch's lengths, evenly spread over [0, L], the longest of them L; one sequence has length L."""
    B, L = case["B"], case["L"]
    return [L] if B == 1 else [(L * i) // (B - 1) for i in range(B)]


def work(case):
    op = case["op"]
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        g = -(-K // GROUP)
        return {"bytes": M * K + N * K + 4 * g * (M + -(-N // GROUP)) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "append":
        T, Hq, Hk, D, R = (case[k] for k in ("T", "Hq", "Hk", "D", "R"))
        rows = T * (Hq + 2 * Hk)
        table = 2 * T * (R // 2) * (4 if case["table"] == "fp32" else 2)
        return {"bytes": rows * D * 3 + rows * 4 + table + 8 * T + 4 * D, "flops": rows * 10 * D}
    B, Hq, Hk, D, page = (case[k] for k in ("B", "Hq", "Hk", "D", "page"))
    lens = _lengths(case)
    tokens, pages = sum(lens), sum(-(-n // page) for n in lens)
    return {"bytes": tokens * Hk * (2 * D + 8) + B * Hq * (D + 4 + 2 * D + 4) + 4 * B + 4 * pages,
            "flops": 4 * tokens * Hq * D}


# ------------------------------------------------------------------------------------------ inputs
def _codes(x, groups=None):
    """e4m3 codes (uint8) and 32-bit scales of the rows of x, or of its groups of columns."""
    if groups is None:
        s = x.abs().amax(-1, keepdim=True).clamp(min=AMAX_FLOOR) / FP8_MAX
        return (x / s).to(torch.float8_e4m3fn).view(torch.uint8), s.squeeze(-1)
    rows, K = x.shape
    n = -(-K // groups)
    y = torch.nn.functional.pad(x, (0, n * groups - K)).view(rows, n, groups)
    s = y.abs().amax(-1).clamp(min=AMAX_FLOOR) / FP8_MAX
    q = (y / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, n * groups)
    return q[:, :K].contiguous(), s


def _cache(shape, gen, std=1.0):
    """A cache's codes [pages, heads, page, D] and scales [pages, heads, page], of normal values."""
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for p in range(0, shape[0], step):
        n = min(step, shape[0] - p)
        codes[p:p + n], scale[p:p + n] = _codes(std * torch.randn((n, *shape[1:]), device="cuda", generator=gen))
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        # Activations after a norm, one scale per token and 128 columns; a projection's weights, one scale
        # per 128 x 128 block.
        s["a"], s["a_scale"] = _codes(torch.randn(M, K, device="cuda", generator=gen), GROUP)
        n, g = -(-N // GROUP), -(-K // GROUP)
        w = torch.randn(n * GROUP, g * GROUP, device="cuda", generator=gen) * (K ** -0.5)
        w[N:], w[:, K:] = 0.0, 0.0
        blocks = w.view(n, GROUP, g, GROUP)
        bs = blocks.abs().amax((1, 3)).clamp(min=AMAX_FLOOR) / FP8_MAX
        q = (blocks / bs[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n * GROUP, g * GROUP)
        s["b"], s["b_scale"] = q[:N, :K].contiguous(), bs
        return s
    if case["op"] == "append":
        T, Hq, Hk, D, R, page = (case[k] for k in ("T", "Hq", "Hk", "D", "R", "page"))
        s["qkv"] = (2.0 * torch.randn(T, (Hq + 2 * Hk) * D, device="cuda", generator=gen)).to(dtype)
        s["wq"], s["wk"] = ((1.0 + 0.1 * torch.randn(D, device="cuda", generator=gen)).to(dtype) for _ in range(2))
        pos = torch.arange(T, device="cuda", dtype=torch.float64) + rng.randrange(4096)
        angle = pos[:, None] * 1e4 ** (-2.0 * torch.arange(R // 2, device="cuda", dtype=torch.float64) / R)
        s["cos"], s["sin"] = angle.cos().to(DTYPES[case["table"]]), angle.sin().to(DTYPES[case["table"]])
        pages = -(-T // page) + 2
        s["k_cache"], s["k_scale"] = _cache((pages, Hk, page, D), gen)
        s["v_cache"], s["v_scale"] = _cache((pages, Hk, page, D), gen)
        # The prompt's tokens fill pages taken from a pool in any order; every 16th token is padding.
        order = torch.randperm(pages, device="cuda", generator=gen)
        t = torch.arange(T, device="cuda") + rng.randrange(page)
        s["slots"] = torch.where(torch.arange(T, device="cuda") % 16 == 15, -1, order[t // page] * page + t % page)
        return s
    B, Hq, Hk, D, page = (case[k] for k in ("B", "Hq", "Hk", "D", "page"))
    lens = _lengths(case)
    rng.shuffle(lens)
    s["q"], s["q_scale"] = _codes(1.5 * torch.randn(B, Hq, D, device="cuda", generator=gen))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    s["k_cache"], s["k_scale"] = _cache((pages, Hk, page, D), gen)
    s["v_cache"], s["v_scale"] = _cache((pages, Hk, page, D), gen)
    order = torch.randperm(pages, device="cuda", generator=gen).int()
    first = torch.tensor([sum(need[:i]) for i in range(B)], device="cuda")
    col = torch.arange(max(need), device="cuda")
    used = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    s["page_table"] = torch.where(used, order[(first[:, None] + col).clamp(max=pages - 1)], -1).int()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------- plain forms
def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _quantise(y):
    scale = y.abs().amax(-1).clamp(min=AMAX_FLOOR) / FP8_MAX
    return (y / scale.unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn), scale


def _plain_matmul(s):
    N, K = s["b"].shape
    a = _values(s["a"]) * s["a_scale"].repeat_interleave(GROUP, 1)[:, :K]
    b = _values(s["b"]) * s["b_scale"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]
    return {"out": (a @ b.t()).to(DTYPES[s["dtype"]])}


def _plain_append(s):
    T, Hq, Hk, D, R, page = (s[k] for k in ("T", "Hq", "Hk", "D", "R", "page"))
    x = s["qkv"].float().view(T, Hq + 2 * Hk, D)
    qk, v = x[:, :Hq + Hk], x[:, Hq + Hk:]
    w = torch.cat([s["wq"].float().expand(Hq, D), s["wk"].float().expand(Hk, D)])
    y = qk * (qk.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
    lo, hi = y[..., D - R:D - R // 2], y[..., D - R // 2:]
    c, n = s["cos"].float()[:, None], s["sin"].float()[:, None]
    y = torch.cat([y[..., :D - R], lo * c - hi * n, hi * c + lo * n], -1)
    codes, scale = _quantise(y)
    v_codes, v_scale = _quantise(v)
    kept = s["slots"] >= 0
    at, off = s["slots"][kept] // page, s["slots"][kept] % page
    s["k_cache"][at, :, off] = codes[kept, Hq:].view(torch.uint8)
    s["k_scale"][at, :, off] = scale[kept, Hq:]
    s["v_cache"][at, :, off] = v_codes[kept].view(torch.uint8)
    s["v_scale"][at, :, off] = v_scale[kept]
    return codes[:, :Hq].contiguous(), scale[:, :Hq].contiguous()


def _plain_attend(s):
    B, Hq, Hk, D, page, L = (s[k] for k in ("B", "Hq", "Hk", "D", "page", "L"))
    pos = torch.arange(L, device="cuda")
    at, off = s["page_table"].clamp(min=0).long()[:, pos // page], (pos % page).expand(B, L)
    k = _values(s["k_cache"][at, :, off]) * s["k_scale"][at, :, off].unsqueeze(-1)  # [B, L, Hk, D]
    q = (_values(s["q"]) * s["q_scale"].unsqueeze(-1)).view(B, Hk, Hq // Hk, D)
    score = torch.einsum("bhgd,blhd->bhgl", q, k) * D ** -0.5
    del k
    score = score.masked_fill(pos >= s["seq_lens"][:, None, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    v = _values(s["v_cache"][at, :, off]) * s["v_scale"][at, :, off].unsqueeze(-1)
    out = torch.einsum("bhgl,blhd->bhgd", p / total.clamp(min=1e-30), v)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return {"out": out.reshape(B, Hq, D).to(DTYPES[s["dtype"]]), "lse": lse.view(B, Hq)}


def run(s):
    op = s["op"]
    if own:
        import fp8_quant_memory_gb300 as fq
    if op == "matmul":
        if own:
            return {"out": fq.fp8_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=DTYPES[s["dtype"]])}
        return _plain_matmul(s)
    if op == "append":
        if own:
            q, q_scale = fq.qkv_norm_rope_append(s["qkv"], s["wq"], s["wk"], s["cos"], s["sin"], s["slots"],
                                                 s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                                 s["Hq"], s["Hk"], eps=EPS, fp8_max=FP8_MAX, rope_dim=s["R"])
            q = q.view(torch.float8_e4m3fn)
        else:
            q, q_scale = _plain_append(s)
        f8 = torch.float8_e4m3fn
        return {"q": q, "q_scale": q_scale, "k_cache": s["k_cache"].view(f8), "k_scale": s["k_scale"],
                "v_cache": s["v_cache"].view(f8), "v_scale": s["v_scale"]}
    if own:
        out, lse = fq.paged_attention(s["q"], s["q_scale"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                      s["page_table"], s["seq_lens"], out_dtype=DTYPES[s["dtype"]],
                                      max_seq_len=s["L"], want_lse=True)
        return {"out": out, "lse": lse}
    return _plain_attend(s)


# ------------------------------------------------------------------------------- 64-bit definitions
def _table64():
    """The value of each e4m3 code: sign, 4 exponent bits (bias 7), 3 fraction bits, no infinities."""
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        m = math.nan if (c & 127) == 127 else math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        v.append(-m if c & 128 else m)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _round64(y):
    """The nearest e4m3 value (ties to the even code) of 64-bit values within +-448."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_matmul(s):
    t = _table64()
    M, K = s["a"].shape
    N = s["b"].shape[0]
    rows = torch.arange(N, device="cuda") // GROUP
    cols = torch.arange(K, device="cuda") // GROUP
    a = t[s["a"].int()] * s["a_scale"].double()[:, cols]
    b = t[s["b"].int()] * s["b_scale"].double()[rows][:, cols]
    return {"out": torch.matmul(a, b.T)}


def _exact_append(s):
    t = _table64()
    T, Hq, Hk, D, R, page = (s[k] for k in ("T", "Hq", "Hk", "D", "R", "page"))
    q, q_scale = [], []
    k_cache, v_cache = t[s["k_cache"].int()], t[s["v_cache"].int()]
    k_scale, v_scale = s["k_scale"].double(), s["v_scale"].double()
    live = (s["slots"] >= 0).nonzero().flatten()
    slot = s["slots"][live]
    for h in range(Hq + 2 * Hk):
        x = s["qkv"][:, h * D:(h + 1) * D].double()
        if h < Hq + Hk:
            x = x / torch.sqrt((x * x).sum(1, keepdim=True) / D + EPS) * (s["wq"] if h < Hq else s["wk"]).double()
            y = x.clone()
            for i in range(R // 2):
                u, v, c, n = x[:, D - R + i], x[:, D - R + R // 2 + i], s["cos"][:, i].double(), s["sin"][:, i].double()
                y[:, D - R + i], y[:, D - R + R // 2 + i] = u * c - v * n, v * c + u * n
            x = y
        scale = torch.clamp(x.abs().max(1).values, min=AMAX_FLOOR) / FP8_MAX
        val = _round64(x / scale[:, None])
        if h < Hq:
            q.append(val)
            q_scale.append(scale)
        else:
            j = (h - Hq) % Hk
            cache, held = (k_cache, k_scale) if h < Hq + Hk else (v_cache, v_scale)
            cache[slot // page, j, slot % page] = val[live]
            held[slot // page, j, slot % page] = scale[live]
    return {"q": torch.stack(q, 1), "q_scale": torch.stack(q_scale, 1), "k_cache": k_cache, "k_scale": k_scale,
            "v_cache": v_cache, "v_scale": v_scale}


def _exact_attend(s):
    t = _table64()
    B, Hq, Hk, D, page = (s[k] for k in ("B", "Hq", "Hk", "D", "page"))
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n == 0:
            continue
        ids = s["page_table"][b, :-(-n // page)].long()
        for h in range(Hk):
            rows = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            k, v = ((t[s[c + "_cache"][ids, h].int()] * s[c + "_scale"][ids, h].double()[..., None]).reshape(-1, D)[:n]
                    for c in "kv")
            x = (t[s["q"][b, rows].int()] * s["q_scale"][b, rows].double()[:, None]) @ k.T / math.sqrt(D)
            lse[b, rows] = torch.logsumexp(x, 1)
            out[b, rows] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"matmul": _exact_matmul, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
