"""GPU parity of the FP8 serving operators against plain 64-bit implementations (serving_ref.py): the
sizes, layouts and masks where each can go wrong, their refusals, streams and graph capture, and a run of
them together as a decoding step uses them."""
import math

import pytest
import torch

import fp8_quant_memory_gb300 as fq
import serving_ref as ref
from fp8_quant_memory_gb300 import workloads as wl
from guards import Guarded
from parity import assert_codes_close, assert_scale_close

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(autouse=True)
def _device_state(cuda_ok):
    yield
    torch.cuda.synchronize()
    assert fq.device_status(clear=True) == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------- matrix product
def matmul_inputs(M, N, K, seed, pad=0):
    g = gen(seed)
    G, NB = -(-K // 128), -(-N // 128)
    a = torch.zeros(M, K + pad, dtype=torch.uint8)
    b = torch.zeros(N, K + pad, dtype=torch.uint8)
    a[:, :K], b[:, :K] = ref.finite_codes((M, K), g), ref.finite_codes((N, K), g)
    sa = torch.rand(M, G, generator=g) * 2e-2 + 1e-4
    sb = torch.rand(NB, G, generator=g) * 2e-4 + 1e-6
    return [t.cuda() for t in (a, sa, b, sb)]


MATMUL_SIZES = [
    (1, 1, 1), (1, 1, 128), (1, 128, 128), (1, 129, 16), (2, 64, 127), (3, 257, 130), (5, 1000, 1040), (8, 128, 256),
    (16, 384, 4096), (17, 640, 2048), (31, 100, 144), (32, 129, 400), (33, 127, 384), (63, 256, 1152), (64, 1024, 512),
    (65, 300, 640), (100, 77, 96), (127, 255, 272), (128, 128, 128), (129, 129, 129), (130, 512, 2048), (200, 1111, 1968),
    (256, 256, 256), (257, 385, 528), (300, 2049, 128), (512, 1000, 16), (777, 500, 1280), (1025, 513, 784), (1, 4096, 8192),
    (2048, 1, 64), (1536, 1280, 256),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("size", MATMUL_SIZES, ids=lambda s: "%dx%dx%d" % s)
def test_matmul(size, dt):
    M, N, K = size
    a, sa, b, sb = matmul_inputs(M, N, K, seed=M + 3 * N + 7 * K)
    out = Guarded((M, N), DT[dt], fill=math.nan)
    got = fq.fp8_matmul(a, sa, b, sb, out=out.t)
    out.check()
    ref.assert_matmul(got, a, sa, b, sb)


@pytest.mark.parametrize("size", [(60, 16000, 1712), (33, 8100, 3216), (64, 4100, 6928)], ids=str)
def test_matmul_weights_of_many_tiles(size):
    """33 to 64 rows of 13 to 14 blocks of k per CTA, whose sums are kept in two halves; k whole, in two, in four."""
    M, N, K = size
    a, sa, b, sb = matmul_inputs(M, N, K, seed=N)
    out = Guarded((M, N), torch.bfloat16, fill=math.nan)
    got = fq.fp8_matmul(a, sa, b, sb, out=out.t)
    out.check()
    ref.assert_matmul(got, a, sa, b, sb)
    assert torch.equal(fq.fp8_matmul(a, sa, b, sb), got)


@pytest.mark.parametrize("size", [(7, 200, 256), (70, 200, 1024), (300, 400, 512)], ids=str)
def test_matmul_strided(size):
    """Padded rows of every operand and of the output; the padding stays as it was."""
    M, N, K = size
    a, sa, b, sb = matmul_inputs(M, N, K, seed=5, pad=48)
    sa2 = torch.full((M, sa.shape[1] + 3), math.nan, device="cuda")
    sa2[:, :sa.shape[1]] = sa
    sb2 = torch.full((sb.shape[0], sb.shape[1] + 1), math.nan, device="cuda")
    sb2[:, :sb.shape[1]] = sb
    buf = torch.full((M, N + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    a[:, K:], b[:, K:] = 0x7F, 0x7F  # NaN codes behind every row
    got = fq.fp8_matmul(a[:, :K], sa2[:, :sa.shape[1]], b[:, :K], sb2[:, :sb.shape[1]], out=buf[:, :N])
    ref.assert_matmul(got, a[:, :K], sa, b[:, :K], sb)
    assert bool((buf[:, N:] == 7.0).all())


@pytest.mark.parametrize("M,N,stride", [(2500, 2300, 2312), (2500, 2297, 2304), (2400, 2302, 2302 * 2), (2400, 2296, 2304), (2400, 2303, 2309)])
def test_matmul_padded_output_of_many_rows(M, N, stride):
    """Rows of the output a multiple of 16 bytes apart whose length is not one: what lies between them stays."""
    a, sa, b, sb = matmul_inputs(M, N, 1040, seed=11)
    buf = torch.full((M, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    got = fq.fp8_matmul(a, sa, b, sb, out=buf[:, :N])
    assert bool((buf[:, N:] == 7.0).all())
    ref.assert_matmul(got, a, sa, b, sb)


@pytest.mark.parametrize("size", [(9, 130, 256), (150, 260, 384)], ids=str)
def test_matmul_misaligned(size):
    """Operands one byte past a 16-byte boundary take the scalar kernel."""
    M, N, K = size
    a, sa, b, sb = matmul_inputs(M, N, K, seed=6)
    flat = torch.zeros(M * K + 16, dtype=torch.uint8, device="cuda")
    a1 = flat[1:1 + M * K].view(M, K)
    a1.copy_(a)
    ref.assert_matmul(fq.fp8_matmul(a1, sa, b, sb), a, sa, b, sb)


def test_matmul_broadcast_row():
    """A stride of 0 over the rows of a and of its scales."""
    a, sa, b, sb = matmul_inputs(1, 200, 256, seed=8)
    out = fq.fp8_matmul(a.expand(40, 256), sa.expand(40, 2), b, sb)
    ref.assert_matmul(out, a.expand(40, 256).contiguous(), sa.expand(40, 2).contiguous(), b, sb)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_matmul_nan_and_zero_scales(M):
    """A NaN code reaches exactly its row or column; a zero scale gives zero."""
    a, sa, b, sb = matmul_inputs(M, 260, 512, seed=9)
    clean = fq.fp8_matmul(a, sa, b, sb)
    a2, b2 = a.clone(), b.clone()
    a2[M - 1, 300], b2[7, 5] = 0x7F, 0xFF
    out = fq.fp8_matmul(a2, sa, b2, sb)
    hit = torch.zeros(M, 260, dtype=torch.bool, device="cuda")
    hit[M - 1], hit[:, 7] = True, True
    assert torch.equal(out.isnan(), hit)
    assert torch.equal(out[~hit], clean[~hit])
    sa2 = sa.clone()
    sa2[0] = 0.0
    assert bool((fq.fp8_matmul(a, sa2, b, sb)[0] == 0).all())


def test_matmul_operand_beyond_32_bits():
    """Rows of a behind its first 2^32 bytes."""
    M, N, K = 33000, 48, 131072
    a = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    sa = torch.ones(M, K // 128, device="cuda")
    tail, stail, b, sb = matmul_inputs(20, N, K, seed=4)
    a[-20:], sa[-20:] = tail, stail
    out = fq.fp8_matmul(a, sa, b, sb)
    ref.assert_matmul(out[-20:], tail, stail, b, sb)
    assert not bool(out[:-20].any())


def test_matmul_columns_beyond_2_to_the_30():
    """One row, more columns than 2^30: those on either side of it, and nothing else, have weights."""
    M, N, K = 1, (1 << 30) + 256, 16
    tail = 512
    a, sa, bt, sbt = matmul_inputs(M, tail, K, seed=12)
    b = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    sb = torch.ones(N // 128, 1, device="cuda")
    b[-tail:], sb[-tail // 128:] = bt, sbt
    out = torch.full((M, N), math.nan, dtype=torch.bfloat16, device="cuda")
    fq.fp8_matmul(a, sa, b, sb, out=out)
    ref.assert_matmul(out[:, -tail:], a, sa, bt, sbt)
    assert not bool(out[:, :-tail].any())


def test_matmul_empty():
    a, sa, b, sb = matmul_inputs(4, 6, 128, seed=1)
    assert fq.fp8_matmul(a[:0], sa[:0], b, sb).shape == (0, 6)
    assert fq.fp8_matmul(a, sa, b[:0], sb[:0]).shape == (4, 0)


@pytest.mark.parametrize("size", [(1, 4096, 4096), (333, 1111, 1968), (1024, 1024, 1024)], ids=str)
def test_matmul_repeats_bit_for_bit(size):
    a, sa, b, sb = matmul_inputs(*size, seed=2)
    first = fq.fp8_matmul(a, sa, b, sb)
    for _ in range(5):
        assert torch.equal(fq.fp8_matmul(a, sa, b, sb), first)


def test_matmul_float8_tensors_and_refusals():
    a, sa, b, sb = matmul_inputs(5, 130, 256, seed=3)
    f8 = torch.float8_e4m3fn
    assert torch.equal(fq.fp8_matmul(a.view(f8), sa, b.view(f8), sb), fq.fp8_matmul(a, sa, b, sb))
    bad = [dict(a=a[:, :128]), dict(a=a.float()), dict(sa=sa[:, :1]), dict(sb=sb[:1]), dict(sa=sa.double()), dict(a=a.cpu()),
           dict(a=a.t().contiguous().t()), dict(out=torch.empty(5, 130, device="cuda")), dict(out_dtype=torch.float32),
           dict(out=torch.empty(5, 131, device="cuda", dtype=torch.bfloat16))]
    for over in bad:
        args = dict(a=a, sa=sa, b=b, sb=sb) | {k: v for k, v in over.items() if k in ("a", "sa", "b", "sb")}
        kw = {k: v for k, v in over.items() if k not in args}
        with pytest.raises((ValueError, fq.FqError)):
            fq.fp8_matmul(args["a"], args["sa"], args["b"], args["sb"], **kw)


# --------------------------------------------------------------------------------------- append
def make_cache(P, Hk, page, D, seed, order="phtd", offset=0):
    """(k, v, ks, vs) viewed as [P, Hk, page, D]; order names the axes in memory."""
    g = gen(seed)
    sizes = dict(p=P, h=Hk, t=page)
    dims = [sizes[c] for c in order if c != "d"]
    perm = [[c for c in order if c != "d"].index(c) for c in "pht"]
    out = []
    for _ in range(2):
        flat = torch.zeros(P * Hk * page * D + 16, dtype=torch.uint8, device="cuda")
        t = flat[offset:offset + P * Hk * page * D].view(*dims, D)
        t.copy_(ref.finite_codes((*dims, D), g))
        out.append(t.permute(*perm, 3))
    for _ in range(2):
        out.append((torch.rand(*dims, generator=g) * 0.01 + 1e-3).cuda().permute(*perm))
    return out


APPEND_CASES = [
    # T, Hq, Hk, D, R, page, dtype, table, extra columns, fp8_max, order
    (1, 32, 8, 128, 128, 64, "bf16", "fp32", 0, 448.0, "phtd"),
    (37, 32, 8, 128, 128, 16, "bf16", "fp32", 0, 448.0, "phtd"),
    (64, 4, 2, 64, 64, 7, "fp16", "fp16", 0, 448.0, "pthd"),
    (50, 6, 2, 128, 64, 24, "bf16", "bf16", 128, 448.0, "pthd"),
    (33, 3, 1, 256, 256, 1, "bf16", "fp32", 0, 240.0, "phtd"),
    (41, 5, 3, 96, 96, 16, "fp16", "fp32", 8, 448.0, "hptd"),
    (29, 2, 2, 192, 96, 32, "bf16", "fp32", 0, 448.0, "phtd"),
    (13, 0, 2, 128, 128, 16, "bf16", "fp32", 0, 448.0, "phtd"),
    (19, 3, 1, 80, 40, 16, "bf16", "fp32", 0, 448.0, "phtd"),
    (11, 2, 2, 100, 50, 16, "bf16", "bf16", 0, 448.0, "phtd"),
    (9, 2, 1, 128, 0, 16, "bf16", "fp32", 0, 448.0, "phtd"),
    (17, 4, 4, 512, 512, 8, "bf16", "fp32", 0, 448.0, "phtd"),
    (23, 4, 4, 128, 128, 16, "bf16", "fp16", 0, 448.0, "phtd"),
    (1500, 8, 2, 128, 128, 64, "bf16", "fp32", 0, 448.0, "phtd"),
    (1300, 7, 3, 128, 128, 64, "fp16", "fp32", 0, 448.0, "pthd"),
    (700, 16, 8, 128, 128, 24, "bf16", "bf16", 0, 240.0, "phtd"),
    (6000, 0, 2, 128, 128, 64, "fp16", "fp16", 0, 448.0, "phtd"),
    (400, 32, 8, 128, 128, 64, "bf16", "fp32", 0, 448.0, "hptd"),
]


def append_inputs(case, seed=40):
    T, Hq, Hk, D, R, page, dt, tdt, extra, fmax, order = case
    d = wl.qk_inputs(T, Hq, 2 * Hk, D, dt, tdt, seed=seed, std=2.0, rope_dim=R,
                     token_stride=(Hq + 2 * Hk) * D + extra)
    pages = -(-T // page) + 2
    cache = make_cache(pages, Hk, page, D, seed + 1, order)
    perm = torch.randperm(pages * page, generator=gen(seed + 2))[:T]
    slots = torch.where(torch.arange(T) % 5 == 3, torch.tensor([-1, pages * page, -(1 << 40), 1 << 40])[torch.arange(T) % 4], perm)
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}, cache, slots.cuda()


def check_append(d, cache0, cache, slots, q, qs, case):
    T, Hq, Hk, D, R, page, dt, tdt, extra, fmax, order = case
    y, scale = ref.append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], Hq, Hk, D, R, fp8_max=fmax)
    codes = ref.e4m3_codes(y / scale[..., None])
    assert_codes_close(q, codes[:, :Hq])
    assert_scale_close(qs, scale[:, :Hq])
    k, v, ks, vs = (t.cpu() for t in cache)
    k0, v0, ks0, vs0 = (t.cpu().clone() for t in cache0)
    P = k.shape[0]
    sl = slots.cpu()
    live = (sl >= 0) & (sl < P * page)
    at, off = sl[live] // page, sl[live] % page
    assert_codes_close(k[at, :, off], codes[live, Hq:Hq + Hk])
    assert_scale_close(ks[at, :, off], scale[live, Hq:Hq + Hk])
    # V: the per-row quantiser of 32-bit division, exactly
    x = d["qk"].cpu()[:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].float().view(T, Hk, D)
    s32 = x.abs().amax(-1).clamp(min=1e-4) / torch.tensor(fmax, dtype=torch.float32)
    want = ref.e4m3_codes((x / s32[..., None]).clamp(-fmax, fmax).double())
    assert torch.equal(vs[at, :, off], s32[live])
    assert torch.equal(v[at, :, off], want[live])
    # every other slot as it was
    for got, was, new in ((k, k0, k[at, :, off]), (v, v0, want[live]), (ks, ks0, ks[at, :, off]), (vs, vs0, s32[live])):
        was[at, :, off] = new
        assert torch.equal(got, was)


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "T%d-%d+%d-D%d-R%d-p%d-%s-%s-x%d-m%g-%s" % c)
def test_append(case):
    T, Hq, Hk, D, R, page, dt, tdt, extra, fmax, order = case
    d, cache, slots = append_inputs(case)
    before = [t.clone() for t in cache]
    q, qs = Guarded((T, Hq, D), torch.uint8), Guarded((T, Hq), torch.float32)
    fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, Hq, Hk, fp8_max=fmax,
                            rope_dim=R, q_out=q.t, q_scale=qs.t)
    q.check("q")
    qs.check("q_scale")
    check_append(d, before, cache, slots, q.t.cpu(), qs.t.cpu(), case)


def test_append_misaligned_cache():
    case = (21, 4, 2, 128, 128, 16, "bf16", "fp32", 0, 448.0, "phtd")
    d, _, slots = append_inputs(case)
    cache = make_cache(4, 2, 16, 128, 9, offset=3)
    slots = torch.where(slots < 64, slots, -1)
    before = [t.clone() for t in cache]
    q, qs = fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, 4, 2)
    check_append(d, before, cache, slots, q.cpu(), qs.cpu(), case)


@pytest.mark.parametrize("T,D,page", [(40, 128, 16), (400, 128, 64), (30, 96, 7), (20, 256, 16), (9, 100, 16)])
def test_append_into_rows_of_a_wider_cache(T, D, page):
    """A cache that is the first D columns of wider rows; what lies behind them stays."""
    Hq, Hk = 32, 8
    case = (T, Hq, Hk, D, D if D % 16 == 0 else 0, page, "bf16", "fp32", 0, 448.0, "phtd")
    d, cache, slots = append_inputs(case)
    wide = [torch.full((*c.shape[:3], D + 32), 0x55, dtype=torch.uint8, device="cuda") for c in cache[:2]]
    for w, c in zip(wide, cache):
        w[..., :D] = c
    cache = [w[..., :D] for w in wide] + cache[2:]
    before = [t.clone() for t in cache]
    q, qs = fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, Hq, Hk, rope_dim=case[4])
    check_append(d, before, cache, slots, q.cpu(), qs.cpu(), case)
    assert all(bool((w[..., D:] == 0x55).all()) for w in wide)


def test_append_matches_prologue():
    """q and k rows are the prologue's, up to the last place of its fp32 arithmetic."""
    case = (300, 32, 8, 128, 128, 64, "bf16", "fp32", 0, 448.0, "phtd")
    d, cache, _ = append_inputs(case)
    slots = torch.arange(300, device="cuda")
    q, qs = fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, 32, 8)
    pq, ps = fq.qk_norm_rope_quant(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], 32, 8)
    assert_codes_close(q, pq[:, :32].cpu())
    assert_scale_close(qs, ps[:, :32].cpu())
    at, off = slots // 64, slots % 64
    assert_codes_close(cache[0][at, :, off], pq[:, 32:].cpu())
    assert_scale_close(cache[2][at, :, off], ps[:, 32:].cpu())


def test_append_rows_beyond_32_bits():
    """A QKV batch of more than 2^31 elements: the last tokens as a small batch of them gives them."""
    T, Hq, Hk, D, page, n = 360000, 32, 8, 128, 64, 40
    d, small, _ = append_inputs((n, Hq, Hk, D, D, page, "bf16", "fp32", 0, 448.0, "phtd"))
    qkv = torch.zeros(T, (Hq + 2 * Hk) * D, dtype=torch.bfloat16, device="cuda")
    cos, sin = torch.ones(T, D // 2, device="cuda"), torch.zeros(T, D // 2, device="cuda")
    qkv[-n:], cos[-n:], sin[-n:] = d["qk"], d["cos"], d["sin"]
    P = T // page
    big = [torch.zeros(P, Hk, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros(P, Hk, page, device="cuda") for _ in range(2)]
    slots = torch.arange(T, device="cuda")
    q, qs = fq.qkv_norm_rope_append(qkv, d["wq"], d["wk"], cos, sin, slots, *big, Hq, Hk)
    q1, qs1 = fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots[:n], *small, Hq, Hk)
    assert_codes_close(q[-n:], q1.cpu())
    assert_scale_close(qs[-n:], qs1.cpu())
    at, off = slots[-n:] // page, slots[-n:] % page
    for x, y in zip(big[:2], small[:2]):
        assert_codes_close(x[at, :, off], y[0, :, :n].transpose(0, 1).cpu())
    for x, y in zip(big[2:], small[2:]):
        assert_scale_close(x[at, :, off], y[0, :, :n].transpose(0, 1).cpu())


def test_append_zero_rows_and_empty():
    case = (6, 4, 2, 128, 128, 16, "bf16", "fp32", 0, 448.0, "phtd")
    d, cache, _ = append_inputs(case)
    d["qk"].zero_()
    slots = torch.arange(6, device="cuda")
    q, qs = fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, 4, 2)
    floor = torch.tensor(1e-4) / torch.tensor(448.0)
    assert bool((qs.cpu() == floor).all()) and bool(((q & 0x7F) == 0).all())
    assert bool((cache[3][0, :, :6].cpu() == floor).all())
    before = [t.clone() for t in cache]
    q, qs = fq.qkv_norm_rope_append(d["qk"][:0], d["wq"], d["wk"], d["cos"][:0], d["sin"][:0], slots[:0], *cache, 4, 2)
    assert q.shape == (0, 4, 128) and all(torch.equal(x, y) for x, y in zip(before, cache))


NON_FINITE = [(400, 32, 8, 128, "bf16"), (400, 32, 8, 128, "fp16"), (9, 4, 2, 128, "bf16"), (7, 2, 2, 64, "fp16"),
              (5, 1, 3, 256, "bf16"), (6, 4, 2, 100, "bf16")]


@pytest.mark.parametrize("fmax", [448.0, 240.0])
@pytest.mark.parametrize("T,Hq,Hk,D,dt", NON_FINITE)
def test_append_infinities_and_nan_in_values(T, Hq, Hk, D, dt, fmax):
    """A V row that holds an infinity has an infinite scale, code 0 for its finite values (x / inf) and NaN for the
    infinity (inf / inf); a NaN is left out of the row's maximum and stays one. Other rows are as without them."""
    case = (T, Hq, Hk, D, D if D % 4 == 0 else 0, 16, dt, "fp32", 0, fmax, "phtd")
    d, cache, _ = append_inputs(case)
    slots = torch.arange(T, device="cuda")
    v = d["qk"][:, (Hq + Hk) * D:(Hq + 2 * Hk) * D].view(T, Hk, D)
    v[0, 0, 3], v[1, Hk - 1, D - 1], v[2, 0, D // 2] = math.inf, -math.inf, math.nan
    v[3, Hk - 1, 1], v[3, Hk - 1, D - 2] = math.inf, math.nan
    fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, Hq, Hk, fp8_max=fmax)
    x = v.cpu().float()
    s = x.abs().nan_to_num(nan=0.0, posinf=math.inf).amax(-1).clamp(min=1e-4) / torch.tensor(fmax)
    want = (x / s[..., None]).double()
    at, off = slots.cpu() // 16, slots.cpu() % 16
    got = cache[1].cpu()[at, :, off]
    assert torch.equal(cache[3].cpu()[at, :, off], s)
    nan = want.isnan()
    assert int(nan.sum()) == 5 and torch.equal((got & 0x7F) == 0x7F, nan)
    assert torch.equal(got[~nan], ref.e4m3_codes(want.clamp(-fmax, fmax))[~nan])


@pytest.mark.parametrize("fmax", [448.0, 240.0])
@pytest.mark.parametrize("T,Hq,Hk,D,dt", NON_FINITE)
def test_append_infinities_and_nan_in_normed_rows(T, Hq, Hk, D, dt, fmax):
    """Of a q or k row with an infinity (rstd = 0) its two rotated places are NaN and the others zero; a NaN makes the
    whole row NaN. Either way the scale is the floor's, and the token's other rows are as without them."""
    case = (T, Hq, Hk, D, D, 16, dt, "fp32", 0, fmax, "phtd")
    d, cache, _ = append_inputs(case)
    slots = torch.arange(T, device="cuda")

    def rows():
        q, qs = fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, Hq, Hk, fp8_max=fmax)
        at, off = slots // 16, slots % 16
        return torch.cat([q, cache[0][at, :, off]], 1).cpu(), torch.cat([qs, cache[2][at, :, off]], 1).cpu()

    clean, clean_scale = rows()
    x = d["qk"][:, :(Hq + Hk) * D].view(T, Hq + Hk, D)
    x[0, 0, 3], x[1, Hq, 5], x[2, Hq + Hk - 1, D - 1], x[3, Hq - 1, 0] = math.inf, -math.inf, math.nan, math.nan
    codes, scale = rows()
    nan = torch.zeros(codes.shape, dtype=torch.bool)
    hit = torch.zeros(scale.shape, dtype=torch.bool)
    for t, h, at in ((0, 0, [3, 3 + D // 2]), (1, Hq, [5, 5 + D // 2]), (2, Hq + Hk - 1, slice(None)), (3, Hq - 1, slice(None))):
        nan[t, h, at], hit[t, h] = True, True
    assert torch.equal((codes & 0x7F) == 0x7F, nan)
    assert bool(((codes[hit] & 0x7F)[~nan[hit]] == 0).all())
    assert bool((scale[hit] == torch.tensor(1e-4) / torch.tensor(fmax)).all())
    assert torch.equal(codes[~hit], clean[~hit]) and torch.equal(scale[~hit], clean_scale[~hit])


@pytest.mark.parametrize("T,Hq,Hk,D", [(400, 32, 8, 128), (9, 4, 2, 128), (7, 2, 2, 64), (6, 4, 2, 100)])
def test_append_rows_whose_squares_leave_fp32(T, Hq, Hk, D):
    """rstd is 0 and so is every finite value of the row, also where x * w or its rotation alone would overflow."""
    case = (T, Hq, Hk, D, D, 16, "bf16", "fp32", 0, 448.0, "phtd")
    d, cache, _ = append_inputs(case)
    slots = torch.arange(T, device="cuda")
    x = d["qk"][:, :(Hq + Hk) * D].view(T, Hq + Hk, D)
    rows = [(0, 0, 3.3e38), (1, Hq, -3e38), (2, Hq + Hk - 1, 1.5e38), (3, 1, 1e30), (4, Hq - 1, 2e19)]
    for t, h, v in rows:
        x[t, h] = v
    x[5, 0, 7:9] = 3.3e38
    q, qs = fq.qkv_norm_rope_append(d["qk"], d["wq"], d["wk"], d["cos"], d["sin"], slots, *cache, Hq, Hk)
    at, off = slots // 16, slots % 16
    codes, scale = torch.cat([q, cache[0][at, :, off]], 1).cpu(), torch.cat([qs, cache[2][at, :, off]], 1).cpu()
    for t, h in [(t, h) for t, h, _ in rows] + [(5, 0)]:
        assert bool(((codes[t, h] & 0x7F) == 0).all()), (t, h)
        assert scale[t, h] == torch.tensor(1e-4) / torch.tensor(448.0)


def test_append_refusals():
    case = (6, 4, 2, 128, 128, 16, "bf16", "fp32", 0, 448.0, "phtd")
    d, cache, slots = append_inputs(case)
    k, v, ks, vs = cache
    base = dict(qkv=d["qk"], wq=d["wq"], wk=d["wk"], cos=d["cos"], sin=d["sin"], slots=slots, k_cache=k, v_cache=v,
                k_scale=ks, v_scale=vs, Hq=4, Hk=2)
    for over in (dict(Hk=1), dict(Hq=-1), dict(Hq=9), dict(slots=slots.int()), dict(slots=slots[:5]), dict(qkv=d["qk"].float()),
                 dict(v_cache=v[:1]), dict(k_scale=ks.double()), dict(cos=d["cos"][:5]), dict(rope_dim=64), dict(rope_dim=63),
                 dict(fp8_max=500.0), dict(eps=-1.0), dict(wq=d["wq"].half()), dict(k_cache=k.cpu()),
                 dict(k_cache=k[:1].expand(k.shape), v_cache=v[:1].expand(v.shape))):
        with pytest.raises((ValueError, fq.FqError)):
            fq.qkv_norm_rope_append(**(base | over))


# ------------------------------------------------------------------------------------ attention
def attention_inputs(lens, Hq, Hk, D, page, seed, order="phtd", extra_pages=3, offset=0, q_extra=0):
    g = gen(seed)
    B = len(lens)
    need = [-(-max(n, 0) // page) for n in lens]
    P = sum(need) + extra_pages
    cache = make_cache(P, Hk, page, D, seed + 1, order, offset)
    qbuf = ref.finite_codes((B, Hq + q_extra, D), g).cuda()
    sbuf = (torch.rand(B, Hq + q_extra, generator=g) * 2e-4 + 1e-5).cuda()
    ids = torch.randperm(P, generator=g)
    table = torch.full((B, max(need + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n].int()
        at += n
    return [qbuf[:, :Hq], sbuf[:, :Hq], *cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")]


def check_attention(x, dt="bf16", scale=None, max_len=None):
    q, qs, k, v, ks, vs, table, lens = x
    B, Hq, D = q.shape
    out, lse = Guarded((B, Hq, D), DT[dt], fill=math.nan), Guarded((B, Hq), torch.float32, fill=math.nan)
    fq.paged_attention(q, qs, k, v, ks, vs, table, lens, softmax_scale=scale, max_seq_len=max_len, out=out.t, lse=lse.t)
    out.check("out")
    lse.check("lse")
    ref.assert_attention(out.t, lse.t, *x, D ** -0.5 if scale is None else scale, max_len=max_len)


ATTENTION_CASES = [
    # lens, Hq, Hk, D, page, dtype, order
    ([1], 1, 1, 128, 16, "bf16", "phtd"),
    ([100], 32, 8, 128, 16, "bf16", "phtd"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 128, 16, "bf16", "phtd"),
    ([127, 128, 129, 0, 255, 257], 8, 8, 64, 24, "fp16", "pthd"),
    ([1000, 3, 0, 400], 16, 1, 128, 1, "bf16", "phtd"),
    ([513, 64, 1], 32, 2, 256, 32, "bf16", "phtd"),
    ([700, 90], 10, 2, 96, 7, "fp16", "hptd"),
    ([333, 1], 12, 4, 192, 64, "bf16", "phtd"),
    ([260], 4, 4, 16, 128, "bf16", "phtd"),
    ([4000], 64, 8, 128, 64, "bf16", "phtd"),
    ([9000, 1, 0, 2500], 8, 1, 128, 64, "fp16", "pthd"),
    ([50, 700], 48, 2, 128, 16, "bf16", "phtd"),
    ([300], 96, 2, 64, 16, "bf16", "phtd"),
    ([129, 200], 6, 2, 80, 16, "bf16", "phtd"),
    ([40, 5], 6, 3, 100, 16, "bf16", "phtd"),
    ([300, 20], 4, 2, 240, 13, "fp16", "phtd"),
]


@pytest.mark.parametrize("case", ATTENTION_CASES, ids=lambda c: "L%d-B%d-%d/%d-D%d-p%d-%s-%s" % (
    max(c[0]), len(c[0]), *c[1:]))
def test_attention(case):
    lens, Hq, Hk, D, page, dt, order = case
    check_attention(attention_inputs(lens, Hq, Hk, D, page, seed=60, order=order), dt)


@pytest.mark.parametrize("Hq,Hk,D,B,step,most", [(32, 2, 128, 48, 97, 1000), (16, 2, 256, 30, 131, 1500), (10, 2, 96, 60, 61, 2000),
                                                 (32, 2, 256, 30, 89, 700), (32, 2, 64, 64, 53, 1100)])
def test_attention_heads_over_few_blocks(Hq, Hk, D, B, step, most):
    """A few units of the work list per block: heads begin, end and are joined at every place in one."""
    lens = [step * i % most for i in range(B)]
    x = attention_inputs(lens, Hq, Hk, D, 32, seed=78)
    check_attention(x)
    first = fq.paged_attention(*x, want_lse=True)
    again = fq.paged_attention(*x, want_lse=True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_many_sequences():
    lens = [(37 * i) % 300 for i in range(700)]
    check_attention(attention_inputs(lens, 4, 2, 64, 16, seed=61))


def test_attention_very_many_sequences():
    """More sequences than the split kernel takes: most of them empty."""
    lens = [0] * 70000
    lens[0], lens[123], lens[69999] = 20, 5, 33
    x = attention_inputs(lens, 2, 1, 64, 16, seed=76)
    check_attention(x)
    small = [t[:3000].contiguous() for t in (x[0], x[1])] + x[2:6] + [x[6][:3000].contiguous(), x[7][:3000].contiguous()]
    check_attention(small)


def test_attention_maxima_that_grow():
    """Scores that rise along the sequence, by less and by more than the slack of the running maxima."""
    for step in (0.02, 0.3, 3.0):
        x = attention_inputs([900, 130], 8, 2, 128, 16, seed=77)
        x[0].fill_(0x38)  # q = 1 throughout
        x[2].fill_(0x38)
        x[1].fill_(1.0)
        table, lens = x[6].cpu(), x[7].cpu()
        for b, n in enumerate(lens.tolist()):
            pos = torch.arange(n)
            x[4][table[b, pos // 16].long().cuda(), :, (pos % 16).cuda()] = (pos * step / 128 + 1e-3).float().cuda()[:, None]
        check_attention(x, scale=1.0)


@pytest.mark.parametrize("Hq,Hk,D,page", [(8, 2, 128, 16), (32, 2, 128, 16), (4, 4, 64, 24), (32, 2, 256, 32), (6, 2, 192, 7)])
def test_attention_small_weights_beside_large_ones(Hq, Hk, D, page):
    """Every 16th token has 2^26 times the weight of the others, but zeros in the upper half of its values: there the
    output is what the small weights give.

    All scores are exact products (codes of 1), so a weight is off by the exponential alone (2^-20 of it, of a
    difference of scores of 26 held in 2^-19), and by its rounding to fp16, at most 2^-11 of it or 2^-32 of the largest:
    2^-6 of a weight 2^-26 of the largest. The sum of weights: 2^-12 of it. Output: half a step of bf16.
    """
    n = 1024
    x = attention_inputs([n, 37], Hq, Hk, D, page, seed=79)
    q, qs, k, v, ks, vs, table, lens = x
    for t, c in ((q, 0x38), (k, 0x38), (v, 0x38)):
        t.fill_(c)
    qs.fill_(1.0)
    ks.fill_(2.0 ** -40)
    vs.fill_(1.0)
    pos = torch.arange(0, n, 16)
    for b, m in enumerate(lens.tolist()):
        at, off = table.cpu()[b, pos[pos < m] // page].long().cuda(), (pos[pos < m] % page).cuda()
        ks[at, :, off] = 26 * math.log(2.0) / D
        v[at, :, off, D // 2:] = 0
    out = fq.paged_attention(*x, softmax_scale=1.0)[0].cpu().double()
    want = ref.attention(*x, 1.0)[0]
    tol = (2.0 ** -6 + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * want
    assert bool(((out - want).abs() <= tol).all()), float(((out - want).abs() / want).max())


@pytest.mark.parametrize("Hq,Hk,D,page", [(8, 2, 128, 16), (32, 2, 256, 32), (4, 4, 64, 24)])
@pytest.mark.parametrize("scale", [1e-36, 1e-35, 1e-34, 1e-32, 1e34])
def test_attention_value_scales_at_the_ends(scale, Hq, Hk, D, page):
    """V scales near the ends of fp32's range, subnormals among them; bf16 outputs share the range.

    Beside the usual bounds (which grant each weight 2^-11 of itself): logarithms of up to 130 are held in steps of
    2^-16, 2^-17 of a weight; 2^(M - m), from 2^-130 on, in steps of 2^-149, 2^-20 of the output, itself at most 2^11
    of the bound; together less than 2^-4 of it. Below 2^-126 half a step of bf16 is 2^-134."""
    x = attention_inputs([900, 20, 130], Hq, Hk, D, page, seed=82)
    x[5].mul_(scale)
    out, lse = fq.paged_attention(*x, want_lse=True)
    want, want_lse, bound, lse_bound = ref.attention(*x, D ** -0.5)
    tol = 2.0 ** -8 * want.abs() + bound * (1 + 2.0 ** -4) + 2.0 ** -134
    assert bool(((out.cpu().double() - want).abs() <= tol).all())
    assert bool(((lse.cpu().double() - want_lse).abs() <= lse_bound).all())


def test_attention_all_empty():
    check_attention(attention_inputs([0, 0, -5], 8, 2, 128, 16, seed=62))


def test_attention_lengths_are_cut():
    """A length above the bound, and above what the page table holds."""
    x = attention_inputs([300, 280], 8, 2, 128, 16, seed=63)
    check_attention(x, max_len=200)
    check_attention(x, max_len=100)
    check_attention(x, max_len=0)
    x[7] = torch.tensor([10 ** 9, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    check_attention(x)


@pytest.mark.parametrize("offset", [0, 5])
def test_attention_absent_pages(offset):
    """Page ids outside the cache in the middle, at the start, and for a whole sequence."""
    x = attention_inputs([300, 280, 60], 8, 2, 128, 16, seed=64, offset=offset)
    table = x[6]
    table[0, 3], table[0, 7], table[1, 0] = -1, 10 ** 6, x[2].shape[0]
    table[2, :] = -7
    check_attention(x)


def test_attention_strided_and_misaligned():
    check_attention(attention_inputs([200, 31, 4], 8, 2, 128, 16, seed=65, q_extra=4))
    check_attention(attention_inputs([200, 31, 4], 8, 2, 128, 16, seed=66, offset=5))
    x = attention_inputs([200, 200], 8, 2, 128, 16, seed=67)
    x[6] = x[6][:1].expand(2, x[6].shape[1])  # two sequences on one page table row
    check_attention(x)


def test_attention_nan_behind_the_end():
    """NaN codes and scales behind a sequence's end and in pages no sequence uses change nothing."""
    x = attention_inputs([100, 37, 0, 1], 8, 2, 128, 16, seed=68)
    q, qs, k, v, ks, vs, table, lens = x
    clean = fq.paged_attention(*x)[0].clone()
    used = torch.zeros(k.shape[0], k.shape[2], dtype=torch.bool)
    for b, n in enumerate(lens.tolist()):
        pos = torch.arange(n)
        used[table.cpu()[b, pos // 16].long(), pos % 16] = True
    dead = (~used).cuda()[:, None].expand(k.shape[:3])
    k[dead], v[dead], ks[dead], vs[dead] = 0x7F, 0xFF, math.nan, math.nan
    assert torch.equal(fq.paged_attention(*x)[0], clean)


def test_attention_nan_inside_reaches_its_heads():
    x = attention_inputs([400, 50], 8, 2, 128, 16, seed=69)
    page = int(x[6][0, 20])
    x[3][page, 1, 3, 17] = 0x7F  # one V element of key head 1
    out = fq.paged_attention(*x)[0].isnan()
    want = torch.zeros_like(out)
    want[0, 4:, 17] = True
    assert torch.equal(out, want)


def test_attention_large_scores_and_scales():
    """Scores of hundreds (one token takes all the weight) and V scales over twelve decades."""
    x = attention_inputs([500, 20], 8, 2, 128, 16, seed=70)
    x[1].mul_(30.0)
    x[5].copy_(10.0 ** (12 * torch.rand(x[5].shape, generator=gen(3)).cuda() - 9))
    check_attention(x)
    x[5].zero_()
    assert bool((fq.paged_attention(*x)[0] == 0).all())


def test_attention_negative_and_zero_softmax_scale():
    x = attention_inputs([300, 20], 8, 2, 128, 16, seed=71)
    check_attention(x, scale=0.0)
    check_attention(x, scale=-0.05)


@pytest.mark.parametrize("case", [ATTENTION_CASES[2], ATTENTION_CASES[9]], ids=["short", "split"])
def test_attention_repeats_bit_for_bit(case):
    lens, Hq, Hk, D, page, dt, order = case
    x = attention_inputs(lens, Hq, Hk, D, page, seed=72, order=order)
    first = fq.paged_attention(*x, want_lse=True)
    for _ in range(5):
        again = fq.paged_attention(*x, want_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes whose last pages hold the sequence."""
    page, Hk, D = 64, 8, 128
    P = (1 << 32) // (page * Hk * D) + 40
    k, v = (torch.zeros(P, Hk, page, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(P, Hk, page, device="cuda") for _ in range(2))
    g = gen(5)
    n = 1500
    ids = torch.arange(P - 1, P - 25, -1)
    small = make_cache(24, Hk, page, D, 6)
    for big, s in zip((k, v, ks, vs), small):
        big[ids.cuda()] = s
    q, qs = ref.finite_codes((1, 32, D), g).cuda(), (torch.rand(1, 32, generator=g) * 2e-4).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = fq.paged_attention(q, qs, k, v, ks, vs, ids[None].int().cuda(), lens, want_lse=True)
    near = fq.paged_attention(q, qs, *small, torch.arange(24, dtype=torch.int32, device="cuda")[None], lens, want_lse=True)
    assert torch.equal(out, near[0]) and torch.equal(lse, near[1])
    # the append writes there too
    d = wl.qk_inputs(3, 32, 2 * Hk, D, seed=7, token_stride=48 * D)
    d = {a: b.cuda() if isinstance(b, torch.Tensor) else b for a, b in d.items()}
    args = (d["qk"], d["wq"], d["wk"], d["cos"], d["sin"])
    slots = torch.tensor([P * page - 1, P * page - 65, 5], device="cuda")
    fq.qkv_norm_rope_append(*args, slots, k, v, ks, vs, 32, Hk)
    fq.qkv_norm_rope_append(*args, torch.tensor([63, 64, 5], device="cuda"), *small, 32, Hk)
    assert torch.equal(k[P - 1, :, 63], small[0][0, :, 63]) and torch.equal(v[P - 2, :, 63], small[1][1, :, 0])
    assert torch.equal(ks[P - 1, :, 63], small[2][0, :, 63]) and torch.equal(vs[P - 2, :, 63], small[3][1, :, 0])


def test_attention_refusals():
    x = attention_inputs([30, 20], 8, 2, 128, 16, seed=73)
    q, qs, k, v, ks, vs, table, lens = x
    base = dict(q=q, q_scale=qs, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, page_table=table, seq_lens=lens)
    for over in (dict(q=q[:, :3]), dict(q=q.float()), dict(q=q[..., :64]), dict(q_scale=qs[:1]), dict(page_table=table.long()),
                 dict(seq_lens=lens.long()), dict(seq_lens=lens[:1]), dict(v_cache=v.transpose(1, 2)), dict(k_scale=ks.half()),
                 dict(max_seq_len=-1), dict(softmax_scale=math.inf), dict(out_dtype=torch.float32),
                 dict(out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda")), dict(seq_lens=lens.cpu()),
                 dict(k_cache=k[:1].expand(k.shape), v_cache=v[:1].expand(v.shape))):
        with pytest.raises((ValueError, TypeError, fq.FqError)):
            fq.paged_attention(**(base | over))
    wide = attention_inputs([30], 2, 1, 272, 16, seed=74)
    with pytest.raises(fq.FqError):
        fq.paged_attention(*wide)
    long = attention_inputs([3000], 8, 2, 128, 16, seed=75)
    need = fq.paged_attention_workspace_bytes(1, 8, 2, 128, 3000)
    if need:
        with pytest.raises(fq.FqError):
            fq.paged_attention(*long, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"), max_seq_len=3000)


@pytest.mark.parametrize("bound", [2 ** 31, 2 ** 62, 2 ** 63 - 1])
def test_attention_workspace_without_a_bound(bound):
    """A max_seq_len that is no bound at all: the workspace of the longest sequence, and the call takes both."""
    x = attention_inputs([3000, 20], 8, 2, 128, 16, seed=81)
    need = fq.paged_attention_workspace_bytes(2, 8, 2, 128, bound)
    assert need == fq.paged_attention_workspace_bytes(2, 8, 2, 128, 2 ** 31 - 1025) > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, _ = fq.paged_attention(*x, max_seq_len=bound, workspace=ws)
    assert torch.equal(out, fq.paged_attention(*x)[0])


# -------------------------------------------------------------------------------- used together
def decode_step(s):
    """Norm + group-wise FP8 of the hidden rows, the QKV projection, the prologue into the cache, attention."""
    none = s["hidden"].new_empty(s["hidden"].shape[0], 0)
    _, a, sa = fq.rmsnorm_rope_quant_groups(s["hidden"], s["w"], none, none, 128, want_y=False)
    qkv = fq.fp8_matmul(a, sa, s["wqkv"], s["wqkv_scale"])
    q, qs = fq.qkv_norm_rope_append(qkv, s["wq"], s["wk"], s["cos"], s["sin"], s["slots"], *s["cache"], s["Hq"], s["Hk"])
    out, lse = fq.paged_attention(q, qs, *s["cache"], s["table"], s["lens"], want_lse=True, max_seq_len=s["most"])
    return a, sa, qkv, q, qs, out, lse


def step_state(B=5, Hq=8, Hk=2, D=128, hidden=512, page=16, seed=90):
    g = gen(seed)
    n = (Hq + 2 * Hk) * D
    lens = [1, 40, 17, 300, 16][:B]
    x = attention_inputs(lens, Hq, Hk, D, page, seed)
    table = x[6].cpu()
    slots = torch.tensor([int(table[b, (m - 1) // page]) * page + (m - 1) % page for b, m in enumerate(lens)])
    cos, sin = wl.rope_table(torch.tensor(lens).numpy() - 1, D, 1e4, "fp32")
    s = dict(hidden=torch.randn(B, hidden, generator=g).bfloat16(), w=(1 + 0.1 * torch.randn(hidden, generator=g)).bfloat16(),
             wqkv=ref.finite_codes((n, hidden), g), wqkv_scale=torch.rand(n // 128, hidden // 128, generator=g) * 1e-3 + 1e-4,
             wq=(1 + 0.1 * torch.randn(D, generator=g)).bfloat16(), wk=(1 + 0.1 * torch.randn(D, generator=g)).bfloat16(),
             cos=cos, sin=sin, slots=slots)
    s = {k: v.cuda() for k, v in s.items()}
    return s | dict(cache=x[2:6], table=x[6], lens=x[7], Hq=Hq, Hk=Hk, most=max(lens), page=page)


def check_step(s, before, got):
    a, sa, qkv, q, qs, out, lse = got
    ref.assert_matmul(qkv, a, sa, s["wqkv"], s["wqkv_scale"])
    D = q.shape[2]
    case = (q.shape[0], s["Hq"], s["Hk"], D, D, s["page"], "bf16", "fp32", 0, 448.0, "phtd")
    d = dict(qk=qkv, wq=s["wq"], wk=s["wk"], cos=s["cos"], sin=s["sin"])
    check_append(d, before, s["cache"], s["slots"], q.cpu(), qs.cpu(), case)
    ref.assert_attention(out, lse, q, qs, *s["cache"], s["table"], s["lens"], D ** -0.5)


def test_decode_step():
    s = step_state()
    before = [t.clone() for t in s["cache"]]
    check_step(s, before, decode_step(s))


def test_decode_step_captured():
    """The step captured into a graph and replayed on other inputs equals the eager step."""
    s = step_state()
    cache0 = [t.clone() for t in s["cache"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode_step(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decode_step(s)
    other = step_state(seed=91)
    s["hidden"].copy_(other["hidden"])
    for _ in range(2):
        for c, c0 in zip(s["cache"], cache0):
            c.copy_(c0)
        graph.replay()
    torch.cuda.synchronize()
    held = [t.clone() for t in got]
    check_step(s, cache0, held)
    for c, c0 in zip(s["cache"], cache0):
        c.copy_(c0)
    for x, y in zip(held, decode_step(s)):
        assert torch.equal(x, y)


def test_decode_steps_on_two_streams():
    """Two steps on two streams at once, each with its own buffers, give what each gives alone."""
    states = [step_state(seed=90), step_state(seed=95)]
    caches = [[t.clone() for t in s["cache"]] for s in states]
    alone = []
    for s, c0 in zip(states, caches):
        alone.append([t.clone() for t in decode_step(s)])
        for c, z in zip(s["cache"], c0):
            c.copy_(z)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                got.append(decode_step(s))
        torch.cuda.synchronize()
        for x, y in zip(alone, got):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
