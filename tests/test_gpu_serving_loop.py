"""GPU parity of the serving loop's operators against plain implementations (serving_loop_ref.py): block tables and slot
maps, paged attention of a window with sinks, the FP8 product with an epilogue, sampling; and a run of them together."""
import math
import random

import pytest
import torch

import fp8_quant_memory_gb300 as fq
import matmul_cases
import serving_loop_ref as ref
import serving_ref
from guards import Guarded
from test_gpu_serving import DT, attention_inputs, gen, matmul_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_state(cuda_ok):
    yield
    torch.cuda.synchronize()
    assert fq.device_status(clear=True) == 0


def ints(v, t=torch.int32):
    return torch.tensor(v, dtype=t, device="cuda")


# ---------------------------------------------------------------------------------- block tables
def make_step(B, W, page, ring, count, seed, ends=0.1, most=None):
    """A consistent state: sequences with pages of their own, free ones in a ring, and what each sequence adds."""
    r = random.Random(seed)
    lens = [r.choice([0, 1, page, r.randrange(W * page + 1)]) for _ in range(B)]
    new = [-1 if r.random() < ends else r.choice([0, 1, 1, 1, r.randrange(most or 2 * page + 2)]) for _ in range(B)]
    owned = [ref.ceil(n, page) for n in lens]
    ids = list(range(sum(owned) + count))
    r.shuffle(ids)
    table, at = [], 0
    for n in owned:
        table.append(ids[at:at + n] + [-1] * (W - n))
        at += n
    head = r.randrange(ring)
    places = [-1] * ring
    for i, id in enumerate(ids[at:]):
        places[(head + i) % ring] = id
    return table, lens, new, places, [head, count, 77]


def check_extend(table, lens, new, ring, pool, page, T, in_place=False, pad=0):
    want = ref.extend(table, lens, new, ring, pool, page, T)
    B = len(lens)
    W = len(table[0]) if B else 0
    big = torch.full((B, W + pad), -5, dtype=torch.int32, device="cuda")
    if B and W:
        big[:, :W] = ints(table)
    t, ln, nw, rg, pl = big[:, :W], ints(lens), ints(new), Guarded((len(ring),), torch.int32), ints(pool)
    rg.t.copy_(ints(ring))
    out = dict(slots=Guarded((T,), torch.int64, fill=9), positions=Guarded((T,), torch.int32, fill=9), starts=Guarded((B + 1,), torch.int32, fill=9))
    given = {k: g.t for k, g in out.items()}
    if in_place:
        given.update(seq_lens_out=ln, pool_out=pl)
    slots, positions, starts, lens_out, pool_out = fq.paged_extend(t, ln, nw, rg.t, pl, page, T, **given)
    for g in [rg, *out.values()]:
        g.check()
    got = dict(slots=slots, positions=positions, starts=starts, seq_lens=lens_out, pool=pool_out, table=t, ring=rg.t)
    for k, v in got.items():
        assert v.tolist() == want[k], k
    assert bool((big[:, W:] == -5).all())
    if not in_place:
        assert ln.tolist() == lens and pl.tolist() == pool
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,W,page,T", [(1, 1, 1, 1), (1, 4, 16, 40), (3, 5, 7, 33), (17, 9, 16, 300), (64, 20, 64, 900), (100, 3, 1, 120),
                                        (1000, 6, 24, 3000), (1024, 4, 8, 8192), (1025, 4, 8, 20000), (5000, 3, 16, 9000), (12288, 2, 8, 20000), (257, 3, 4, 100), (255, 3, 4, 257)])
def test_extend(B, W, page, T, in_place):
    state = make_step(B, W, page, ring=B * W + 5, count=B * W // 2 + 3, seed=B + T)
    check_extend(*state, page, T, in_place=in_place)


@pytest.mark.parametrize("count", [0, 1, 3, 10, 11, 12, 40])
def test_extend_without_enough_pages(count):
    """The first sequences get theirs, later ones that need none too, nothing else changes."""
    want = check_extend(*make_step(60, 8, 4, ring=400, count=count, seed=count, ends=0.05, most=12), 4, 500)
    assert (want["pool"][2] > 0) == (count < 40)


@pytest.mark.parametrize("T", [0, 1, 10, 57])
def test_extend_without_enough_places(T):
    """Sequences whose tokens pass the step's last are not granted them; starts say so."""
    want = check_extend(*make_step(50, 8, 4, ring=400, count=300, seed=T, most=12), 4, T, pad=3)
    assert want["starts"][-1] > T


def test_extend_table_too_narrow():
    table, lens, new, ring, pool = make_step(40, 4, 8, ring=300, count=200, seed=3, most=40)
    want = check_extend(table, lens, new, ring, pool, 8, 900)
    assert any(m > 0 and o == n for n, m, o in zip(lens, new, want["seq_lens"]))


def test_extend_ring_goes_round():
    """Steps in a row in a ring of exactly as many places as pages; every page is somewhere once all along."""
    r = random.Random(8)
    page, B, W, pages = 4, 12, 10, 60
    table, lens, ring, pool = [[-1] * W for _ in range(B)], [0] * B, list(range(pages)), [0, pages, 0]
    for step in range(40):
        new = [-1 if lens[b] and r.random() < 0.15 else r.choice([0, 1, 1, 5, 9]) for b in range(B)]
        w = check_extend(table, lens, new, ring, pool, page, 200, in_place=step % 2 == 0)
        table, lens, ring, pool = w["table"], w["seq_lens"], w["ring"], w["pool"]
        held = [id for b in range(B) for id in table[b][:ref.ceil(lens[b], page)]]
        free = [ring[(pool[0] + i) % pages] for i in range(pool[1])]
        assert sorted(held + free) == list(range(pages))


def test_extend_empty_and_odd_states():
    check_extend([], [], [], [3, 4], [1, 2, 0], 16, 5)
    check_extend([], [], [], [3], [0, 0, 0], 16, 0)
    check_extend([[], []], [0, 0], [0, 1], [3], [0, 1, 0], 16, 4)  # a table without columns
    check_extend([[1, 2], [-1, -1]], [-9, 0], [3, -2 ** 31], [5, 6, 7], [-1, 9, 0], 2, 4)  # a negative length, front and count out of range
    check_extend([[-1, -1], [4, -1]], [2, 3], [1, 1], [5, 6, 7], [2, 3, 0], 2, 4)  # an absent page in the row
    check_extend([[0, 1]], [4], [-1], [5, 6, 7], [1, 2, 0], 2, 4)  # two pages return, the ring has one place
    big = 2 ** 31 - 1
    check_extend([[0, 1], [2, 3]], [big, big], [big, big], [5, 6], [0, 2, 0], 3, 4)  # lengths and sums at the end of 32 bits
    check_extend([[0, 1], [2, 3]], [big, 2], [-1, 1], [5, 6, 7, 8], [3, 1, 0], 3, 4)


def test_extend_captured_step_advances():
    table, lens, new, ring, pool = make_step(30, 12, 4, ring=400, count=200, seed=4, ends=0.0, most=3)
    lens = [min(n, 8) for n in lens]
    t, ln, nw, rg, pl = ints(table), ints(lens), ints(new), ints(ring), ints(pool)
    side = torch.cuda.Stream()
    keep = [x.clone() for x in (t, ln, rg, pl)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.paged_extend(t, ln, nw, rg, pl, 4, 64, seq_lens_out=ln, pool_out=pl)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((t, ln, rg, pl), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fq.paged_extend(t, ln, nw, rg, pl, 4, 64, seq_lens_out=ln, pool_out=pl)
    for step in range(4):
        if step == 2:
            new = [-1 if b % 3 == 0 else 2 for b in range(30)]
            nw.copy_(ints(new))
        graph.replay()
        w = ref.extend(table, lens, new, ring, pool, 4, 64)
        assert out[0].tolist() == w["slots"] and ln.tolist() == w["seq_lens"] and t.tolist() == w["table"] and rg.tolist() == w["ring"]
        table, lens, ring, pool = w["table"], w["seq_lens"], w["ring"], w["pool"]
        assert pl.tolist() == pool


# -------------------------------------------------------------------------------------- attention
def check_window(x, window, sinks, scale=None, max_len=None, dt="bf16"):
    B, Hq, D = x[0].shape
    out, lse = Guarded((B, Hq, D), DT[dt], fill=math.nan), Guarded((B, Hq), torch.float32, fill=math.nan)
    fq.paged_attention(*x, softmax_scale=scale, max_seq_len=max_len, window=window, sinks=sinks, out=out.t, lse=lse.t)
    out.check()
    lse.check()
    seen = ref.windowed(*x, window, sinks, max_len)
    serving_ref.assert_attention(out.t, lse.t, *seen, D ** -0.5 if scale is None else scale)


WINDOWS = [(1, 0), (1, 1), (2, 5), (15, 0), (16, 16), (17, 3), (100, 0), (100, 64), (128, 128), (129, 1), (300, 7), (1000, 200), (10 ** 9, 3)]
LENS = [0, 1, 2, 15, 16, 17, 33, 100, 128, 129, 255, 256, 300, 511, 777, 1300, 2111]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hk,D,page,dt", [(8, 2, 128, 16, "bf16"), (4, 4, 64, 24, "fp16"), (32, 2, 256, 32, "bf16"), (6, 1, 192, 8, "fp16"),
                                             (5, 1, 96, 7, "bf16"), (4, 2, 100, 16, "bf16"), (16, 2, 64, 128, "bf16")])
def test_window(window, sinks, Hq, Hk, D, page, dt):
    check_window(attention_inputs(LENS, Hq, Hk, D, page, seed=window % 1000 + sinks), window, sinks, dt=dt)


@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (2000, 0), (4096, 64), (4097, 129)])
def test_window_of_a_long_sequence(window, sinks):
    check_window(attention_inputs([20011], 16, 2, 128, 16, seed=sinks), window, sinks)
    check_window(attention_inputs([20011, 5], 4, 2, 64, 12, seed=sinks), window, sinks)


def test_window_that_sees_everything_is_the_whole_attention():
    x = attention_inputs([1000, 20, 0, 333], 8, 2, 128, 16, seed=3)
    whole = fq.paged_attention(*x, want_lse=True)
    most = x[6].shape[1] * 16
    for window, sinks in ((most, 0), (most + 5, 9), (2 ** 62, 2 ** 62)):
        got = fq.paged_attention(*x, want_lse=True, window=window, sinks=sinks)
        assert torch.equal(whole[0], got[0]) and torch.equal(whole[1], got[1])


@pytest.mark.parametrize("window,sinks", [(10, 2), (40, 0), (5, 33), (200, 17)])
def test_window_lengths_are_cut(window, sinks):
    x = attention_inputs([300, 280, 31], 8, 2, 128, 16, seed=63)
    check_window(x, window, sinks, max_len=200)
    check_window(x, window, sinks, max_len=0)
    x[7] = torch.tensor([10 ** 9, 2 ** 31 - 1, -4], dtype=torch.int32, device="cuda")
    check_window(x, window, sinks)


@pytest.mark.parametrize("page,D", [(16, 128), (24, 64), (5, 100)])
@pytest.mark.parametrize("offset", [0, 5])
def test_window_absent_and_unread_pages(offset, page, D):
    """Absent pages inside the window and among the sinks, a row whose window has none left; pages in between may be
    anything: their ids are out of range or name a page of NaN."""
    x = attention_inputs([600, 580, 60, 900], 8, 2, D, page, seed=64, offset=offset)
    table, window, sinks = x[6], 200, 2 * page + 1
    table[0, 1], table[0, (600 - 90) // page], table[1, 0] = -1, 10 ** 6, x[2].shape[0]
    table[2, :] = -7
    nan = int(table[3, 11])
    x[2][nan], x[3][nan], x[4][nan], x[5][nan] = 0x7F, 0x7F, math.nan, math.nan
    for b, n in ((0, 600), (1, 580), (3, 900)):
        table[b, sinks // page + 1:(n - window) // page] = nan if b == 3 else 2 ** 31 - 1
    check_window(x, window, sinks)
    table[0, (600 - 7) // page:] = -1
    check_window(x, 7, 0)


def test_window_masks_inside_boxes():
    """NaN rows right before the window's first token and behind the last sink change nothing."""
    x = attention_inputs([700], 8, 2, 128, 16, seed=9)
    clean = fq.paged_attention(*x, window=333, sinks=21, want_lse=True)
    for j in (21, 22, 31, 365, 366, 352):
        page = int(x[6][0, j // 16])
        x[2][page, :, j % 16], x[3][page, :, j % 16] = 0x7F, 0x7F
        x[4][page, :, j % 16], x[5][page, :, j % 16] = math.nan, math.inf
    got = fq.paged_attention(*x, window=333, sinks=21, want_lse=True)
    assert torch.equal(clean[0], got[0]) and torch.equal(clean[1], got[1])


def test_window_repeats_bit_for_bit_and_replays():
    x = attention_inputs([5000, 20, 1300, 0, 2222], 32, 8, 128, 64, seed=10)
    first = fq.paged_attention(*x, window=1000, sinks=4, want_lse=True)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = fq.paged_attention(*x, window=1000, sinks=4, want_lse=True)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    with torch.cuda.graph(graph):
        out, lse = fq.paged_attention(*x, window=1000, sinks=4, want_lse=True)
    graph.replay()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    x[7].copy_(torch.tensor([17, 5100, 900, 1001, 1004], dtype=torch.int32))
    x[6].clamp_(min=0)
    graph.replay()
    want = fq.paged_attention(*x, window=1000, sinks=4, want_lse=True)
    assert torch.equal(want[0], out) and torch.equal(want[1], lse)


# ----------------------------------------------------------------------------------------- linear
def linear_inputs(M, N, K, seed, dt, which):
    a, sa, b, sb = matmul_inputs(M, N, K, seed=seed)
    sa.mul_(2.0 ** -5 * K ** -0.5 / float(sa.mean() * sb.mean() * 2 ** 6))  # outputs of a few units
    g = gen(seed + 1)
    bias = torch.randn(N, generator=g).to(DT[dt]).cuda() if "b" in which else None
    res = (2 * torch.randn(M, N, generator=g)).to(DT[dt]).cuda() if "r" in which else None
    return (a, sa, b, sb), bias, res


LINEAR = [
    (1, 1, 1, "bf16", "br", "silu"), (1, 129, 16, "fp16", "b", "gelu"), (3, 257, 130, "bf16", "br", "gelu_tanh"), (1, 4096, 8192, "bf16", "br", "silu"),
    (8, 128, 256, "fp16", "r", None), (16, 384, 4096, "bf16", "b", "relu"), (31, 100, 144, "fp16", "br", "gelu"), (33, 127, 384, "bf16", "br", "silu"),
    (64, 1024, 512, "bf16", "br", "gelu"), (64, 4100, 6928, "bf16", "br", "gelu_tanh"), (65, 300, 640, "fp16", "", "silu"), (128, 128, 128, "bf16", "br", None),
    (129, 129, 129, "fp16", "br", "gelu_tanh"), (333, 1111, 1968, "fp16", "br", "gelu"), (300, 2049, 128, "bf16", "br", "relu"), (512, 1000, 16, "bf16", "b", "gelu"),
    (1025, 513, 784, "fp16", "br", "silu"), (1536, 1280, 256, "bf16", "r", "gelu_tanh"), (2500, 2296, 1040, "bf16", "br", "silu"),
    (2500, 2303, 528, "fp16", "br", "gelu"), (300, 4096, 96, "bf16", "br", "relu"), (2048, 1, 64, "bf16", "br", "silu"),
]


@pytest.mark.parametrize("M,N,K,dt,which,act", LINEAR)
def test_linear(M, N, K, dt, which, act):
    x, bias, res = linear_inputs(M, N, K, M + N, dt, which)
    out = Guarded((M, N), DT[dt], fill=math.nan)
    got = fq.fp8_matmul(*x, out=out.t, bias=bias, activation=act, residual=res)
    out.check()
    ref.assert_epilogue(got, *x, bias, act, res)


@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (40, 520, 512), (64, 1000, 4096), (200, 300, 256), (2400, 2304, 256), (2400, 2305, 128)])
def test_linear_in_place_strided_and_broadcast(M, N, K):
    """The residual is the output; rows of both further apart; one residual row for all; misaligned pointers."""
    x, bias, res = linear_inputs(M, N, K, 7, "bf16", "br")
    buf = torch.full((M, N + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    buf[:, :N] = res
    got = fq.fp8_matmul(*x, out=buf[:, :N], bias=bias, activation="silu", residual=buf[:, :N])
    ref.assert_epilogue(got, *x, bias, "silu", res)
    assert bool((buf[:, N:] == 7.0).all())
    same = fq.fp8_matmul(*x, bias=bias, activation="silu", residual=res)
    assert torch.equal(same, got)
    one = fq.fp8_matmul(*x, bias=bias, residual=res[:1].expand(M, N))
    ref.assert_epilogue(one, *x, bias, None, res[:1].expand(M, N))
    odd = torch.zeros(N + 1, dtype=torch.bfloat16, device="cuda")
    odd[1:] = bias
    shifted = torch.zeros(M * N + 1, dtype=torch.bfloat16, device="cuda")
    shifted[1:] = res.flatten()
    assert torch.equal(fq.fp8_matmul(*x, bias=odd[1:], activation="silu", residual=shifted[1:].view(M, N)), got)


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("want, size", [*matmul_cases.NARROW.items(), *matmul_cases.WIDE.items(), *matmul_cases.WIDE_MORE], ids=str)
def test_linear_every_kernel(want, size, aligned):
    """Each kernel and variant of the product; bias, residual and output in whole 16-byte pieces or not."""
    M, N, K = size
    dt, act = ("bf16", "silu") if aligned else ("fp16", "gelu")
    N = N // 8 * 8 if aligned and want[0] == 256 else N
    if torch.cuda.get_device_properties(0).multi_processor_count == matmul_cases.SMS:
        assert matmul_cases.plan(M, N, K) == want
    x, bias, res = linear_inputs(M, N, K, 21, dt, "br")
    stride = (N + 15) // 8 * 8 if aligned else N + 3
    buf = torch.full((2, M, stride), 7.0, dtype=DT[dt], device="cuda")
    buf[1, :, :N] = res
    out, res = buf[0, :, :N], buf[1, :, :N]
    fq.fp8_matmul(*x, out=out, bias=bias, activation=act, residual=res)
    ref.assert_epilogue(out, *x, bias, act, res)
    assert bool((buf[:, :, N:] == 7.0).all())
    assert torch.equal(fq.fp8_matmul(*x, out=res, bias=bias, activation=act, residual=res), out)
    assert bool((buf[:, :, N:] == 7.0).all())


@pytest.mark.parametrize("M", [5, 64, 150, 2400])
def test_linear_without_an_epilogue_is_the_product(M):
    x, _, _ = linear_inputs(M, 2304, 512, 5, "bf16", "")
    plain = fq.fp8_matmul(*x)
    zero = torch.zeros(2304, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fq.fp8_matmul(*x, bias=zero), plain)
    relu = fq.fp8_matmul(*x, activation="relu")
    assert torch.equal(relu, plain.clamp(min=0))


@pytest.mark.parametrize("M", [1, 100, 600])
@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_ends_of_the_range(M, act):
    """Infinite and NaN biases, sums far out on both sides."""
    x, _, _ = linear_inputs(M, 264, 256, 6, "bf16", "")
    bias = torch.zeros(264, dtype=torch.bfloat16, device="cuda")
    bias[:8] = torch.tensor([1e4, -1e4, 1e30, -1e30, -90.0, 3e38, -3e38, -60.0])
    out = fq.fp8_matmul(*x, bias=bias, activation=act)
    ref.assert_epilogue(out, *x, bias, act, None)
    bias[8:10] = torch.tensor([math.inf, math.nan])
    out = fq.fp8_matmul(*x, bias=bias, activation=act)
    assert bool((out[:, 8] == math.inf).all()) and bool(out[:, 9].isnan().all())
    assert not bool(out[:, :8].isnan().any()) and not bool(out[:, 10:].isnan().any())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", [(1, 264, 256), (100, 264, 256), (600, 264, 256), (20, 264, 250)])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_linear_far_below_zero(M, N, K, act, dt):
    """What a smooth activation leaves far below zero: up to 1e-17 off, and the output's rounding, whatever the value is,
    beside NaN and infinite neighbours, which share an instruction. Products are zero: the bias is what is activated."""
    x, _, _ = linear_inputs(M, N, K, 6, "bf16", "")
    x[0].zero_()
    far = [-1e30, -3e38, -1e20, -65504.0, -1e4, -300.0, -90.0, -50.0, -44.0, -43.5, -43.0, -42.5, -42.0, -30.0, -20.0, -14.0, -10.0, -9.0, -8.5, -8.0, -7.5, -7.0]
    far = torch.tensor(far, dtype=torch.float64).clamp(min=float(torch.finfo(DT[dt]).min)).repeat(3)
    odd = torch.tensor([math.nan, math.inf, -math.inf], dtype=torch.float64).repeat_interleave(22)
    bias = torch.zeros(N, dtype=torch.float64)
    bias[0:132:2], bias[1:132:2] = far, odd
    bias[132:264:2], bias[133:264:2] = odd, far
    bias = bias.to(DT[dt])
    out = fq.fp8_matmul(*x, out_dtype=DT[dt], bias=bias.cuda(), activation=act).cpu().double()
    y = bias.double()
    want = ref.ACTIVATIONS[act](y).expand(M, N)
    finite = y.isfinite().expand(M, N)
    # 2^-15: exponents of up to 2^6 (gelu: x^2 log2(e) of x = y / sqrt(2), rounded three times), 2^-24 of that each, times
    # ln 2, and 2^-20 of the approximations; what is smaller than e^-43 is below 1e-17 itself
    half = torch.finfo(DT[dt]).eps / 2
    tol = (half + 2.0 ** -15) * want.abs() + 1e-17 + (2.0 ** -25 if dt == "fp16" else 0.0)
    assert bool(((out - want).abs() <= tol)[finite].all())
    assert bool(out[:, y.isnan()].isnan().all()) and bool((out[:, y == math.inf] == math.inf).all())
    left = out[:, y == -math.inf]
    assert bool(left.isnan().all()) if act == "gelu" else bool((left.abs() <= 1e-17).all())


# ---------------------------------------------------------------------------------------- sampling
def check_sample(x, u, heat=None, k=None, top_p=None, min_p=None, exact=True):
    """x: [B, V] on the GPU; lists of settings. Rows whose borders are met to 2^-38 may take a neighbour."""
    B = x.shape[0]
    given = {n: None if v is None else torch.tensor(v, dtype=t, device="cuda")
             for n, v, t in (("temperature", heat, torch.float32), ("top_k", k, torch.int32), ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32))}
    us = torch.tensor(u, dtype=torch.float32, device="cuda")
    token, logprob = Guarded((B,), torch.int64, fill=-9), Guarded((B,), torch.float32, fill=math.nan)
    fq.sample(x, us, **given, token=token.t, logprob=logprob.t)
    token.check()
    logprob.check()
    rows = {n: [d] * B if g is None else g.double().tolist() for (n, g), d in zip(given.items(), (1.0, 0, 1.0, 0.0))}
    close = 0
    for b in range(B):
        t, lp, margin = ref.sample(x[b].cpu().double(), us[b].double().item(), rows["temperature"][b], int(rows["top_k"][b]), rows["top_p"][b],
                                   rows["min_p"][b])
        if margin < 2.0 ** -38:
            close += 1
            continue
        assert int(token.t[b]) == t, (b, int(token.t[b]), t, margin)
        got = float(logprob.t[b])
        assert got == lp or abs(got - lp) <= 2.0 ** -20 * abs(lp) + 2.0 ** -22, (b, got, lp)
    assert close <= (B // 20 if exact else B)
    bare, none = fq.sample(x, us, **given)
    assert none is None and torch.equal(bare, token.t)


def logits(B, V, dt, seed, spread=3.0):
    return (spread * torch.randn(B, V, generator=gen(seed))).to(DT[dt]).cuda()


def settings(B, seed):
    r = random.Random(seed)
    return dict(u=[r.random() for _ in range(B)], heat=[r.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5, 4.0]) for _ in range(B)],
                k=[r.choice([0, -1, 1, 2, 5, 50, 1000, 10 ** 6]) for _ in range(B)], top_p=[r.choice([0.0, 0.1, 0.5, 0.9, 0.99, 1.0, 2.0]) for _ in range(B)],
                min_p=[r.choice([0.0, 0.0, 0.01, 0.2, 1.0, 3.0]) for _ in range(B)])


VOCABULARIES = [1, 2, 7, 8, 9, 15, 17, 31, 64, 100, 255, 1000, 4099, 8192, 32000, 50001, 65535, 65537, 151936, 200003]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("V", VOCABULARIES)
def test_sample(V, dt):
    B = 40 if V < 10000 else 24
    check_sample(logits(B, V, dt, V), **settings(B, V))


@pytest.mark.parametrize("kind", ["heat", "k", "top_p", "min_p", "none"])
@pytest.mark.parametrize("B", [1, 2, 5, 30, 160, 400])
def test_sample_each_setting_alone(B, kind):
    s = settings(B, B)
    check_sample(logits(B, 3001, "bf16", B), s["u"], **({} if kind == "none" else {kind: s[kind]}))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_sample_ties(dt):
    """Rows of few distinct values, of one, of both zeros: the lowest index comes first."""
    B = 60
    x = logits(B, 5003, dt, 5, spread=1.0).round()
    x[40:50] = 2.5
    x[50:] = torch.where(torch.rand(10, 5003, generator=gen(1)) < 0.5, -0.0, 0.0).cuda()
    check_sample(x, **settings(B, 5))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_sample_masks_infinities_and_nan(dt):
    B, V = 48, 2003
    x = logits(B, V, dt, 6)
    low = torch.finfo(DT[dt]).min
    g = gen(7)
    hide = (torch.rand(B, V, generator=g) < 0.98).cuda()
    x[:8] = x[:8].masked_fill(hide[:8], -math.inf)
    x[8:16] = x[8:16].masked_fill(hide[8:16], low)
    x[16:24] = x[16:24].masked_fill(hide[16:24], math.nan)
    x[24] = -math.inf
    x[25] = math.nan
    x[26, ::2], x[26, 1::2] = -math.inf, -math.nan
    x[27] = low
    x[28] = -math.inf
    x[28, V - 1] = low
    x[29, 3], x[29, 700] = math.inf, math.inf
    x[30] = math.inf
    x[31, 0], x[31, 1:] = 1.0, -math.inf
    x[32:] *= 100.0
    check_sample(x, **settings(B, 7))


@pytest.mark.parametrize("dt,heat", [("bf16", 1e38), ("bf16", 3e38), ("bf16", math.inf), ("bf16", 1e-30), ("bf16", 1.2e-38), ("bf16", 1e20), ("fp16", 2000.0), ("fp16", 3e4),
                                     ("fp16", 1e-6), ("fp16", math.inf)])
def test_sample_all_magnitudes(dt, heat):
    """Values of every exponent and both signs, at temperatures that keep them all (two rounds of bins), or few."""
    V = 60000
    raw = torch.randint(0, 65536, (12, V), generator=gen(9), dtype=torch.int64)
    top = 0x7F80 if dt == "bf16" else 0x7C00
    raw = torch.where((raw & 0x7FFF) >= top, raw & 0x8000, raw)
    x = (raw - 65536 * (raw >= 32768).long()).to(torch.int16).view(DT[dt]).cuda()
    s = settings(12, 3)
    s["heat"] = [heat] * 12
    check_sample(x, **s)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("least", [0x8001, 0x8002, 0x801F, 0x8020, 0x8021])
def test_sample_largest_next_to_zero(least, dt):
    """The largest is a few steps below zero (there is no zero to count with it), or is zero, of either sign."""
    raw = torch.randint(least, least + 400, (20, 5003), generator=gen(least), dtype=torch.int64)
    raw[:, 17], raw[10:15, ::7], raw[15:, ::5] = least, 0x8000, 0
    x = (raw - 65536 * (raw >= 32768).long()).to(torch.int16).view(DT[dt]).cuda()
    s = settings(20, least)
    s["k"] = [0, 2000, 3000, -1] * 5
    s["heat"] = [1.0, 1e-5, 1e-6, 3e-39 if dt == "fp16" else 3e-38] * 5
    check_sample(x, **s)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("V", [8193, 9001, 30000])
def test_sample_largest_behind_the_first_thousands(V, dt):
    """The first 8192 of a row, from whose largest the bins are laid out, are far below the rest, or nothing at all."""
    B, n = 28, 8192
    x = logits(B, V, dt, V)
    top = float(torch.finfo(DT[dt]).max)
    for b in range(B):
        head, tail = x[b, :n], x[b, n:]
        kind = b % 14
        if kind == 0: head.fill_(-math.inf)
        if kind == 1: head.fill_(math.nan)
        if kind == 2: head[::2], head[1::2] = -math.inf, math.nan
        if kind == 3: head.fill_(torch.finfo(DT[dt]).min)
        if kind == 4: head.sub_(1000.0), tail.mul_(50.0)
        if kind == 5: head.mul_(2.0 ** -20).abs_().neg_(), tail.abs_()
        if kind == 6: head.mul_(2.0 ** -20), tail.mul_(100.0)
        if kind == 7: head.zero_(), tail.fill_(-0.0)
        if kind == 8: head.fill_(-0.0), tail.abs_().neg_()
        if kind == 9: tail[-1] = math.inf
        if kind == 10: tail[-1] = top
        if kind == 11: tail.fill_(math.nan)
        if kind == 12: head.fill_(-1e-30), tail.fill_(1e-30)
        if kind == 13: tail[:] = -math.inf
    s = settings(B, V)
    s["heat"] = [r or 2.0 for r in s["heat"]]
    s["k"], s["top_p"] = [0, 3000] * 14, [1.0, 0.9, 0.99, 0.5] * 7
    check_sample(x, **s)
    s["heat"] = [30000.0 if dt == "fp16" else 1e30] * B
    check_sample(x, **s)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("B", [1, 2, 18, 20, 39, 77])
@pytest.mark.parametrize("V", [8191, 8193, 16385, 33000, 70001])
def test_sample_rows_cut_among_blocks(B, V, dt):
    """One to 77 rows of lengths that one, two, four or eight blocks share, ties across their parts."""
    x = logits(B, V, dt, V + B)
    x[:, ::3] = x[:, ::3].round()
    s = settings(B, V)
    s["k"] = [r if r != 1000 else 3000 for r in s["k"]]
    check_sample(x, **s)


@pytest.mark.parametrize("V", [9000, 20000, 40000])
def test_sample_blocks_without_tokens(V):
    """Parts of a row that hold nothing, the largest alone, or NaN; the largest in several parts."""
    B = 19
    x = torch.full((B, V), -math.inf, dtype=torch.bfloat16, device="cuda")
    y = logits(B, V, "bf16", V)
    for b in range(B):
        lo, hi = b * V // B, min(V, (b * V) // B + 300)
        x[b, lo:hi] = y[b, lo:hi]
    x[3], x[4], x[5, ::2] = -math.inf, math.nan, math.nan
    x[6], x[6, [5, V // 2, V - 1]] = -math.inf, 3.0
    x[7, [V - 1, V // 3]], x[8, 1] = math.inf, math.inf
    x[9] = 0.0
    check_sample(x, **settings(B, 1))
    check_sample(x, u=[0.99 - b / 40 for b in range(B)], heat=[1.0] * B, top_p=[0.95] * B)


@pytest.mark.parametrize("heat", [1e38, 3e38])
def test_sample_two_rounds_cut_among_blocks(heat):
    raw = torch.randint(0, 65536, (3, 40000), generator=gen(19), dtype=torch.int64)
    raw = torch.where((raw & 0x7FFF) >= 0x7F80, raw & 0x8000, raw)
    x = (raw - 65536 * (raw >= 32768).long()).to(torch.int16).view(torch.bfloat16).cuda()
    check_sample(x, u=[0.1, 0.6, 0.999], heat=[heat] * 3, k=[0, 20000, 5000], top_p=[0.99, 1.0, 0.7], min_p=[0.0, 0.01, 0.0])


def test_sample_border_numbers():
    """u at 0, just below 1, outside and NaN; settings that are NaN switch their step off."""
    x = logits(9, 777, "bf16", 11)
    nan = math.nan
    check_sample(x[:6], [0.0, 1 - 2.0 ** -24, 1.0, 7.0, -3.0, nan])
    s = dict(u=[0.3, 0.6, 0.9])
    u = torch.tensor(s["u"], device="cuda")
    three = lambda v: torch.tensor([v] * 3, device="cuda")
    plain = fq.sample(x[:3], u)[0]
    assert torch.equal(fq.sample(x[:3], u, top_p=three(nan), min_p=three(nan))[0], plain)
    assert torch.equal(fq.sample(x[:3], u, temperature=three(nan))[0], x[:3].float().argmax(1))
    assert torch.equal(fq.sample(x[:3], u, temperature=three(-1.0))[0], x[:3].float().argmax(1))


def test_sample_strided_and_misaligned_rows():
    big = logits(10, 5000, "bf16", 12)
    for view in (big[:, 1:4001], big[:, 3:4], big[::2, 7:3006], big[:1].expand(6, 5000), big[:, :4000]):
        u = torch.rand(view.shape[0], generator=gen(2)).cuda()
        k = torch.full((view.shape[0],), 40, dtype=torch.int32, device="cuda")
        assert torch.equal(fq.sample(view, u, top_k=k)[0], fq.sample(view.contiguous(), u, top_k=k)[0])
        assert torch.equal(fq.sample(view, u)[0], fq.sample(view.contiguous(), u)[0])


def test_sample_rows_beyond_32_bits():
    x = torch.full((40000, 1 << 17), -4.0, dtype=torch.bfloat16, device="cuda")  # 10.5 GB
    x[39999, 100001] = 20.0
    token = fq.sample(x[39990:], torch.full((10,), 0.5, device="cuda"))[0]
    assert int(token[9]) == 100001
    token = fq.sample(x, torch.full((40000,), 0.5, device="cuda"), temperature=torch.zeros(40000, device="cuda"))[0]
    assert int(token[39999]) == 100001 and int(token[39998]) == 0


def test_sample_many_equal_values_count_beyond_16_bits():
    x = torch.full((3, 300000), 1.0, dtype=torch.bfloat16, device="cuda")
    x[1, 200000:] = 1.0078125
    x[2, ::2] = 1.0078125
    check_sample(x, [0.999, 0.7, 0.75], top_p=[0.9, 1.0, 0.8])


def test_sample_empty_and_replayed():
    assert fq.sample(torch.zeros(0, 7, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, device="cuda"))[0].shape == (0,)
    x, u = logits(9, 3000, "bf16", 13), torch.rand(9, generator=gen(3)).cuda()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fq.sample(x, u, want_logprob=True)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = fq.sample(x, u, want_logprob=True)
    for seed in (14, 15):
        x.copy_(logits(9, 3000, "bf16", seed))
        u.copy_(torch.rand(9, generator=gen(seed)))
        graph.replay()
        want = fq.sample(x, u, want_logprob=True)
        assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])


# ------------------------------------------------------------------------------------- a serving loop
class Loop:
    """One block of a model with random weights, its cache, and the requests' state."""

    def __init__(self, B=5, Hq=8, Hk=2, D=128, hidden=512, V=1003, page=16, seed=90):
        g = gen(seed)
        self.B, self.Hq, self.Hk, self.D, self.hidden, self.V, self.page, self.width, self.window, self.sinks = B, Hq, Hk, D, hidden, V, page, 6, 20, 3
        pages = 40

        def weight(n, k):
            codes = serving_ref.finite_codes((n, k), g)
            return codes.cuda(), (torch.rand(-(-n // 128), k // 128, generator=g) * 2e-4 + 1e-4).cuda()
        self.w_qkv, self.w_out, self.w_logits = weight((Hq + 2 * Hk) * D, hidden), weight(hidden, Hq * D), weight(V, hidden)
        self.b_qkv = (0.1 * torch.randn((Hq + 2 * Hk) * D, generator=g)).bfloat16().cuda()
        self.w_in, self.w_mid, self.w_last = ((1 + 0.1 * torch.randn(n, generator=g)).bfloat16().cuda() for n in (hidden, Hq * D, hidden))
        self.wq, self.wk = ((1 + 0.1 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2))
        self.embedding = torch.randn(V, hidden, generator=g).bfloat16().cuda()
        angle = torch.arange(self.width * page)[:, None] * 1e4 ** (-torch.arange(D // 2) * 2.0 / D)
        self.cos, self.sin = angle.cos().cuda(), angle.sin().cuda()
        self.none = torch.zeros(0, device="cuda")
        self.cache = [torch.zeros(pages, Hk, page, D, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
            [torch.ones(pages, Hk, page, device="cuda") for _ in range(2)]
        self.table = torch.full((B, self.width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.new = torch.ones(B, dtype=torch.int32, device="cuda")
        self.ring = torch.randperm(pages, generator=g).int().cuda()
        self.pool = ints([3, pages, 0])
        self.u = torch.rand(B, generator=g).cuda()
        self.heat, self.k = torch.full((B,), 0.7, device="cuda"), ints([50] * B)
        self.top_p = torch.full((B,), 0.9, device="cuda")

    def quantise(self, x, w):
        tables = torch.empty(x.shape[0], 0, dtype=torch.bfloat16, device="cuda")
        return fq.rmsnorm_rope_quant_groups(x, w, tables, tables, 128, want_y=False)[1:]

    def step(self, ids, max_tokens, seen=None):
        """ids: [max_tokens] token ids, the sequences' new ones in order; returns the next token of each sequence."""
        B, Hq, D = self.B, self.Hq, self.D
        before = [t.clone() for t in (self.table, self.lens, self.ring, self.pool)]
        slots, pos, starts, _, _ = fq.paged_extend(self.table, self.lens, self.new, self.ring, self.pool, self.page, max_tokens,
                                                   seq_lens_out=self.lens, pool_out=self.pool)
        x = self.embedding[ids]
        a = self.quantise(x, self.w_in)
        qkv = fq.fp8_matmul(*a, *self.w_qkv, bias=self.b_qkv)
        q, qs = fq.qkv_norm_rope_append(qkv, self.wq, self.wk, self.cos[pos], self.sin[pos], slots, *self.cache, Hq, self.Hk)
        last = (starts[1:] - 1).long()
        args = (q[last], qs[last], *self.cache, self.table, self.lens)
        out, lse = fq.paged_attention(*args, window=self.window, sinks=self.sinks, want_lse=True)
        m = self.quantise(out.view(B, Hq * D), self.w_mid)
        stream = x[last]
        y = fq.fp8_matmul(*m, *self.w_out, activation="silu", residual=stream)
        n = self.quantise(y, self.w_last)
        logits = fq.fp8_matmul(*n, *self.w_logits)
        token, logprob = fq.sample(logits, self.u, temperature=self.heat, top_k=self.k, top_p=self.top_p, want_logprob=True)
        if seen is not None:
            seen.update(before=before, slots=slots, pos=pos, starts=starts, qkv=(qkv, a), attention=(args, out, lse), y=(y, m, stream), logits=logits,
                        token=token, logprob=logprob)
        return token

    def check(self, s, max_tokens):
        table, lens, ring, pool = (t.tolist() for t in s["before"])
        w = ref.extend(table, lens, self.new.tolist(), ring, pool, self.page, max_tokens)
        assert s["slots"].tolist() == w["slots"] and s["pos"].tolist() == w["positions"] and s["starts"].tolist() == w["starts"]
        assert self.lens.tolist() == w["seq_lens"] and self.table.tolist() == w["table"] and self.ring.tolist() == w["ring"] and self.pool.tolist() == w["pool"]
        qkv, a = s["qkv"]
        ref.assert_epilogue(qkv, *a, *self.w_qkv, self.b_qkv, None, None)
        args, out, lse = s["attention"]
        serving_ref.assert_attention(out, lse, *ref.windowed(*args, self.window, self.sinks), self.D ** -0.5)
        y, m, stream = s["y"]
        ref.assert_epilogue(y, *m, *self.w_out, None, "silu", stream)
        for b in range(self.B):
            t, lp, margin = ref.sample(s["logits"][b].cpu().double(), self.u[b].double().item(), self.heat[b].double().item(), int(self.k[b]), self.top_p[b].double().item())
            assert margin < 2.0 ** -38 or int(s["token"][b]) == t
            assert margin < 2.0 ** -38 or abs(float(s["logprob"][b]) - lp) <= 2.0 ** -20 * abs(lp) + 2.0 ** -22


def started(seed=90):
    """A loop whose five prompts of 59 tokens in all are in the cache, and the tokens that follow them."""
    s = Loop(seed=seed)
    s.new.copy_(ints([7, 1, 18, 30, 3]))
    ids = torch.randint(0, s.V, (64,), generator=gen(seed + 1)).cuda()
    seen = {}
    token = s.step(ids, 64, seen)
    s.check(seen, 64)
    s.new.fill_(1)
    return s, token


def test_serving_loop():
    """Prompts, then steps of one token each: every operator against 64 bits on its own inputs, the requests' state too; a
    sequence ends and another takes its place."""
    s, token = started()
    for step in range(8):
        if step == 4:
            s.new.copy_(ints([1, -1, 1, 1, 1]))
            ids = torch.cat([token[[0, 2, 3, 4]], token[:1]])
        else:
            s.new.fill_(1)
            ids = token
        s.u.copy_(torch.rand(5, generator=gen(step)))
        seen = {}
        token = s.step(ids, 5, seen)
        assert bool(((token >= 0) & (token < s.V)).all())
        s.check(seen, 5)
    assert s.lens.tolist() == [7 + 8, 3, 18 + 8, 30 + 8, 3 + 8]


def test_serving_loop_captured():
    """The step captured with its state updated in place, replayed with the tokens that it gave, equals the eager steps."""
    a, token_a = started(91)
    b, token = started(91)
    assert torch.equal(token_a, token)
    ids, side = token.clone(), torch.cuda.Stream()
    keep = [t.clone() for t in (b.table, b.lens, b.ring, b.pool, *b.cache)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(ids, 5)
    torch.cuda.current_stream().wait_stream(side)
    for t, k in zip((b.table, b.lens, b.ring, b.pool, *b.cache), keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids.copy_(b.step(ids, 5))
    for step in range(6):
        u = torch.rand(5, generator=gen(step)).cuda()
        a.u.copy_(u)
        b.u.copy_(u)
        token_a = a.step(token_a, 5)
        graph.replay()
        assert torch.equal(token_a, ids)
    for x, y in zip((a.table, a.lens, a.ring, a.pool, *a.cache), (b.table, b.lens, b.ring, b.pool, *b.cache)):
        assert torch.equal(x, y)


def test_serving_loops_on_two_streams():
    """Two loops at once, each on its stream, as each alone."""
    alone = []
    for seed in (92, 93):
        s, token = started(seed)
        for _ in range(5):
            token = s.step(token, 5)
        alone.append((token, s.lens.clone()))
    loops = [started(92), started(93)]
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    tokens = [t for _, t in loops]
    for _ in range(5):
        for i, (s, _) in enumerate(loops):
            with torch.cuda.stream(streams[i]):
                tokens[i] = s.step(tokens[i], 5)
    torch.cuda.synchronize()
    for (token, lens), got, (s, _) in zip(alone, tokens, loops):
        assert torch.equal(token, got) and torch.equal(lens, s.lens)
