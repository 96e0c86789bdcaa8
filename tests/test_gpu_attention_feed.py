"""GPU parity of how paged attention brings the cache to the SMs: scales that are not contiguous or not aligned, page
tables read far ahead, and runs of units long enough for the rings of stages to go round several times."""
import pytest
import torch

import fp8_quant_memory_gb300 as fq
import serving_ref as ref
from test_gpu_serving import attention_inputs, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_state(cuda_ok):
    yield
    torch.cuda.synchronize()
    assert fq.device_status(clear=True) == 0


@pytest.mark.parametrize("order", ["pthd", "hptd", "htpd"])
@pytest.mark.parametrize("Hq,Hk,D,page", [(32, 4, 128, 16), (8, 4, 128, 64), (16, 4, 192, 16), (64, 4, 256, 32), (8, 4, 64, 16), (12, 4, 96, 8)])
def test_scales_apart(Hq, Hk, D, page, order):
    """Boxes of codes whose scales lie a stride apart, in caches whose page, head and token axes come in any order."""
    lens = [700, 0, 1, 129, 333, 64]
    x = attention_inputs(lens, Hq, Hk, D, page, seed=110, order=order)
    assert x[4].stride(2) != 1 or order == "hptd"
    x[6][0, 2], x[6][4, 1] = -1, x[2].shape[0]
    check_attention(x)


@pytest.mark.parametrize("Hq,Hk,D,page", [(32, 8, 128, 64), (32, 2, 256, 32)])
def test_scales_off_a_16_byte_boundary(Hq, Hk, D, page):
    x = attention_inputs([500, 3, 130], Hq, Hk, D, page, seed=111)
    for i in (4, 5):
        flat = torch.empty(x[i].numel() + 1, device="cuda")
        flat[1:].copy_(x[i].flatten())
        x[i] = flat[1:].view(x[i].shape)
        assert x[i].data_ptr() % 16 == 4
    check_attention(x)


@pytest.mark.parametrize("Hq,Hk,D,page,order", [(16, 8, 128, 8, "phtd"), (8, 8, 128, 16, "pthd"), (10, 5, 64, 16, "phtd"), (16, 4, 96, 24, "phtd")])
def test_page_tables_of_many_windows(Hq, Hk, D, page, order):
    """Tens of units of one head per block, each up to 16 pages: the table row is read 32 entries at a time, several
    times over; absent pages beyond the first of these."""
    lens = [3000 + 97 * i for i in range(32)]
    x = attention_inputs(lens, Hq, Hk, D, page, seed=112, order=order)
    for b in range(32):
        x[6][b, 33 + 3 * b], x[6][b, 64 + b], x[6][b, lens[b] // page - 1] = -1, 10 ** 6, -3
    check_attention(x)


@pytest.mark.parametrize("Hq,Hk,D,page", [(8, 2, 128, 64), (32, 2, 128, 64), (8, 2, 256, 32), (32, 2, 256, 32), (48, 2, 192, 16), (4, 4, 64, 64),
                                          (32, 2, 64, 7)])
def test_many_units_per_block(Hq, Hk, D, page):
    """Ten units and more per block: every ring of stages goes round several times, within a head and across heads."""
    lens = [8000 + 61 * i for i in range(24)] + [100 * i for i in range(24)]
    check_attention(attention_inputs(lens, Hq, Hk, D, page, seed=113))


def test_one_block_long_ring():
    """Batches far larger than the grid, heads short and long in turn."""
    lens = [9000 if i % 7 == 0 else 40 * (i % 11) for i in range(120)]
    x = attention_inputs(lens, 4, 2, 128, 32, seed=114)
    check_attention(x)
    first = fq.paged_attention(*x, want_lse=True)
    again = fq.paged_attention(*x, want_lse=True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("page", [7, 32])
@pytest.mark.parametrize("G", [5, 12, 20])
@pytest.mark.parametrize("D", [48, 112, 176, 240])
def test_every_kernel(D, G, page):
    """Head sizes below each padded one, groups of up to 8 query heads, up to 16 and more, rows copied one by one and as
    boxes; heads that end in the middle of a block and of a unit."""
    lens = [1700, 0, 900, 33, 16, 511, 1, 1024, 77]
    x = attention_inputs(lens, 2 * G, 2, D, page, seed=115, q_extra=1)
    x[6][0, 9], x[6][5, 0] = -1, -1
    check_attention(x, "fp16" if G == 12 else "bf16")


@pytest.mark.parametrize("D,page", [(128, 16), (96, 32), (80, 7), (240, 16), (64, 24), (16, 64)])
def test_rows_of_a_wider_cache(D, page):
    """A cache that is the first D columns of wider rows, NaN codes behind them."""
    x = attention_inputs([400, 31, 0, 1000], 8, 2, D, page, seed=116)
    for i in (2, 3):
        wide = torch.full((*x[i].shape[:3], D + 32), 0x7F, dtype=torch.uint8, device="cuda")
        wide[..., :D] = x[i]
        x[i] = wide[..., :D]
    check_attention(x)


@pytest.mark.parametrize("Hq,Hk,D", [(32, 8, 128), (32, 2, 256)])
def test_captured_with_other_lengths(Hq, Hk, D):
    """One captured call, replayed as sequences grow, end and start: its split follows the lengths of each replay."""
    most, page = 3000, 16
    x = attention_inputs([most] * 6, Hq, Hk, D, page, seed=117)
    lens = x[7]
    held = lens.clone()
    fq.paged_attention(*x, max_seq_len=most, want_lse=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fq.paged_attention(*x, max_seq_len=most, want_lse=True)
    for now in ([0] * 6, [1, 0, most, 5, 0, 0], [2999, 2048, 0, 1, 130, 700], [0, 0, 0, 0, 0, 17], [most] * 6, [1] * 6):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        ref.assert_attention(out, lse, *x, D ** -0.5)
        eager = fq.paged_attention(*x, max_seq_len=most, want_lse=True)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
    lens.copy_(held)


def test_two_threads():
    """Calls of two host threads at once, each on its own stream with its own tensors."""
    from concurrent.futures import ThreadPoolExecutor

    xs = [attention_inputs([500 + 300 * i, 40, 0, 1200], 8, 2, 128, 16, seed=118 + i) for i in range(2)]
    alone = [fq.paged_attention(*x, want_lse=True) for x in xs]
    torch.cuda.synchronize()

    def many(x):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            got = [fq.paged_attention(*x, want_lse=True) for _ in range(50)]
        stream.synchronize()
        return got

    with ThreadPoolExecutor(2) as pool:
        for want, got in zip(alone, pool.map(many, xs)):
            assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
