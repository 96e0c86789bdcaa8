"""GPU parity of paged_extend where its ring and its rows are not as a fresh server has them: rings with fewer places than there
are pages, rows whose pages were given back before their sequences end."""
import random

import pytest
import torch

import block_table_ref as ref
import fp8_quant_memory_gb300 as fq
from guards import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_state(cuda_ok):
    yield
    torch.cuda.synchronize()
    assert fq.device_status(clear=True) == 0


def ints(v, t=torch.int32):
    return torch.tensor(v, dtype=t, device="cuda")


def check(table, lens, new, ring, pool, page, T, in_place):
    want = ref.extend(table, lens, new, ring, pool, page, T)
    t, ln, nw, pl, rg = ints(table), ints(lens), ints(new), ints(pool), Guarded((len(ring),), torch.int32)
    rg.t.copy_(ints(ring))
    given = dict(seq_lens_out=ln, pool_out=pl) if in_place else {}
    slots, positions, starts, lens_out, pool_out = fq.paged_extend(t, ln, nw, rg.t, pl, page, T, **given)
    rg.check()
    for k, v in dict(slots=slots, positions=positions, starts=starts, seq_lens=lens_out, pool=pool_out, table=t, ring=rg.t).items():
        assert v.tolist() == want[k], k
    return want


# sequences and tokens of a step: one small block, one block, several (in place a cluster of two, four and eight)
STEPS = [(7, 40), (60, 250), (300, 900), (300, 1500), (500, 3000), (1100, 9000), (900, 20000)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,T", STEPS)
@pytest.mark.parametrize("fill", [0.0, 0.5, 0.9, 1.0])
def test_ring_smaller_than_the_pages(fill, B, T, in_place):
    """Steps that take and return pages, of a ring filled to that part: returned pages go to places that are being emptied,
    whose pages the step's tokens and rows still have to see."""
    r = random.Random(B + T)
    page, W = 8, max(6, 2 * T // (8 * B) + 4)
    lens = [r.choice([0, 1, page, r.randrange(W * page // 2)]) for _ in range(B)]
    new = [-1 if r.random() < 0.4 else 0 for _ in range(B)]
    run = [b for b in range(B) if new[b] == 0]
    for b in run:
        new[b] = r.randrange(2 * T // len(run) + 1)
    own = iter(range(10 ** 6))
    table = [[next(own) if i < ref.ceil(n, page) else -1 for i in range(W)] for n in lens]
    ended = sum(ref.ceil(n, page) for n, m in zip(lens, new) if m < 0)
    F = max(4, ended + 7)
    ring, pool = [next(own) for _ in range(F)], [r.randrange(F), round(fill * F), 5]
    want = check(table, lens, new, ring, pool, page, T, in_place)
    taken = sum(x != y for old, row in zip(table, want["table"]) for x, y in zip(old, row))
    if fill == 1.0 and ended:  # every page that returned is in a place that the step has emptied
        assert 0 < want["pool"][1] - (F - taken) <= taken


def absent(kind, ids, r):
    """A row's ids with some of them absent."""
    n = len(ids)
    if kind == "some": return [-1 if r.random() < 0.3 else x for x in ids]
    if kind == "one": return [-5 if i == n // 2 and r.random() < 0.2 else x for i, x in enumerate(ids)]
    if kind == "window": return [x if i < 1 or i >= n - 3 else -1 for i, x in enumerate(ids)]
    return [-2 ** 31] * n if kind == "all" or r.random() < 0.5 else ids


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,T,W", [(5, 40, 9), (64, 250, 40), (300, 900, 60), (400, 9000, 200), (900, 5000, 40), (3, 2000, 20000)])
@pytest.mark.parametrize("kind", ["some", "one", "window", "all", "rows"])
@pytest.mark.parametrize("small", [False, True])
def test_absent_pages_do_not_return(small, kind, B, T, W, in_place):
    """Rows of up to several thousand pages, of which some are absent; rings of enough places and of too few."""
    r = random.Random(B + T + len(kind))
    page = 4
    lens = [r.randrange(W * page - 4 * page) for _ in range(B)]
    new = [-1 if r.random() < 0.5 else r.choice([0, 1, 1, 5]) for _ in range(B)]
    new[0], new[-1] = -1, 3
    order = list(range(B * W + 200))
    r.shuffle(order)
    own = iter(order)
    table = [absent(kind if m < 0 else "", ids, r) if m < 0 else ids for ids, m in
             (([next(own) for _ in range(ref.ceil(n, page))], m) for n, m in zip(lens, new))]
    returned = sum(x >= 0 for ids, m in zip(table, new) if m < 0 for x in ids)
    table = [ids + [-1] * (W - len(ids)) for ids in table]
    free = 100
    F = max(free, free + returned // 2 if small else free + returned + 5)
    ring = [next(own) if i < free else -1 for i in range(F)]
    head = r.randrange(F)
    ring = [ring[(i - head) % F] for i in range(F)]
    want = check(table, lens, new, ring, [head, free, 0], page, T, in_place)
    held = [want["ring"][(want["pool"][0] + i) % F] for i in range(want["pool"][1])]
    assert min(held, default=0) >= 0 and len(set(held)) == len(held)


def test_pages_given_back_before_the_end_are_granted_once():
    """A window of one page over sequences of four: the two in between go back to the ring by hand, then the sequences end and
    others take all the pages."""
    page, B = 4, 6
    table = [[4 * b + i for i in range(4)] for b in range(B)]
    ring, pool = [-1] * 24, [20, 0, 0]
    back = [id for row in table for id in row[1:3]]
    for row in table:
        row[1] = row[2] = -1
    for j, id in enumerate(back):
        ring[(pool[0] + j) % 24] = id
    pool[1] = len(back)
    w = check(table, [16] * B, [-1] * B, ring, pool, page, 1, False)
    w = check([[-1] * 4] * B, [0] * B, [16] * B, w["ring"], w["pool"], page, 16 * B, True)
    assert sorted(id for row in w["table"] for id in row) == list(range(24)) and min(w["slots"]) >= 0 and w["pool"][2] == 0


def state(B, W, page, seed):
    """A state with pages to spare, some sequences of which end."""
    r = random.Random(seed)
    lens = [r.randrange(W * page // 2) for _ in range(B)]
    new = [-1 if r.random() < 0.2 else r.choice([0, 1, 1, 9]) for _ in range(B)]
    own = iter(r.sample(range(2 * B * W), 2 * B * W))
    table = [[next(own) if i < ref.ceil(n, page) else -1 for i in range(W)] for n in lens]
    return table, lens, new, [next(own) for _ in range(B * W)], [r.randrange(B * W), B * W // 2, 0]


@pytest.mark.parametrize("which", ["seq_lens_out", "pool_out"])
@pytest.mark.parametrize("B,T", [(20, 100), (300, 1000), (500, 5000), (600, 12000)])
def test_lengths_or_pool_alone_in_place(B, T, which):
    table, lens, new, ring, pool = state(B, 12, 4, B)
    want = ref.extend(table, lens, new, ring, pool, 4, T)
    t, ln, nw, rg, pl = (ints(x) for x in (table, lens, new, ring, pool))
    out = fq.paged_extend(t, ln, nw, rg, pl, 4, T, **{which: ln if which == "seq_lens_out" else pl})
    for k, v in zip(("slots", "positions", "starts", "seq_lens", "pool"), out):
        assert v.tolist() == want[k], k
    assert t.tolist() == want["table"] and rg.tolist() == want["ring"]
    assert (pl if which == "seq_lens_out" else ln).tolist() == (pool if which == "seq_lens_out" else lens)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,T", [(300, 700), (500, 5000), (600, 12000)])
def test_steps_of_many_blocks_captured(B, T, in_place):
    """Replayed with other lengths to add: as the same steps one by one."""
    page = 4
    table, lens, new, ring, pool = state(B, 12, page, B)
    t, ln, nw, rg, pl = (ints(x) for x in (table, lens, new, ring, pool))
    given = dict(seq_lens_out=ln, pool_out=pl) if in_place else {}
    call = lambda: fq.paged_extend(t, ln, nw, rg, pl, page, T, **given)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in ((t, table), (ln, lens), (rg, ring), (pl, pool)):
        x.copy_(ints(y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    r = random.Random(T)
    for _ in range(3):
        graph.replay()
        want = ref.extend(table, lens, new, ring, pool, page, T)
        for k, v in zip(("slots", "positions", "starts", "seq_lens", "pool"), out):
            assert v.tolist() == want[k], k
        assert t.tolist() == want["table"] and rg.tolist() == want["ring"]
        table, ring = want["table"], want["ring"]
        if in_place:
            lens, pool = want["seq_lens"], want["pool"]
        else:
            ln.copy_(ints(want["seq_lens"]))
            pl.copy_(ints(want["pool"]))
            lens, pool = want["seq_lens"], want["pool"]
        new = [-1 if r.random() < 0.2 else r.choice([0, 1, 5]) for _ in range(B)]
        nw.copy_(ints(new))
