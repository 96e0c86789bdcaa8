"""GPU parity of paged_extend where its ring and its rows are not as a fresh server has them: rings with fewer places than there
are pages."""
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
