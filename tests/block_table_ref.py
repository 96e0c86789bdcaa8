"""A plain implementation of block tables and slot maps as include/fq.h states them, around a list of the free pages: pages are
taken from its front, then those of sequences that end (absent ones, negative, aside) go behind its last, as far as the ring
has places."""
from __future__ import annotations

MAX32 = 2 ** 31 - 1


def ceil(a, b):
    return -(-a // b)


def extend(table, lens, new, ring, pool, page, T):
    """Lists in, a dict of lists out. Places of the ring without a free page keep what they held."""
    table, ring = [list(r) for r in table], list(ring)
    F, W = len(ring), len(table[0]) if table else 0
    head, count = pool[0] % F, min(max(pool[1], 0), F)
    free = [ring[(head + i) % F] for i in range(count)]
    taken, asked, missing, ended = 0, 0, 0, []
    slots, positions, starts, out = [-1] * T, [0] * T, [0], []
    for b, (n, m) in enumerate(zip(lens, new)):
        n, start = max(n, 0), starts[-1]
        starts.append(start + max(m, 0))
        held = ceil(n, page)
        if m < 0:
            ended += [id for id in table[b][:min(held, W)] if id >= 0]
            out.append(0)
            continue
        fits = ceil(n + m, page) <= W and starts[-1] <= T
        need = ceil(n + m, page) - held if fits else 0
        asked += need
        granted = fits and (need == 0 or asked <= count)
        if granted:
            table[b][held:held + need] = free[taken:taken + need]
            taken += need
        else:
            missing += need
        out.append(n + m if granted else n)
        for i in range(min(m, max(T - start, 0))):
            positions[start + i] = min(n + i, MAX32)
            if granted and table[b][(n + i) // page] >= 0:
                slots[start + i] = table[b][(n + i) // page] * page + (n + i) % page
    ended = ended[:F - (count - taken)]
    for j, id in enumerate(ended):
        ring[(head + count + j) % F] = id
    return dict(slots=slots, positions=positions, starts=[min(s, MAX32) for s in starts], seq_lens=out,
                pool=[(head + taken) % F, count - taken + len(ended), min(missing, MAX32)], table=table, ring=ring)
