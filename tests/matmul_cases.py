"""Sizes of the block-scaled FP8 product that take each kernel and variant on a GPU of 152 SMs: (rows of a per tile, CTAs
that share a tile's k, groups of epilogue warps, cuts of the last round's tiles) -> (M, N, K), as fq_fp8_matmul_plan
names them. Ragged in every direction, and with enough blocks of k for each ring of stages to wrap."""
from __future__ import annotations

import ctypes

from fp8_quant_memory_gb300 import _capi

SMS = 152
NARROW = {
    (16, 1, 1, 1): (5, 9977, 1712), (16, 2, 1, 1): (9, 4903, 3344), (16, 4, 1, 1): (13, 66, 6688),
    (32, 1, 1, 1): (29, 10279, 1552), (32, 2, 1, 1): (18, 4869, 3232), (32, 4, 1, 1): (309, 129, 6208),
    (64, 1, 1, 1): (51, 10059, 1328), (64, 2, 1, 1): (47, 5243, 2576), (64, 4, 1, 1): (1252, 65, 5200),
    (64, 1, 2, 1): (50, 9769, 1440), (64, 2, 2, 1): (61, 4973, 3024), (64, 4, 2, 1): (1222, 68, 6320),
    (128, 1, 1, 1): (101, 19343, 976), (128, 2, 1, 1): (125, 6497, 2960), (128, 4, 1, 1): (1217, 137, 4048),
}
# Nine or ten rows of tiles (the walk takes eight at a time) and several columns of them, more pieces than CTA pairs;
# the last one fills its round to the last pair.
WIDE = {
    (256, 1, 1, 4): (2500, 2300, 1040), (256, 1, 1, 2): (2311, 2711, 1040), (256, 1, 1, 1): (2500, 3303, 1168),
}
WIDE_MORE = [((256, 1, 1, 4), (1000, 1001, 1040)), ((256, 1, 1, 1), (1000, 4850, 784))]


def plan(M, N, K, sms=SMS):
    p = (ctypes.c_int * 4)()
    rc = _capi.load().fq_fp8_matmul_plan(M, N, K, sms, p)
    assert rc == 0, rc
    return tuple(p)
