"""Which kernel the block-scaled FP8 product takes (fq_fp8_matmul_plan, no GPU needed): the sizes that the GPU tests use
reach every kernel and variant there is, so a change of the choice cannot leave one without its test."""
import ctypes

import pytest

import matmul_cases as cases
from fp8_quant_memory_gb300 import _capi


@pytest.fixture(scope="module", autouse=True)
def lib():
    from fp8_quant_memory_gb300 import build

    try:
        build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    return _capi.load()


@pytest.mark.parametrize("want, size", [*cases.NARROW.items(), *cases.WIDE.items(), *cases.WIDE_MORE], ids=str)
def test_sizes_take_their_kernel(want, size):
    assert cases.plan(*size) == want


def test_every_variant_has_a_size():
    narrow = {(rows, split, 1, 1) for rows in (16, 32, 64, 128) for split in (1, 2, 4)} | {(64, split, 2, 1) for split in (1, 2, 4)}
    assert set(cases.NARROW) == narrow
    assert set(cases.WIDE) == {(256, 1, 1, cuts) for cuts in (1, 2, 4)}


@pytest.mark.parametrize("size", [(1, 128 * 65535 + 1, 16384), (16, 128 * 65536, 12000), (40, 1 << 30, 1 << 16), (128 * 65535 + 1, 16, 1 << 20)], ids=str)
def test_more_tiles_than_a_grid_axis(size):
    """The few-row kernel has a tile per place of two grid axes of at most 65535: beyond, the CTA pairs take it."""
    assert cases.plan(*size)[0] == 256


def test_plan_refusals(lib):
    p = (ctypes.c_int * 4)()
    assert lib.fq_fp8_matmul_plan(1, 1, 1, 2, p) == 0
    for bad in ((0, 1, 1, 152), (1, 0, 1, 152), (1, 1, 0, 152), (1 << 31, 1, 1, 152), (1, 1 << 31, 1, 152), (1, 1, 1 << 31, 152), (1, 1, 1, 1)):
        assert lib.fq_fp8_matmul_plan(*bad, p) == _capi.FQ_ERR_INVALID_ARG
    assert lib.fq_fp8_matmul_plan(1, 1, 1, 152, None) == _capi.FQ_ERR_INVALID_ARG
