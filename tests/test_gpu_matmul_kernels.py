"""GPU parity of every kernel and variant of the block-scaled FP8 product against 64 bits, at sizes whose choice
tests/test_matmul_plan_host.py pins down."""
import math

import pytest
import torch

import fp8_quant_memory_gb300 as fq
import matmul_cases as cases
import serving_ref as ref
from test_gpu_serving import DT, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_state(cuda_ok):
    yield
    torch.cuda.synchronize()
    assert fq.device_status(clear=True) == 0


def inputs(M, N, K, seed, operand_pad=0):
    """Operands with `operand_pad` NaN codes behind each row."""
    g = gen(seed)
    G, NB = -(-K // 128), -(-N // 128)
    a, b = (torch.full((rows, K + operand_pad), 0x7F, dtype=torch.uint8) for rows in (M, N))
    a[:, :K], b[:, :K] = ref.finite_codes((M, K), g), ref.finite_codes((N, K), g)
    sa = torch.rand(M, G, generator=g) * 2e-2 + 1e-4
    sb = torch.rand(NB, G, generator=g) * 2e-4 + 1e-6
    a, sa, b, sb = (t.cuda() for t in (a, sa, b, sb))
    return a[:, :K], sa, b[:, :K], sb


def output(M, N, dtype, tensor_map):
    """(buffer of 7s, view [M, N]): rows whole 16-byte pieces apart, or an odd number of elements."""
    stride = (N + 15) // 8 * 8 if tensor_map else (N + 2) // 2 * 2 + 1
    buf = torch.full((M, stride), 7.0, dtype=dtype, device="cuda")
    return buf, buf[:, :N]


def chosen(want, size):
    if torch.cuda.get_device_properties(0).multi_processor_count == cases.SMS:
        assert cases.plan(*size) == want


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("want, size", cases.NARROW.items(), ids=str)
def test_few_rows(want, size, dt):
    chosen(want, size)
    M, N, K = size
    x = inputs(M, N, K, seed=M + N + K)
    buf, out = output(M, N, DT[dt], False)
    fq.fp8_matmul(*x, out=out)
    ref.assert_matmul(out, *x)
    assert bool((buf[:, N:] == 7.0).all())
    assert torch.equal(fq.fp8_matmul(*x, out_dtype=DT[dt]), out)


@pytest.mark.parametrize("tensor_map", [True, False], ids=["map", "direct"])
@pytest.mark.parametrize("want, size", [*cases.WIDE.items(), *cases.WIDE_MORE], ids=str)
def test_many_rows(want, size, tensor_map):
    M, N, K = size
    if tensor_map:
        N = N // 8 * 8
    chosen(want, (M, N, K))
    dtype = torch.bfloat16 if tensor_map else torch.float16
    x = inputs(M, N, K, seed=M + N + K)
    buf, out = output(M, N, dtype, tensor_map)
    fq.fp8_matmul(*x, out=out)
    ref.assert_matmul(out, *x)
    assert bool((buf[:, N:] == 7.0).all())
    again = output(M, N, dtype, tensor_map)[1]
    assert torch.equal(fq.fp8_matmul(*x, out=again), out)


@pytest.mark.parametrize("want, size", [*cases.WIDE.items(), ((128, 2, 1, 1), cases.NARROW[(128, 2, 1, 1)])], ids=str)
def test_strided_operands_and_nan(want, size):
    """Rows of the operands and their scales apart, of a length that is no multiple of 16, NaN between them; a NaN code
    inside reaches its row or column only."""
    M, N, K = size
    K -= 7
    chosen(want, (M, N, K))
    a, sa, b, sb = inputs(M, N, K, seed=3, operand_pad=55)
    sa2, sb2 = (torch.full((t.shape[0], t.shape[1] + 3), math.nan, device="cuda") for t in (sa, sb))
    sa2[:, :-3], sb2[:, :-3] = sa, sb
    clean = fq.fp8_matmul(a, sa2[:, :-3], b, sb2[:, :-3])
    ref.assert_matmul(clean, a.contiguous(), sa, b.contiguous(), sb)
    rows, cols = [0, M // 2, M - 1], [1, 257 % N, N - 1]
    a[rows, 100], b[cols, K - 1] = 0x7F, 0xFF
    out = fq.fp8_matmul(a, sa, b, sb)
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[rows], hit[:, cols] = True, True
    assert torch.equal(out.isnan(), hit) and torch.equal(out[~hit], clean[~hit])


def test_many_rows_beyond_32_bits_of_output():
    """An output of more than 2^31 elements: its last tile rows against the same rows alone."""
    M, N, K = 300000, 8200, 144
    a, sa, b, sb = inputs(4000, N, K, seed=8)
    big = a.repeat(M // 4000, 1)
    out = fq.fp8_matmul(big, sa.repeat(M // 4000, 1), b, sb)
    assert out.numel() > 2 ** 31
    few = fq.fp8_matmul(a, sa, b, sb)
    ref.assert_matmul(few[-300:], a[-300:].contiguous(), sa[-300:], b, sb)
    for at in (0, 148000, M - 4000):
        assert torch.equal(out[at:at + 4000], few)
