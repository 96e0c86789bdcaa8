"""Host-side checks of the serving loop's operators (no GPU needed): refusals of the C ABI and the bindings, and the plain
implementations that the GPU tests compare with."""
import math

import pytest
import torch

import fp8_quant_memory_gb300 as fq
import serving_loop_ref as ref
from test_serving_host import ATTEND, INVALID, MATMUL, P16, UNSUPPORTED, call, lib  # noqa: F401

LINEAR = {}
for _k, _v in MATMUL.items():
    LINEAR[_k] = _v
    if _k == "out_stride":
        LINEAR.update(bias=P16, act=4, residual=P16, residual_stride=130)


@pytest.mark.parametrize("over, code", [
    (dict(a=None), INVALID), (dict(out=None), INVALID), (dict(K=0), INVALID), (dict(out_stride=129), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(act=5), UNSUPPORTED), (dict(act=-1), UNSUPPORTED), (dict(residual_stride=-1), INVALID), (dict(residual_stride=1 << 41), INVALID),
    (dict(bias=P16 + 1), INVALID), (dict(residual=P16 + 1), INVALID)], ids=str)
def test_linear_refusals(lib, over, code):  # noqa: F811
    rc, msg = call(lib, "fq_fp8_matmul_epilogue", LINEAR, over)
    assert rc == code and "fq_fp8_matmul_epilogue" in msg


def test_linear_empty_needs_no_device(lib):  # noqa: F811
    assert call(lib, "fq_fp8_matmul_epilogue", LINEAR, dict(M=0, a=None))[0] == 0


WINDOW = {}
for _k, _v in ATTEND.items():
    if _k == "scale":
        WINDOW.update(window=20, sinks=4)
    WINDOW[_k] = _v


@pytest.mark.parametrize("over", [dict(window=0), dict(window=-5), dict(sinks=-1), dict(q=None), dict(D=0), dict(max_len=-1), dict(out=P16 + 1)], ids=str)
def test_window_refusals(lib, over):  # noqa: F811
    rc, msg = call(lib, "fq_paged_attention_window", WINDOW, over)
    assert rc == INVALID and "fq_paged_attention_window" in msg


def test_window_empty_needs_no_device(lib):  # noqa: F811
    assert call(lib, "fq_paged_attention_window", WINDOW, dict(B=0, q=None, lens=None, out=None))[0] == 0


EXTEND = dict(table=P16, table_stride=9, lens=P16, new=P16, ring=P16, F=100, pool=P16, lens_out=P16, pool_out=P16, slots=P16, positions=P16, starts=P16,
              B=3, W=9, page=16, T=50, stream=None)


@pytest.mark.parametrize("over, code", [
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(new=None), INVALID), (dict(ring=None), INVALID), (dict(pool=None), INVALID),
    (dict(lens_out=None), INVALID), (dict(pool_out=None), INVALID), (dict(slots=None), INVALID), (dict(positions=None), INVALID),
    (dict(starts=None), INVALID), (dict(B=-1), INVALID), (dict(W=-1), INVALID), (dict(page=0), INVALID), (dict(T=-1), INVALID), (dict(F=0), INVALID),
    (dict(table_stride=8), INVALID), (dict(table_stride=1 << 41), INVALID), (dict(T=1 << 31), INVALID), (dict(F=1 << 31), INVALID),
    (dict(W=1 << 20, table_stride=1 << 20, page=1 << 12), INVALID), (dict(B=12289), UNSUPPORTED), (dict(slots=P16 + 4), INVALID),
    (dict(lens=P16 + 2), INVALID), (dict(table=P16 + 1), INVALID)], ids=str)
def test_extend_refusals(lib, over, code):  # noqa: F811
    rc, msg = call(lib, "fq_paged_extend", EXTEND, over)
    assert rc == code and "fq_paged_extend" in msg


SAMPLE = dict(logits=P16, stride=1000, u=P16, heat=P16, k=P16, top_p=P16, min_p=P16, token=P16, logprob=P16, B=4, V=1000, dtype=0, stream=None)


@pytest.mark.parametrize("over, code", [
    (dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(token=None), INVALID), (dict(B=-1), INVALID), (dict(B=1 << 31), INVALID),
    (dict(V=0), INVALID), (dict(V=1 << 31), INVALID), (dict(stride=-1), INVALID), (dict(stride=1 << 41), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(logits=P16 + 1), INVALID), (dict(u=P16 + 2), INVALID), (dict(heat=P16 + 1), INVALID), (dict(k=P16 + 2), INVALID), (dict(token=P16 + 4), INVALID),
    (dict(logprob=P16 + 2), INVALID)], ids=str)
def test_sample_refusals(lib, over, code):  # noqa: F811
    rc, msg = call(lib, "fq_sample", SAMPLE, over)
    assert rc == code and "fq_sample" in msg


def test_sample_empty_needs_no_device(lib):  # noqa: F811
    assert call(lib, "fq_sample", SAMPLE, dict(B=0, logits=None, u=None, token=None))[0] == 0


def test_bindings_refuse_host_tensors():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fq.paged_extend(i.view(3, 1), i, i, i, i, 16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        fq.sample(torch.zeros(2, 9, dtype=torch.bfloat16), torch.zeros(2))
    u8, f = torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 1)
    with pytest.raises(ValueError, match="activation"):
        fq.fp8_matmul(u8, f, u8, f, activation="tanh")


def test_reference_step_by_hand():
    """Three sequences on pages of 4: one grows into a new page, one ends, one starts; then none are left for a fourth."""
    w = ref.extend([[7, -1], [3, 9], [-1, -1], [-1, -1]], [3, 5, 0, 0], [2, -1, 5, 1], [10, 11, 12, 13, 14], [3, 3, 0], 4, 9)
    assert w["table"] == [[7, 13], [3, 9], [14, 10], [-1, -1]] and w["seq_lens"] == [5, 0, 5, 0]
    assert w["starts"] == [0, 2, 2, 7, 8] and w["slots"] == [31, 52, 56, 57, 58, 59, 40, -1, -1]
    assert w["positions"] == [3, 4, 0, 1, 2, 3, 4, 0, 0]
    assert w["pool"] == [1, 2, 1] and w["ring"] == [10, 3, 9, 13, 14]


def test_reference_sample_by_hand():
    x = torch.log(torch.tensor([1.0, 4.0, 2.0, 4.0, 0.5], dtype=torch.float64))
    assert [ref.sample(x, u)[0] for u in (0.0, 0.34, 0.36, 0.69, 0.7, 0.86, 0.88, 0.95, 0.97)] == [1, 1, 3, 3, 2, 2, 0, 0, 4]
    assert ref.sample(x, 0.99, k=2)[0] == 3 and ref.sample(x, 0.99, top_p=0.36)[0] == 3 and ref.sample(x, 0.99, min_p=0.3)[0] == 2
    assert ref.sample(x, 0.99, heat=0.0)[0] == 1 and abs(ref.sample(x, 0.99, k=3)[1] - math.log(0.2)) < 1e-12
    assert ref.sample(torch.full((3,), -math.inf, dtype=torch.float64), 0.5)[:2] == (-1, -math.inf)
