"""Host-side checks of the FP8 serving operators (no GPU needed): the C ABI refuses invalid arguments on
the host, before any CUDA call, and the bindings refuse tensors that are not on a CUDA device."""
import ctypes

import pytest
import torch

import fp8_quant_memory_gb300 as fq
import serving_ref as ref
from fp8_quant_memory_gb300 import _capi

P16 = 1 << 20  # a 16-byte aligned address that nothing reads
INVALID, UNSUPPORTED = _capi.FQ_ERR_INVALID_ARG, _capi.FQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from fp8_quant_memory_gb300 import build

    try:
        build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    return _capi.load()


def call(lib, name, args, over):
    a = dict(args)
    a.update(over)
    vals = [ctypes.byref(v) if isinstance(v, ctypes.Structure) else v for v in a.values()]
    return getattr(lib, name)(*vals), lib.fq_last_error().decode()


MATMUL = dict(a=P16, a_stride=256, a_scale=P16, sas=2, b=P16, b_stride=256, b_scale=P16, sbs=2, out=P16, out_stride=130,
              M=4, N=130, K=256, dtype=0, stream=None)


@pytest.mark.parametrize("over, code", [
    (dict(a=None), INVALID), (dict(a_scale=None), INVALID), (dict(b=None), INVALID), (dict(b_scale=None), INVALID),
    (dict(out=None), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(M=1 << 31), INVALID),
    (dict(K=1 << 31), INVALID), (dict(a_stride=-1), INVALID), (dict(b_stride=1 << 41), INVALID), (dict(out_stride=129), INVALID),
    (dict(a_scale=P16 + 2), INVALID), (dict(out=P16 + 1), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(dtype=9), UNSUPPORTED),
], ids=str)
def test_matmul_refusals(lib, over, code):
    rc, msg = call(lib, "fq_fp8_matmul", MATMUL, over)
    assert rc == code and "fq_fp8_matmul" in msg


def test_matmul_empty_needs_no_device(lib):
    assert call(lib, "fq_fp8_matmul", MATMUL, dict(M=0, a=None))[0] == 0
    assert call(lib, "fq_fp8_matmul", MATMUL, dict(N=0, b=None))[0] == 0


def cache(**over):
    f = dict(k=P16, v=P16, k_scale=P16, v_scale=P16, pages=10, page_size=16, page_stride=2 * 16 * 128, head_stride=16 * 128,
             token_stride=128, scale_page_stride=32, scale_head_stride=16, scale_token_stride=1)
    f.update(over)
    return _capi.PagedCache(**f)


BAD_CACHES = [dict(k=None), dict(v_scale=None), dict(pages=-1), dict(page_size=0), dict(pages=1 << 31), dict(token_stride=127),
              dict(token_stride=0), dict(head_stride=0), dict(page_stride=16 * 128), dict(page_stride=-4096),
              dict(scale_token_stride=0), dict(scale_head_stride=15), dict(scale_page_stride=31), dict(k_scale=P16 + 2),
              dict(page_stride=1 << 62)]

APPEND = dict(qkv=P16, ts=8 * 128, wq=P16, wk=P16, cos=P16, sin=P16, slots=P16, q=P16, qs=P16, cache=cache(), T=3, Hq=4, Hk=2,
              D=128, R=128, dtype=0, tdt=2, eps=1e-6, fp8_max=448.0, stream=None)


@pytest.mark.parametrize("over, code", [
    (dict(qkv=None), INVALID), (dict(wq=None), INVALID), (dict(wk=None), INVALID), (dict(cos=None), INVALID), (dict(slots=None), INVALID),
    (dict(q=None), INVALID), (dict(qs=None), INVALID), (dict(cache=None), INVALID), (dict(ts=8 * 128 - 1), INVALID), (dict(T=-1), INVALID),
    (dict(Hq=-1), INVALID), (dict(Hk=0), INVALID), (dict(D=0), INVALID), (dict(R=127), INVALID), (dict(R=130), INVALID), (dict(R=-2), INVALID),
    (dict(T=1 << 30), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(fp8_max=0.0), INVALID),
    (dict(fp8_max=449.0), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(tdt=5), UNSUPPORTED), (dict(qkv=P16 + 1), INVALID),
    (dict(slots=P16 + 4), INVALID), (dict(qs=P16 + 2), INVALID), (dict(cos=P16 + 2), INVALID)], ids=str)
def test_append_refusals(lib, over, code):
    rc, msg = call(lib, "fq_qkv_norm_rope_append", APPEND, over)
    assert rc == code and "fq_qkv_norm_rope_append" in msg


@pytest.mark.parametrize("over", BAD_CACHES, ids=str)
def test_append_refuses_bad_caches(lib, over):
    assert call(lib, "fq_qkv_norm_rope_append", APPEND, dict(cache=cache(**over)))[0] == INVALID


def test_append_empty_needs_no_device(lib):
    assert call(lib, "fq_qkv_norm_rope_append", APPEND, dict(T=0, qkv=None, slots=None))[0] == 0


ATTEND = dict(q=P16, q_stride=8 * 128, qs=P16, qss=8, cache=cache(), table=P16, ts=9, lens=P16, out=P16, lse=P16, ws=P16,
              wsb=1 << 40, B=2, Hq=8, Hk=2, D=128, max_pages=9, max_len=140, scale=0.1, dtype=0, stream=None)


@pytest.mark.parametrize("over, code", [
    (dict(q=None), INVALID), (dict(qs=None), INVALID), (dict(cache=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(B=-1), INVALID), (dict(Hq=7), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(D=0), INVALID),
    (dict(D=257), UNSUPPORTED), (dict(max_pages=-1), INVALID), (dict(max_len=-1), INVALID), (dict(ts=-1), INVALID), (dict(q_stride=-1), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(lens=P16 + 2), INVALID),
    (dict(out=P16 + 1), INVALID), (dict(lse=P16 + 2), INVALID), (dict(B=1 << 30), INVALID), (dict(Hq=1 << 17), INVALID)], ids=str)
def test_attention_refusals(lib, over, code):
    rc, msg = call(lib, "fq_paged_attention", ATTEND, over)
    assert rc == code and "fq_paged_attention" in msg


@pytest.mark.parametrize("over", BAD_CACHES, ids=str)
def test_attention_refuses_bad_caches(lib, over):
    assert call(lib, "fq_paged_attention", ATTEND, dict(cache=cache(**over)))[0] == INVALID


def test_attention_empty_needs_no_device(lib):
    assert call(lib, "fq_paged_attention", ATTEND, dict(B=0, q=None, lens=None, out=None))[0] == 0


def test_attention_workspace_is_checked(lib):
    sizes = [lib.fq_paged_attention_workspace_bytes(2, 8, 2, 128, n) for n in (0, 1, 16, 128, 1000, 10 ** 6)]
    assert sizes == sorted(sizes)
    long = dict(max_pages=9000, ts=9000, max_len=140000)
    need = lib.fq_paged_attention_workspace_bytes(2, 8, 2, 128, 140000)
    if need:
        assert call(lib, "fq_paged_attention", ATTEND, long | dict(wsb=need - 1))[0] == INVALID
        assert call(lib, "fq_paged_attention", ATTEND, long | dict(ws=None))[0] == INVALID
        assert call(lib, "fq_paged_attention", ATTEND, long | dict(ws=P16 + 8))[0] == INVALID
    for bad in ((0, 8, 2, 128, 9), (2, 7, 2, 128, 9), (2, 8, 0, 128, 9), (2, 8, 2, 300, 9), (-1, 8, 2, 128, 9)):
        assert lib.fq_paged_attention_workspace_bytes(*bad) == 0


def test_bindings_refuse_host_tensors():
    u8, f = torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8_matmul(u8, f, u8, f)
    c, s = torch.zeros(1, 1, 16, 128, dtype=torch.uint8), torch.zeros(1, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        fq.paged_attention(u8.view(2, 1, 128), f, c, c, s, s, torch.zeros(2, 1).int(), torch.zeros(2).int())


def test_reference_quantiser_and_values():
    """The 64-bit reference's e4m3 tables against torch's conversions."""
    codes = torch.arange(256, dtype=torch.int64).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    got = ref.values(codes)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got[~got.isnan()], want[~want.isnan()])
    y = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-4, 2.3, 20000)
    y = y.clamp(-448, 448)
    assert torch.equal(ref.e4m3_codes(y.double()), y.to(torch.float8_e4m3fn).view(torch.uint8))
