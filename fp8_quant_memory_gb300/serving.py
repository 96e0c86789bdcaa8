"""Bindings of the FP8 serving operators (include/fq.h): the block-scaled FP8 matrix product, the QKV
prologue that appends to a paged FP8 cache, and paged attention of one new token.

A cache is four tensors: ``k_cache``, ``v_cache`` [pages, Hk, page_size, D] of e4m3 codes and
``k_scale``, ``v_scale`` [pages, Hk, page_size] fp32, one scale per row. Any strides that keep rows
contiguous will do (``t.transpose(1, 2)`` of a [pages, page_size, Hk, D] tensor, say), as long as k and v
share theirs. Codes are torch.uint8 or torch.float8_e4m3fn tensors of the same bytes.

Each call checks devices, dtypes and shapes on the host, runs on the current stream of the tensors'
device (which need not be the current device) and returns once its work is enqueued.
"""
from __future__ import annotations

import ctypes

import torch

from . import _capi

_CODES = (torch.uint8, torch.float8_e4m3fn)
_OUT = {torch.bfloat16: _capi.FQ_BF16, torch.float16: _capi.FQ_FP16}
_TABLE = {torch.bfloat16: _capi.FQ_BF16, torch.float16: _capi.FQ_FP16, torch.float32: _capi.FQ_FP32}


def _device(name: str, *ts) -> torch.device:
    dev = ts[0].device
    if dev.type != "cuda":
        raise ValueError(f"{name}: every tensor must be on a CUDA device")
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError(f"{name}: tensors are on different devices")
    return dev


def _need(ok: bool, name: str, what: str) -> None:
    if not ok:
        raise ValueError(f"{name}: {what}")


def _launch(fn: str, dev: torch.device, *args) -> None:
    """Call an entry point on dev's current stream, with dev the current device while it launches."""
    stream = torch.cuda.current_stream(dev).cuda_stream
    if dev.index == torch.cuda.current_device():
        _capi.call(fn, *args, stream)
    else:
        with torch.cuda.device(dev):
            _capi.call(fn, *args, stream)


def fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """out = dtype(a @ b.T) of block-scaled e4m3 operands.

    a: [M, K] codes with a_scale [M, ceil(K/128)] (what rmsnorm_rope_quant_groups(group_size=128) returns);
    b: [N, K] codes with b_scale [ceil(N/128), ceil(K/128)], one scale per 128 x 128 block of the weight.
    Returns [M, N] bfloat16 or float16, every sum in fp32 and rounded once.
    """
    name = "fp8_matmul"
    dev = _device(name, a, a_scale, b, b_scale, out)
    _need(a.dim() == 2 and b.dim() == 2 and a.shape[1] == b.shape[1] and a.shape[1] > 0, name,
          "a and b must be [M, K] and [N, K] with the same K >= 1")
    _need(a.dtype in _CODES and b.dtype in _CODES, name, "a and b must hold e4m3 codes (uint8 or float8_e4m3fn)")
    M, K = a.shape
    N = b.shape[0]
    g = -(-K // 128)
    _need(a_scale.dtype == torch.float32 and b_scale.dtype == torch.float32, name, "scales must be float32")
    _need(a_scale.shape == (M, g) and b_scale.shape == (-(-N // 128), g), name,
          f"a_scale must be [{M}, {g}] and b_scale [{-(-N // 128)}, {g}]")
    _need(a.stride(1) == 1 and b.stride(1) == 1 or K == 1, name, "rows of a and b must be contiguous")
    _need((a_scale.stride(1) == 1 and b_scale.stride(1) == 1) or g == 1, name, "rows of the scales must be contiguous")
    if out is None:
        _need(out_dtype in _OUT, name, f"out_dtype must be bfloat16 or float16, got {out_dtype}")
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    else:
        _need(out.dtype in _OUT and out.shape == (M, N) and (out.stride(1) == 1 or N == 1), name,
              f"out must be [{M}, {N}] bfloat16 or float16 with contiguous rows")
    _launch("fq_fp8_matmul", dev, a.data_ptr(), a.stride(0), a_scale.data_ptr(), a_scale.stride(0), b.data_ptr(),
            b.stride(0), b_scale.data_ptr(), b_scale.stride(0), out.data_ptr(), out.stride(0), M, N, K, _OUT[out.dtype])
    return out


def _cache(name: str, k_cache, v_cache, k_scale, v_scale) -> _capi.PagedCache:
    _need(k_cache.dim() == 4 and k_cache.shape == v_cache.shape, name,
          "k_cache and v_cache must be [pages, Hk, page_size, D] of the same shape")
    _need(k_scale.shape == k_cache.shape[:3] and v_scale.shape == k_cache.shape[:3], name,
          "k_scale and v_scale must be [pages, Hk, page_size]")
    _need(k_cache.dtype in _CODES and v_cache.dtype in _CODES, name, "the cache must hold e4m3 codes (uint8 or float8_e4m3fn)")
    _need(k_scale.dtype == torch.float32 and v_scale.dtype == torch.float32, name, "scales must be float32")
    s, z = k_cache.stride(), k_scale.stride()
    _need(v_cache.stride() == s and v_scale.stride() == z, name, "k and v must share their strides")
    _need(s[3] == 1 or k_cache.shape[3] == 1, name, "rows of the cache must be contiguous")
    return _capi.PagedCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                            k_cache.shape[0], k_cache.shape[2], s[0], s[1], s[2], z[0], z[1], z[2])


def qkv_norm_rope_append(qkv: torch.Tensor, wq: torch.Tensor, wk: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                         slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, Hq: int, Hk: int, eps: float = 1e-6, fp8_max: float = 448.0,
                         rope_dim: int | None = None, q_out: torch.Tensor | None = None,
                         q_scale: torch.Tensor | None = None):
    """QK-Norm + RoPE + FP8 prologue of whole QKV rows, K and V placed in the paged cache.

    qkv: [T, S], S >= (Hq + 2*Hk)*D: q heads, k heads, v heads. slots: [T] int64, page * page_size +
    offset per token; a slot outside the cache (-1) writes nothing there. The tokens' slots must differ.
    Returns (q codes uint8 [T, Hq, D], q_scale fp32 [T, Hq]); the cache is updated in place.
    """
    name = "qkv_norm_rope_append"
    dev = _device(name, qkv, wq, wk, cos, sin, slots, k_cache, v_cache, k_scale, v_scale, q_out, q_scale)
    cache = _cache(name, k_cache, v_cache, k_scale, v_scale)
    D = k_cache.shape[3]
    _need(Hq >= 0 and Hk >= 1 and k_cache.shape[1] == Hk, name, "need Hq >= 0 and a cache of Hk >= 1 heads")
    _need(qkv.dim() == 2 and qkv.shape[1] >= (Hq + 2 * Hk) * D and qkv.stride(1) == 1, name,
          "qkv must be [T, S] with contiguous rows of S >= (Hq + 2*Hk)*D")
    T = qkv.shape[0]
    dt = _OUT.get(qkv.dtype)
    _need(dt is not None and wq.dtype == qkv.dtype and wk.dtype == qkv.dtype, name,
          "qkv, wq and wk must share bfloat16 or float16")
    _need(wq.shape == (D,) and wk.shape == (D,) and wq.is_contiguous() and wk.is_contiguous(), name,
          f"wq and wk must be contiguous [{D}]")
    R = D if rope_dim is None else rope_dim
    _need(0 <= R <= D and R % 2 == 0, name, f"rope_dim must be even and in [0, {D}]")
    td = _TABLE.get(cos.dtype)
    _need(td is not None and sin.dtype == cos.dtype, name, "cos and sin must share one of bfloat16/float16/float32")
    _need(cos.shape == (T, R // 2) and sin.shape == (T, R // 2) and cos.is_contiguous() and sin.is_contiguous(), name,
          f"cos and sin must be contiguous [{T}, {R // 2}]")
    _need(slots.dtype == torch.int64 and slots.shape == (T,) and slots.is_contiguous(), name,
          f"slots must be contiguous int64 [{T}]")
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=torch.uint8, device=dev)
    else:
        _need(q_out.dtype in _CODES and q_out.shape == (T, Hq, D) and q_out.is_contiguous(), name,
              f"q_out must be contiguous codes [{T}, {Hq}, {D}]")
    if q_scale is None:
        q_scale = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    else:
        _need(q_scale.dtype == torch.float32 and q_scale.shape == (T, Hq) and q_scale.is_contiguous(), name,
              f"q_scale must be contiguous float32 [{T}, {Hq}]")
    _launch("fq_qkv_norm_rope_append", dev, qkv.data_ptr(), qkv.stride(0), wq.data_ptr(), wk.data_ptr(),
            cos.data_ptr(), sin.data_ptr(), slots.data_ptr(), q_out.data_ptr(), q_scale.data_ptr(),
            ctypes.byref(cache), T, Hq, Hk, D, R, dt, td, eps, fp8_max)
    return q_out, q_scale


def paged_attention_workspace_bytes(B: int, Hq: int, Hk: int, D: int, max_seq_len: int) -> int:
    """Workspace bytes of paged_attention on the current device."""
    return int(_capi.load().fq_paged_attention_workspace_bytes(B, Hq, Hk, D, max_seq_len))


def paged_attention(q: torch.Tensor, q_scale: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    k_scale: torch.Tensor, v_scale: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                    softmax_scale: float | None = None, out_dtype: torch.dtype = torch.bfloat16,
                    max_seq_len: int | None = None, want_lse: bool = False, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Attention of one new token per sequence over the paged FP8 cache. Returns (out, lse or None).

    q: [B, Hq, D] codes (rows of a sequence contiguous, any stride between sequences) with q_scale
    [B, Hq]; page_table: [B, max_pages] int32; seq_lens: [B] int32. softmax_scale defaults to D ** -0.5.
    max_seq_len: an upper bound of the lengths known on the host (default: what the page table holds);
    longer sequences are cut to it. out: [B, Hq, D]; lse: fp32 [B, Hq]. A workspace that is passed
    (uint8) must not be in use by another call that may run at the same time.
    """
    name = "paged_attention"
    dev = _device(name, q, q_scale, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, out, lse, workspace)
    cache = _cache(name, k_cache, v_cache, k_scale, v_scale)
    _need(q.dim() == 3 and q.dtype in _CODES, name, "q must hold e4m3 codes [B, Hq, D]")
    B, Hq, D = q.shape
    Hk = k_cache.shape[1]
    _need(k_cache.shape[3] == D and Hk > 0 and Hq > 0 and Hq % Hk == 0, name,
          "q and the cache must share D, and Hq must be a multiple of the cache's heads")
    _need((q.stride(2) == 1 or D == 1) and (q.stride(1) == D or Hq == 1), name, "the heads of a sequence must be contiguous in q")
    _need(q_scale.dtype == torch.float32 and q_scale.shape == (B, Hq) and (q_scale.stride(1) == 1 or Hq == 1), name,
          f"q_scale must be float32 [{B}, {Hq}] with contiguous rows")
    _need(page_table.dtype == torch.int32 and page_table.dim() == 2 and page_table.shape[0] == B and
          (page_table.stride(1) == 1 or page_table.shape[1] <= 1), name, f"page_table must be int32 [{B}, max_pages] with contiguous rows")
    _need(seq_lens.dtype == torch.int32 and seq_lens.shape == (B,) and (seq_lens.stride(0) == 1 or B <= 1), name,
          f"seq_lens must be contiguous int32 [{B}]")
    max_pages = page_table.shape[1]
    most = max_pages * k_cache.shape[2]
    max_len = most if max_seq_len is None else min(int(max_seq_len), most)
    _need(max_len >= 0, name, "max_seq_len must be >= 0")
    if out is None:
        _need(out_dtype in _OUT, name, f"out_dtype must be bfloat16 or float16, got {out_dtype}")
        out = torch.empty((B, Hq, D), dtype=out_dtype, device=dev)
    else:
        _need(out.dtype in _OUT and out.shape == (B, Hq, D) and out.is_contiguous(), name,
              f"out must be contiguous bfloat16 or float16 [{B}, {Hq}, {D}]")
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if want_lse else None
    else:
        _need(lse.dtype == torch.float32 and lse.shape == (B, Hq) and lse.is_contiguous(), name,
              f"lse must be contiguous float32 [{B}, {Hq}]")
    if workspace is None:
        with torch.cuda.device(dev):
            need = paged_attention_workspace_bytes(B, Hq, Hk, D, max_len)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    else:
        _need(workspace.is_contiguous(), name, "workspace must be contiguous")
    ws = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (None, 0)
    _launch("fq_paged_attention", dev, q.data_ptr(), q.stride(0), q_scale.data_ptr(), q_scale.stride(0),
            ctypes.byref(cache), page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr(), out.data_ptr(),
            None if lse is None else lse.data_ptr(), *ws, B, Hq, Hk, D, max_pages, max_len,
            D ** -0.5 if softmax_scale is None else softmax_scale, _OUT[out.dtype])
    return out, lse
