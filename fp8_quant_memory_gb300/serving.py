"""Bindings of the FP8 serving operators (include/fq.h): the block-scaled FP8 matrix product, the QKV
prologue that appends to a paged FP8 cache, and paged attention of one new token.

A cache is four tensors: ``k_cache``, ``v_cache`` [pages, Hk, page_size, D] of e4m3 codes and
``k_scale``, ``v_scale`` [pages, Hk, page_size] fp32, one scale per row. Any strides that keep rows
contiguous will do (``t.transpose(1, 2)`` of a [pages, page_size, Hk, D] tensor, say), as long as k and v
share theirs. Codes are torch.uint8 or torch.float8_e4m3fn tensors of the same bytes.

Each call checks devices, dtypes and shapes on the host (ValueError), runs on the current stream of the
tensors' device (which need not be the current device) and returns once its work is enqueued. The checks
and the calls are compiled (csrc/fq_binding.cpp): a decoding step makes them with little work in each.
"""
from __future__ import annotations

import importlib.util
import os
import threading

import torch

from . import _capi
from . import build as _build

_native = None
_lock = threading.Lock()


def _load():
    """The compiled binding (raises if it has not been built)."""
    global _native
    with _lock:
        if _native is None:
            _capi.load()
            path = _build.BINDING
            if not os.path.exists(path):
                raise RuntimeError(f"the binding is not built ({path} missing): run "
                                   "`python -c \"import __graft_entry__ as g; g.build()\"` on a machine with nvcc")
            spec = importlib.util.spec_from_file_location("_fq_binding", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.set_error_class(_capi.FqError)
            _native = module
    return _native


def fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """out = dtype(a @ b.T) of block-scaled e4m3 operands.

    a: [M, K] codes with a_scale [M, ceil(K/128)] (what rmsnorm_rope_quant_groups(group_size=128) returns);
    b: [N, K] codes with b_scale [ceil(N/128), ceil(K/128)], one scale per 128 x 128 block of the weight.
    Returns [M, N] bfloat16 or float16, every sum in fp32 and rounded once.
    """
    return (_native or _load()).fp8_matmul(a, a_scale, b, b_scale, out_dtype, out)


def qkv_norm_rope_append(qkv: torch.Tensor, wq: torch.Tensor, wk: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                         slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, Hq: int, Hk: int, eps: float = 1e-6, fp8_max: float = 448.0,
                         rope_dim: int | None = None, q_out: torch.Tensor | None = None,
                         q_scale: torch.Tensor | None = None):
    """QK-Norm + RoPE + FP8 prologue of whole QKV rows, K and V placed in the paged cache.

    qkv: [T, S], S >= (Hq + 2*Hk)*D: q heads, k heads, v heads. slots: [T] int64, page * page_size +
    offset per token; a slot outside the cache (-1) writes nothing there. The tokens' slots must differ.
    Returns (q codes uint8 [T, Hq, D], q_scale fp32 [T, Hq]); the cache is updated in place. The last place of q and k
    scales, and a few of their codes in a million, at ties, depend on how a prompt is cut into calls.
    """
    return (_native or _load()).qkv_norm_rope_append(qkv, wq, wk, cos, sin, slots, k_cache, v_cache, k_scale, v_scale,
                                                     Hq, Hk, eps, fp8_max, rope_dim, q_out, q_scale)


def paged_attention_workspace_bytes(B: int, Hq: int, Hk: int, D: int, max_seq_len: int) -> int:
    """Workspace bytes of paged_attention on the current device (enough for any smaller max_seq_len too)."""
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
    return (_native or _load()).paged_attention(q, q_scale, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                                softmax_scale, out_dtype, max_seq_len, want_lse, out, lse, workspace)
