"""Bindings of the serving operators (include/fq.h): the block-scaled FP8 matrix product (with an epilogue), the QKV
prologue that appends to a paged FP8 cache, paged attention of one new token (of everything, or of a sliding window with
sinks), the block tables and slot maps of a step, and the sampling of its tokens.

A cache is four tensors: ``k_cache``, ``v_cache`` [pages, Hk, page_size, D] of e4m3 codes and
``k_scale``, ``v_scale`` [pages, Hk, page_size] fp32, one scale per row. Any strides that keep rows
contiguous will do (``t.transpose(1, 2)`` of a [pages, page_size, Hk, D] tensor, say), as long as k and v
share theirs. Codes are torch.uint8 or torch.float8_e4m3fn tensors of the same bytes.

Each call checks devices, dtypes and shapes on the host (ValueError), runs on the current stream of the
tensors' device (which need not be the current device) and returns once its work is enqueued. The checks
and the calls are compiled (csrc/fq_binding.cpp): a decoding step makes them with little work in each. The tensors that
paged_extend and sample return, where none are passed, are parts of one allocation.
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
               out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               activation: str | None = None, residual: torch.Tensor | None = None) -> torch.Tensor:
    """out = dtype(activation(a @ b.T + bias) + residual) of block-scaled e4m3 operands.

    a: [M, K] codes with a_scale [M, ceil(K/128)] (what rmsnorm_rope_quant_groups(group_size=128) returns);
    b: [N, K] codes with b_scale [ceil(N/128), ceil(K/128)], one scale per 128 x 128 block of the weight.
    bias: [N] and residual: [M, N] (any row stride, 0 too; it may be ``out`` itself) of the output's type; activation:
    None, "relu", "gelu" (erf), "gelu_tanh" or "silu".
    Returns [M, N] bfloat16 or float16, every sum and the epilogue in fp32, rounded once.
    """
    return (_native or _load()).fp8_matmul(a, a_scale, b, b_scale, out_dtype, out, bias, activation, residual)


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
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, window: int | None = None,
                    sinks: int = 0):
    """Attention of one new token per sequence over the paged FP8 cache. Returns (out, lse or None).

    q: [B, Hq, D] codes (rows of a sequence contiguous, any stride between sequences) with q_scale
    [B, Hq]; page_table: [B, max_pages] int32; seq_lens: [B] int32. softmax_scale defaults to D ** -0.5.
    max_seq_len: an upper bound of the lengths known on the host (default: what the page table holds);
    longer sequences are cut to it. out: [B, Hq, D]; lse: fp32 [B, Hq]. A workspace that is passed
    (uint8) must not be in use by another call that may run at the same time.
    window: only the last ``window`` tokens of a sequence take part, and the first ``sinks`` (None: all of them). Whoever
    returns a page that a window has passed writes a negative id in its place of page_table.
    """
    return (_native or _load()).paged_attention(q, q_scale, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                                softmax_scale, out_dtype, max_seq_len, want_lse, out, lse, workspace, window,
                                                sinks)


def paged_extend(page_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                 pool: torch.Tensor, page_size: int, max_tokens: int, slots: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, starts: torch.Tensor | None = None,
                 seq_lens_out: torch.Tensor | None = None, pool_out: torch.Tensor | None = None):
    """Block tables and slot maps of a step: adds new_lens[b] tokens to each sequence of seq_lens[b], or ends it (< 0).

    page_table: [B, max_pages], seq_lens and new_lens: [B], free_pages: [ring], a ring of the ids of free pages, pool:
    [3] = its front, how many are free, (not read); all int32. New pages come from the ring's front and enter page_table;
    those of sequences that end, but for negative (absent) ids, go behind its last (a ring of at least as many places as
    there are pages holds them all; others are dropped). Sequences whose tokens fit neither the table, nor max_tokens, nor the
    free pages are left as they are (include/fq.h has the rule).
    Returns (slots int64 [max_tokens], positions int32 [max_tokens], starts int32 [B + 1], seq_lens_out, pool_out): what
    qkv_norm_rope_append and paged_attention take, slots of -1 behind the last token. pool_out[2] counts the pages that
    were asked for and not there. seq_lens_out and pool_out may be seq_lens and pool: a captured step then advances.
    """
    return (_native or _load()).paged_extend(page_table, seq_lens, new_lens, free_pages, pool, page_size, max_tokens, slots,
                                             positions, starts, seq_lens_out, pool_out)


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None, top_k: torch.Tensor | None = None,
           top_p: torch.Tensor | None = None, min_p: torch.Tensor | None = None, want_logprob: bool = False,
           token: torch.Tensor | None = None, logprob: torch.Tensor | None = None):
    """The next token of each row of logits [B, V] (bfloat16 or float16), from uniform numbers u in [0, 1).

    temperature, top_p, min_p: fp32 [B], top_k: int32 [B], each row its own; None leaves a step out. The cuts apply in the
    order top-k, top-p, min-p to the tokens by falling logit (equal ones by rising index); u picks along that order.
    temperature 0 takes the largest; a min_p above 1 counts as 1 (the largest and its equals stay). Returns (token int64 [B], logprob fp32 [B] of the token among those kept, or None);
    -1 for a row whose mask (-inf) leaves nothing.
    """
    return (_native or _load()).sample(logits, u, temperature, top_k, top_p, min_p, want_logprob, token, logprob)
