"""GB300-native fused attention for large head dimensions (D = 64..1024).

The computation runs in libffpa.so (hand-written sm_103a kernels behind a C
ABI, declared in include/ffpa.h).  This package only builds and loads that
library and marshals torch tensors into its descriptors; PyTorch supplies
device memory and streams.

    from head_dim_attention_gb300 import attention_fwd, attention_bwd
    out, lse = attention_fwd(q, k, v, causal=True)
    dq, dk, dv = attention_bwd(q, k, v, out, lse, dout, causal=True)

Sequences of different lengths, packed along the rows (cu_seqlens: int32
starts on the device):

    out, lse = attention_varlen_fwd(q, k, v, cu_seqlens, causal=True)
    dq, dk, dv = attention_varlen_bwd(q, k, v, cu_seqlens, out, lse, dout, causal=True)

A serving step over a cache of pages (lengths, tables and slots stay on the
device):

    cu, slots, lens, free_head = cache_plan(lens, new_lens, block_table, free_pages, free_head, page_size, max_new)
    cache_append(k, v, k_cache, v_cache, slots)
    out, lse = attention_tree_fwd(q, k_cache, v_cache, block_table, lens, draft_lens=new_lens, tree_mask=mask)
"""
from __future__ import annotations

import math

import torch

from ._lib import (  # noqa: F401
    FfpaError,
    ffpa_bwd,
    ffpa_bwd_dropout,
    ffpa_bwd_varlen,
    ffpa_cache_append,
    ffpa_cache_plan,
    ffpa_check_status,
    ffpa_fwd,
    ffpa_fwd_dropout,
    ffpa_fwd_tree,
    ffpa_fwd_varlen,
    ffpa_status_string,
    ffpa_version,
    load,
)

__all__ = ["attention_fwd", "attention_bwd", "attention_varlen_fwd", "attention_varlen_bwd",
           "attention_tree_fwd", "cache_plan", "cache_append", "ffpa_fwd_tree", "ffpa_cache_plan", "ffpa_cache_append",
           "ffpa_fwd_varlen", "ffpa_bwd_varlen", "ffpa_fwd", "ffpa_bwd", "ffpa_fwd_dropout", "ffpa_bwd_dropout",
           "ffpa_check_status",
           "ffpa_status_string", "ffpa_version", "FfpaError", "load"]


def attention_fwd(q, k, v, bias=None, causal=False, scale=None, out=None, lse=None, stream=None,
                  dropout_p=0.0, seed=0, offset=0):
    """O and lse for q [B,Hq,Nq,D], k/v [B,Hkv,Nkv,D] (CUDA f16/bf16); allocates out/lse if not given.

    dropout_p > 0 drops attention probabilities under the library's Philox
    contract (include/ffpa.h, ffpa_fwd_dropout) with the given seed and offset.
    """
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if dropout_p:
        ffpa_fwd_dropout(q, k, v, bias, causal, scale, dropout_p, seed, offset, out, lse, stream)
    else:
        ffpa_fwd(q, k, v, bias, causal, scale, out, lse, stream)
    return out, lse


def attention_bwd(q, k, v, out, lse, dout, bias=None, causal=False, scale=None, dq=None, dk=None, dv=None,
                  stream=None, dropout_p=0.0, seed=0, offset=0):
    """dQ, dK, dV for the forward that produced ``out`` and ``lse`` (with the same
    dropout_p, seed and offset); allocates outputs if not given."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if dropout_p:
        ffpa_bwd_dropout(q, k, v, bias, causal, scale, dropout_p, seed, offset, out, lse, dout, dq, dk, dv, stream)
    else:
        ffpa_bwd(q, k, v, bias, causal, scale, out, lse, dout, dq, dk, dv, stream)
    return dq, dk, dv


def attention_varlen_fwd(q, k, v, cu_seqlens, causal=False, scale=None, out=None, lse=None, stream=None):
    """O and lse of self-attention over packed sequences: q [1,Hq,T,D], k/v [1,Hkv,T,D] (any strides; a
    token-major [T,H,D] tensor x is x.transpose(0, 1)[None]), sequence s in rows cu_seqlens[s] ..
    cu_seqlens[s+1]-1 (int32, on the device); T = 0 does nothing.  Rows outside the sequences are left as they
    are (unset where out/lse are allocated here)."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    ffpa_fwd_varlen(q, k, v, cu_seqlens, causal, scale, out, lse, stream)
    return out, lse


def attention_varlen_bwd(q, k, v, cu_seqlens, out, lse, dout, causal=False, scale=None, dq=None, dk=None, dv=None,
                         stream=None):
    """dQ, dK, dV of attention_varlen_fwd; allocates outputs if not given.  Rows outside the sequences are left
    as they are."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ffpa_bwd_varlen(q, k, v, cu_seqlens, causal, scale, out, lse, dout, dq, dk, dv, stream)
    return dq, dk, dv


def attention_tree_fwd(q, k_cache, v_cache, block_table, seq_lens, draft_lens=None, tree_mask=None, scale=None,
                       out=None, lse=None, stream=None):
    """O and lse of drafted tokens q [B,Hq,T,D] over a paged cache [pages,Hkv,page,D] (any strides).

    seq_lens [B] counts a request's tokens in the cache, its drafts (the last
    draft_lens[b] of them, T each if not given) included.  A draft sees every
    token before the drafts and the drafts its row of tree_mask (bool [B or 1,
    T, T]) marks, without one those up to itself.  T = 1 is plain decoding, T <=
    128: a longer chunk of new tokens takes a call for each 128 of them.
    Rows past a request's drafts are left as they are (unset where out/lse are
    allocated here)."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    ffpa_fwd_tree(q, k_cache, v_cache, block_table, seq_lens, draft_lens, tree_mask, scale, out, lse, stream)
    return out, lse


def cache_plan(lens, new_lens, block_table, free_pages, free_head, page_size, max_new, cu_new=None, slots=None,
               lens_out=None, free_head_out=None, stream=None):
    """Pages, starts and slots of a step that adds new_lens[b] tokens to requests of lens[b] (int32 [B]).

    New pages come from free_pages (int32) from free_head (int32 [1]) on and go
    into block_table (int32 [B,max_pages]).  Returns cu_new (int32 [B+1], the
    starts of the packed new tokens), slots (int64 [max_new], -1 behind the last
    one), lens_out and free_head_out; lens and free_head themselves may be
    given for the last two."""
    # (torch.empty: Tensor.new_empty takes the host 2 us longer)
    cu_new = torch.empty(lens.shape[0] + 1, dtype=torch.int32, device=lens.device) if cu_new is None else cu_new
    slots = torch.empty(max_new, dtype=torch.int64, device=lens.device) if slots is None else slots
    if slots.shape[0] != max_new:
        raise ValueError(f"slots must have max_new = {max_new} entries, got {slots.shape[0]}")
    lens_out = torch.empty_like(lens) if lens_out is None else lens_out
    free_head_out = torch.empty_like(free_head) if free_head_out is None else free_head_out
    ffpa_cache_plan(lens, new_lens, page_size, block_table, free_pages, free_head, cu_new, slots, lens_out,
                    free_head_out, stream)
    return cu_new, slots, lens_out, free_head_out


def cache_append(k, v, k_cache, v_cache, slots, stream=None):
    """Writes the rows of k, v [1,Hkv,T,D] into pages [pages,Hkv,page,D]: row t to slot slots[t] (int64,
    page * page_size + row; negative: skipped)."""
    ffpa_cache_append(k, v, k_cache, v_cache, slots, stream)
