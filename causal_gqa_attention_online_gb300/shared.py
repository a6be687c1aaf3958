"""Attention of a batch whose sequences begin alike: the keys that they share are read
once for all of them (``attn_fwd_paged_shared``).

Beams and samples of one prompt, as ``attn_pages_fork`` leaves them, and requests behind
one system prompt share the pages of their beginnings::

    o, lse = attn_fwd_paged_shared(q, k_pages, v_pages, table, lens, cu_groups, shared_lens)

is ``attn_fwd_paged(q, k_pages, v_pages, table, lens)`` for tables whose rows
``cu_groups[n] .. cu_groups[n + 1]`` name the same pages for their first
``shared_lens[n]`` keys.  As the rest of the package this is argument marshalling only.
"""
from __future__ import annotations

import math

import torch

from .binding import _DTYPE_CODE, ALGOS, _check, load_library
from .cache import _elsewhere, _here, _raw_stream, _tensor


def attn_fwd_paged_shared(q, k_pages, v_pages, block_table, seqlens_k, cu_groups, shared_lens,
                          o=None, lse=None, *, seqlens_q=None, scale=None, algo="auto", stream=None,
                          want_lse=True):
    """Causal attention (bottom-right) of q [B,Q,Hq,D] over k_pages [P,page,Hkv,D] and
    v_pages [P,page,Hkv,Dv], tables and lengths as in attn_fwd_paged.  Group n is the
    sequences ``cu_groups[n] .. cu_groups[n + 1]`` (int32 [N + 1], ascending); the first
    ``shared_lens[n]`` keys (int32 [N]) of all of them are in the same pages, or in pages
    of equal contents.  Sequences outside every group share nothing.  ``algo``: "auto",
    "tcgen05" (the kernel that reads shared keys once) or one of attn_fwd_paged's; "auto"
    does not weigh them, and where few keys are shared (up to 8192 by four sequences of one
    token, up to 320 by 64) attn_fwd_paged is faster.
    Returns (o [B,Q,Hq,Dv], lse [B,Q,Hq] or None)."""
    i = q.get_device()
    if q.dim() != 4 or k_pages.dim() != 4 or v_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q is [B, Q, Hq, D], pages are [P, page, Hkv, D] and the block table "
                         "[B, max_pages]")
    B, Q, Hq, D = q.shape
    P, page, Hkv = k_pages.shape[:3]
    Dv, M, N = v_pages.shape[3], block_table.shape[1], shared_lens.numel()
    dtype = _DTYPE_CODE.get(q.dtype)
    if dtype is None:
        raise TypeError(f"q: dtype {q.dtype}, expected float32, float16 or bfloat16")
    qx = _tensor("q", q, q.dtype, (B, Q, Hq, D), i)
    kx = _tensor("k_pages", k_pages, q.dtype, (P, page, Hkv, D), i)
    vx = _tensor("v_pages", v_pages, q.dtype, (P, page, Hkv, Dv), i)
    table = _tensor("block_table", block_table, torch.int32, (B, M), i)
    lens = _tensor("seqlens_k", seqlens_k, torch.int32, (B,), i)
    cu = _tensor("cu_groups", cu_groups, torch.int32, (N + 1,), i)
    pre = _tensor("shared_lens", shared_lens, torch.int32, (N,), i)
    sq = None if seqlens_q is None else _tensor("seqlens_q", seqlens_q, torch.int32, (B,), i)
    if not _here(i, stream):
        with _elsewhere(q, stream):
            return attn_fwd_paged_shared(q, k_pages, v_pages, block_table, seqlens_k, cu_groups,
                                         shared_lens, o, lse, seqlens_q=seqlens_q, scale=scale,
                                         algo=algo, want_lse=want_lse)
    if o is None:
        o = torch.empty((B, Q, Hq, Dv), dtype=q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Q, Hq), dtype=torch.float32, device=q.device)
    ox = _tensor("o", o, q.dtype, (B, Q, Hq, Dv), i)
    lx = None if lse is None else _tensor("lse", lse, torch.float32, (B, Q, Hq), i)
    _check(load_library().attn_fwd_paged_shared(
        qx, kx, vx, ox, lx, B, Hq, Hkv, Q, D, Dv, table, M, page, P, sq, lens, cu, pre, N,
        1.0 / math.sqrt(D) if scale is None else float(scale), dtype, ALGOS[algo], _raw_stream(i)))
    return o, lse
