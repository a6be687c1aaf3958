"""The 8-bit paged K/V cache: appending rows, attention over it, and the
management of its pages (the entry points of include/attn_gqa.h that begin with
``attn_cache_`` and ``attn_pages_``, and ``attn_fwd_paged_q8``).

A cache is a pair of pools, ``k_pages`` [P, page, Hkv, D] and ``v_pages``
[P, page, Hkv, Dv] of ``torch.int8`` or ``torch.float8_e4m3fn`` codes, with one
float32 scale for each block of tokens of a page and head, ``k_scale`` and
``v_scale`` [P, page / block, Hkv]; key j of sequence b is row j % page of page
``block_table[b, j // page]`` and stands for code * scale.

One decoding step of a batch::

    table, lens, refs, status = attn_pages_fork(pools, table, lens, refs, parents, page,
                                                new_tokens=new)   # pages for the step
    attn_cache_append(k, v, kp, vp, ks, vs, table, lens, seqlens_new=new)   # per layer
    o, lse = attn_fwd_paged_q8(q, kp, vp, ks, vs, table, lens + new)
    lens += new

As the rest of the package this is argument marshalling only: calls enqueue
kernels on ``stream`` (default: the current stream of the tensors' device) and
return.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import (_DTYPE_CODE, ALGOS, MASKS, _check, _check_tensor, _ptr, load_library)

ATTN_CACHE_E4M3, ATTN_CACHE_INT8 = 0, 1
_CACHE_CODE = {torch.float8_e4m3fn: ATTN_CACHE_E4M3, torch.int8: ATTN_CACHE_INT8}


class _Launch:
    """The device and stream of a call: ``dev`` is made current while the
    library runs (it works on the current device), and outputs that the call
    allocates belong to its stream."""

    def __init__(self, dev, stream):
        if dev.type != "cuda":
            raise ValueError(f"the tensors are on {dev}: the library runs on CUDA devices only")
        if stream is not None and stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        self.stream, self.guard, self.dev = stream, None, dev

    def __enter__(self):
        if self.stream is not None:  # makes its device current, too
            self.guard = torch.cuda.stream(self.stream)
            self.guard.__enter__()
            return ctypes.c_void_p(self.stream.cuda_stream)
        if torch.cuda.current_device() != self.dev.index:
            self.guard = torch.cuda.device(self.dev)
            self.guard.__enter__()
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _check_cache(k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, dev):
    """Checks a cache; returns (P, page, block, Hkv, D, Dv, B, max_pages, code)."""
    if k_pages.dim() != 4 or v_pages.dim() != 4 or k_scale.dim() != 3 or block_table.dim() != 2:
        raise ValueError("pages are [P, page, Hkv, D], scales [P, page / block, Hkv] and the "
                         "block table [B, max_pages]")
    if k_pages.dtype not in _CACHE_CODE:
        raise TypeError(f"k_pages: dtype {k_pages.dtype}, expected torch.int8 or "
                        "torch.float8_e4m3fn")
    P, page, Hkv, D = k_pages.shape
    Dv, nblk = v_pages.shape[3], k_scale.shape[1]
    B, max_pages = block_table.shape
    if tuple(v_pages.shape) != (P, page, Hkv, Dv):
        raise ValueError(f"v_pages: shape {tuple(v_pages.shape)} beside k_pages "
                         f"{tuple(k_pages.shape)}")
    if nblk < 1 or page % nblk:
        raise ValueError(f"k_scale: {nblk} blocks do not divide a page of {page} tokens")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if tuple(t.shape) != (P, nblk, Hkv):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(P, nblk, Hkv)}")
    _check_tensor("k_pages", k_pages, k_pages.dtype, P * page * Hkv * D, dev)
    _check_tensor("v_pages", v_pages, k_pages.dtype, P * page * Hkv * Dv, dev)
    _check_tensor("k_scale", k_scale, torch.float32, P * nblk * Hkv, dev)
    _check_tensor("v_scale", v_scale, torch.float32, P * nblk * Hkv, dev)
    _check_tensor("block_table", block_table, torch.int32, B * max_pages, dev)
    _check_tensor("seqlens_k", seqlens_k, torch.int32, B, dev)
    return P, page, page // nblk, Hkv, D, Dv, B, max_pages, _CACHE_CODE[k_pages.dtype]


def attn_cache_append(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, *,
                      seqlens_new=None, stream=None):
    """Writes new rows k [B,N,Hkv,D], v [B,N,Hkv,Dv] (fp32, fp16 or bf16) into
    the cache behind the ``seqlens_k`` rows each sequence has; ``seqlens_new``
    int32 [B]: how many of the N are there (default: all).  The pages they go to
    are in ``block_table`` already.  ``seqlens_k`` is not changed."""
    lib = load_library()
    dev = k.device
    P, page, block, Hkv, D, Dv, B, M, code = _check_cache(k_pages, v_pages, k_scale, v_scale,
                                                          block_table, seqlens_k, dev)
    if k.dim() != 4 or k.shape[0] != B or tuple(k.shape[2:]) != (Hkv, D):
        raise ValueError(f"k: shape {tuple(k.shape)}, expected [{B}, N, {Hkv}, {D}]")
    if k.dtype not in _DTYPE_CODE:
        raise TypeError(f"k: dtype {k.dtype}, expected float32, float16 or bfloat16")
    N = k.shape[1]
    _check_tensor("k", k, k.dtype, B * N * Hkv * D, dev)
    _check_tensor("v", v, k.dtype, B * N * Hkv * Dv, dev)
    if seqlens_new is not None:
        _check_tensor("seqlens_new", seqlens_new, torch.int32, B, dev)
    with _Launch(dev, stream) as st:
        _check(lib.attn_cache_append(_ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages),
                                     _ptr(k_scale), _ptr(v_scale), B, N, Hkv, D, Dv,
                                     _ptr(seqlens_new), _ptr(seqlens_k), _ptr(block_table), M,
                                     page, P, block, code, _DTYPE_CODE[k.dtype], st))


def attn_cache_append_varlen(k, v, cu_seqlens_new, max_new, k_pages, v_pages, k_scale, v_scale,
                             block_table, seqlens_k, *, stream=None):
    """attn_cache_append with the new rows packed: k [T,Hkv,D], v [T,Hkv,Dv],
    sequence b's rows [cu_seqlens_new[b], cu_seqlens_new[b + 1]), at most
    ``max_new`` of them."""
    lib = load_library()
    dev = k.device
    P, page, block, Hkv, D, Dv, B, M, code = _check_cache(k_pages, v_pages, k_scale, v_scale,
                                                          block_table, seqlens_k, dev)
    if k.dim() != 3 or tuple(k.shape[1:]) != (Hkv, D):
        raise ValueError(f"k: shape {tuple(k.shape)}, expected [T, {Hkv}, {D}]")
    if k.dtype not in _DTYPE_CODE:
        raise TypeError(f"k: dtype {k.dtype}, expected float32, float16 or bfloat16")
    T = k.shape[0]
    _check_tensor("k", k, k.dtype, T * Hkv * D, dev)
    _check_tensor("v", v, k.dtype, T * Hkv * Dv, dev)
    _check_tensor("cu_seqlens_new", cu_seqlens_new, torch.int32, B + 1, dev)
    with _Launch(dev, stream) as st:
        _check(lib.attn_cache_append_varlen(_ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages),
                                            _ptr(k_scale), _ptr(v_scale), B, T, int(max_new),
                                            Hkv, D, Dv, _ptr(cu_seqlens_new), _ptr(seqlens_k),
                                            _ptr(block_table), M, page, P, block, code,
                                            _DTYPE_CODE[k.dtype], st))


def attn_fwd_paged_q8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, o=None,
                      lse=None, *, seqlens_q=None, window=0, scale=None, algo="auto",
                      mask="causal", stream=None, want_lse=True):
    """attn_fwd_paged over an 8-bit cache: q [B,Q,Hq,D]; ``seqlens_k`` counts the
    keys to attend to (append first).  Returns (o [B,Q,Hq,Dv], lse [B,Q,Hq] or
    None)."""
    lib = load_library()
    dev = q.device
    P, page, block, Hkv, D, Dv, B, M, code = _check_cache(k_pages, v_pages, k_scale, v_scale,
                                                          block_table, seqlens_k, dev)
    if q.dim() != 4 or q.shape[0] != B or q.shape[3] != D:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [{B}, Q, Hq, {D}]")
    if q.dtype not in _DTYPE_CODE:
        raise TypeError(f"q: dtype {q.dtype}, expected float32, float16 or bfloat16")
    Q, Hq = q.shape[1], q.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with _Launch(dev, stream) as st:
        if o is None:
            o = torch.empty((B, Q, Hq, Dv), dtype=q.dtype, device=dev)
        if lse is None and want_lse:
            lse = torch.empty((B, Q, Hq), dtype=torch.float32, device=dev)
        _check_tensor("q", q, q.dtype, B * Q * Hq * D, dev)
        _check_tensor("o", o, q.dtype, B * Q * Hq * Dv, dev)
        if lse is not None:
            _check_tensor("lse", lse, torch.float32, B * Q * Hq, dev)
        if seqlens_q is not None:
            _check_tensor("seqlens_q", seqlens_q, torch.int32, B, dev)
        _check(lib.attn_fwd_paged_q8(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale),
                                     _ptr(v_scale), _ptr(o), _ptr(lse), B, Hq, Hkv, Q, D, Dv,
                                     _ptr(block_table), M, page, P, block, code,
                                     _ptr(seqlens_q), _ptr(seqlens_k), int(window), float(scale),
                                     MASKS[mask], _DTYPE_CODE[q.dtype], ALGOS[algo], st))
    return o, lse


def _pool_arrays(pools, pages, dev, what):
    """Pointers and page bytes of pools whose first axis counts ``pages`` pages."""
    n = len(pools)
    ptrs, sizes = (ctypes.c_void_p * max(n, 1))(), (ctypes.c_longlong * max(n, 1))()
    for i, t in enumerate(pools):
        if t.dim() < 1 or t.shape[0] != pages:
            raise ValueError(f"{what}[{i}]: shape {tuple(t.shape)}, expected {pages} pages first")
        if not t.is_contiguous():
            raise ValueError(f"{what}[{i}] must be contiguous")
        if t.device != dev:
            raise ValueError(f"{what}[{i}] is on {t.device}, expected {dev}")
        ptrs[i] = t.data_ptr()
        sizes[i] = t.numel() // pages * t.element_size()
    return ptrs, sizes, n


def attn_pages_copy(src_pools, dst_pools, src, dst, *, stream=None):
    """Copies page ``src[i]`` of each of ``src_pools`` to page ``dst[i]`` of the
    pool at the same place of ``dst_pools`` (the same list to copy within it).
    ``src``, ``dst``: int32 [n]; the dst pages are distinct, and none of them is
    a src page of the same pool.  Pairs with a page that does not exist are
    skipped."""
    lib = load_library()
    dev = src.device
    if len(src_pools) != len(dst_pools):
        raise ValueError(f"{len(src_pools)} source pools and {len(dst_pools)} destinations")
    n = src.numel()
    _check_tensor("src", src, torch.int32, n, dev)
    _check_tensor("dst", dst, torch.int32, n, dev)
    sp = src_pools[0].shape[0] if len(src_pools) else 0
    dp = dst_pools[0].shape[0] if len(dst_pools) else 0
    sptr, sbytes, npools = _pool_arrays(src_pools, sp, dev, "src_pools")
    dptr, dbytes, _ = _pool_arrays(dst_pools, dp, dev, "dst_pools")
    if any(sbytes[i] != dbytes[i] for i in range(npools)):
        raise ValueError("the pages of a source pool and of its destination differ in size")
    with _Launch(dev, stream) as st:
        _check(lib.attn_pages_copy(sptr, dptr, sbytes, npools, sp, dp, _ptr(src), _ptr(dst), n, st))


def attn_pages_fork(pools, block_table, seqlens, refcount, parents, page_size, *, new_tokens=None,
                    stream=None):
    """The next version of a block table: slot i goes on from slot
    ``parents[i]`` of ``block_table`` [S,max_pages] (int32; -1: an empty slot; old
    slots that nobody names are freed), with pages for ``new_tokens[i]`` more
    tokens.  Full pages are shared, the pages that the slot's next rows go to are
    its own: taken from the free ones (``refcount`` [P] is 0) and, where tokens
    are in them already, copied in every one of ``pools``.

    Returns (block_table [N,max_pages], seqlens [N], refcount [P], status [4]),
    new tensors; status: pages that were missing, slots that do not fit
    max_pages, pages taken, pages copied.  Where one of the first two is not 0,
    nothing was copied, the new table is empty and the old version still stands."""
    lib = load_library()
    dev = block_table.device
    S, M = block_table.shape
    P, N = refcount.numel(), parents.numel()
    _check_tensor("block_table", block_table, torch.int32, S * M, dev)
    _check_tensor("seqlens", seqlens, torch.int32, S, dev)
    _check_tensor("refcount", refcount, torch.int32, P, dev)
    _check_tensor("parents", parents, torch.int32, N, dev)
    if new_tokens is not None:
        _check_tensor("new_tokens", new_tokens, torch.int32, N, dev)
    ptrs, sizes, npools = _pool_arrays(pools, P, dev, "pools")
    with _Launch(dev, stream) as st:
        table_out = torch.empty((N, M), dtype=torch.int32, device=dev)
        lens_out = torch.empty((N,), dtype=torch.int32, device=dev)
        refs_out = torch.empty((P,), dtype=torch.int32, device=dev)
        status = torch.empty((4,), dtype=torch.int32, device=dev)
        _check(lib.attn_pages_fork(ptrs, sizes, npools, _ptr(block_table), _ptr(seqlens),
                                   _ptr(refcount), S, M, P, int(page_size), _ptr(parents),
                                   _ptr(new_tokens), N, _ptr(table_out), _ptr(lens_out),
                                   _ptr(refs_out), _ptr(status), st))
    return table_out, lens_out, refs_out, status


def attn_pages_compact(pools, block_table, refcount, *, stream=None):
    """Moves the live pages (``refcount`` [P] int32 > 0) to the front of every
    pool, in place, and renumbers them: returns (block_table, refcount, remap
    [P], n_live []), new tensors; remap: a live page's new number, -1 for a free
    one."""
    lib = load_library()
    dev = block_table.device
    S, M = block_table.shape
    P = refcount.numel()
    _check_tensor("block_table", block_table, torch.int32, S * M, dev)
    _check_tensor("refcount", refcount, torch.int32, P, dev)
    ptrs, sizes, npools = _pool_arrays(pools, P, dev, "pools")
    with _Launch(dev, stream) as st:
        table_out = torch.empty((S, M), dtype=torch.int32, device=dev)
        refs_out = torch.empty((P,), dtype=torch.int32, device=dev)
        remap = torch.empty((P,), dtype=torch.int32, device=dev)
        n_live = torch.empty((), dtype=torch.int32, device=dev)
        _check(lib.attn_pages_compact(ptrs, sizes, npools, _ptr(block_table), _ptr(refcount), S, M,
                                      P, _ptr(table_out), _ptr(refs_out), _ptr(remap),
                                      _ptr(n_live), st))
    return table_out, refs_out, remap, n_live
