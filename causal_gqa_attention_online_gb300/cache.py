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

import array
import math
import operator

import torch

from .binding import _DTYPE_CODE, ALGOS, MASKS, _check, _check_tensor, load_library

ATTN_CACHE_E4M3, ATTN_CACHE_INT8 = 0, 1
_CACHE_CODE = {torch.float8_e4m3fn: ATTN_CACHE_E4M3, torch.int8: ATTN_CACHE_INT8}


def _public_stream(i):
    return torch.cuda.current_stream(i).cuda_stream


def _public_device():
    return torch.cuda.current_device()


# The handle of device i's current stream and the current device: what the functions
# above give, without their objects and checks (0.2 us against 4 a call) where torch has
# what it takes (a build without CUDA has not).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", _public_device)

# Checks of many tensors go through these (half the time of a loop's method calls).
_is_contiguous, _get_device = torch.Tensor.is_contiguous, torch.Tensor.get_device
_data_ptr, _nbytes = torch.Tensor.data_ptr, operator.attrgetter("nbytes")


def _here(i, stream):
    """Whether a call on device ``i`` can go to the current stream as it is.
    (Otherwise the entry points call themselves with ``_elsewhere`` in force.)"""
    return stream is None and i >= 0 and i == _current_device()


def _elsewhere(t, stream):
    """Makes t's device and ``stream`` current: the library works on the current
    device, and outputs that a call allocates belong to its stream."""
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"the tensors are on {dev}: the library runs on CUDA devices only")
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _tensor(name, t, dtype, shape, i):
    """Checks one tensor (of device ``i``, -1: the CPU); returns its address."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == i:
        return t.data_ptr()
    n = 1
    for x in shape:
        n *= x
    _check_tensor(name, t, dtype, n, torch.device("cuda", i) if i >= 0 else torch.device("cpu"))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _cache(k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, i):
    """Checks a cache; returns its addresses (k_pages, v_pages, k_scale,
    v_scale, block_table, seqlens_k), sizes (P, page, block, Hkv, D, Dv, B,
    max_pages) and code."""
    code = _CACHE_CODE.get(k_pages.dtype)
    if code is None:
        raise TypeError(f"k_pages: dtype {k_pages.dtype}, expected torch.int8 or "
                        "torch.float8_e4m3fn")
    if k_pages.dim() != 4 or v_pages.dim() != 4 or k_scale.dim() != 3 or block_table.dim() != 2:
        raise ValueError("pages are [P, page, Hkv, D], scales [P, page / block, Hkv] and the "
                         "block table [B, max_pages]")
    pages, scales = k_pages.shape, k_scale.shape
    P, page, Hkv, D = pages
    Dv, nblk = v_pages.size(3), scales[1]
    B, M = block_table.shape
    if nblk < 1 or page % nblk:
        raise ValueError(f"k_scale: {nblk} blocks do not divide a page of {page} tokens")
    tensors = (k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k)
    if not (all(map(_is_contiguous, tensors)) and all(map(i.__eq__, map(_get_device, tensors))) and
            v_pages.dtype is k_pages.dtype and k_scale.dtype is torch.float32 and
            v_scale.dtype is torch.float32 and block_table.dtype is torch.int32 and
            seqlens_k.dtype is torch.int32 and (Dv == D or v_pages.shape[:3] == pages[:3]) and
            (Dv != D or v_pages.shape == pages) and scales == (P, nblk, Hkv) and
            v_scale.shape == scales and seqlens_k.shape == (B,)):
        for name, t, dtype, shape in (
                ("k_pages", k_pages, k_pages.dtype, (P, page, Hkv, D)),
                ("v_pages", v_pages, k_pages.dtype, (P, page, Hkv, Dv)),
                ("k_scale", k_scale, torch.float32, (P, nblk, Hkv)),
                ("v_scale", v_scale, torch.float32, (P, nblk, Hkv)),
                ("block_table", block_table, torch.int32, (B, M)),
                ("seqlens_k", seqlens_k, torch.int32, (B,))):
            _tensor(name, t, dtype, shape, i)
    return map(_data_ptr, tensors), (P, page, page // nblk, Hkv, D, Dv, B, M), code


def attn_cache_append(k, v, k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, *,
                      seqlens_new=None, stream=None):
    """Writes new rows k [B,N,Hkv,D], v [B,N,Hkv,Dv] (fp32, fp16 or bf16) into
    the cache behind the ``seqlens_k`` rows each sequence has; ``seqlens_new``
    int32 [B]: how many of the N are there (default: all).  The pages they go to
    are in ``block_table`` already.  ``seqlens_k`` is not changed."""
    i = k.get_device()
    (kp, vp, ks, vs, table, lens), (P, page, block, Hkv, D, Dv, B, M), code = _cache(
        k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, i)
    if k.dim() != 4 or k.shape[0] != B or k.shape[2:] != (Hkv, D):
        raise ValueError(f"k: shape {tuple(k.shape)}, expected [{B}, N, {Hkv}, {D}]")
    dtype = _DTYPE_CODE.get(k.dtype)
    if dtype is None:
        raise TypeError(f"k: dtype {k.dtype}, expected float32, float16 or bfloat16")
    N = k.shape[1]
    kx = _tensor("k", k, k.dtype, (B, N, Hkv, D), i)
    vx = _tensor("v", v, k.dtype, (B, N, Hkv, Dv), i)
    new = None
    if seqlens_new is not None:
        new = _tensor("seqlens_new", seqlens_new, torch.int32, (B,), i)
    if not _here(i, stream):
        with _elsewhere(k, stream):
            return attn_cache_append(k, v, k_pages, v_pages, k_scale, v_scale, block_table,
                                     seqlens_k, seqlens_new=seqlens_new)
    _check(load_library().attn_cache_append(kx, vx, kp, vp, ks, vs, B, N, Hkv, D, Dv, new, lens,
                                            table, M, page, P, block, code, dtype,
                                            _raw_stream(i)))


def attn_cache_append_varlen(k, v, cu_seqlens_new, max_new, k_pages, v_pages, k_scale, v_scale,
                             block_table, seqlens_k, *, stream=None):
    """attn_cache_append with the new rows packed: k [T,Hkv,D], v [T,Hkv,Dv],
    sequence b's rows [cu_seqlens_new[b], cu_seqlens_new[b + 1]), at most
    ``max_new`` of them."""
    i = k.get_device()
    (kp, vp, ks, vs, table, lens), (P, page, block, Hkv, D, Dv, B, M), code = _cache(
        k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, i)
    if k.dim() != 3 or k.shape[1:] != (Hkv, D):
        raise ValueError(f"k: shape {tuple(k.shape)}, expected [T, {Hkv}, {D}]")
    dtype = _DTYPE_CODE.get(k.dtype)
    if dtype is None:
        raise TypeError(f"k: dtype {k.dtype}, expected float32, float16 or bfloat16")
    T = k.shape[0]
    kx = _tensor("k", k, k.dtype, (T, Hkv, D), i)
    vx = _tensor("v", v, k.dtype, (T, Hkv, Dv), i)
    cu = _tensor("cu_seqlens_new", cu_seqlens_new, torch.int32, (B + 1,), i)
    if not _here(i, stream):
        with _elsewhere(k, stream):
            return attn_cache_append_varlen(k, v, cu_seqlens_new, max_new, k_pages, v_pages,
                                            k_scale, v_scale, block_table, seqlens_k)
    _check(load_library().attn_cache_append_varlen(kx, vx, kp, vp, ks, vs, B, T, int(max_new), Hkv,
                                                   D, Dv, cu, lens, table, M, page, P, block, code,
                                                   dtype, _raw_stream(i)))


def attn_fwd_paged_q8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, o=None,
                      lse=None, *, seqlens_q=None, window=0, scale=None, algo="auto",
                      mask="causal", stream=None, want_lse=True):
    """attn_fwd_paged over an 8-bit cache: q [B,Q,Hq,D]; ``seqlens_k`` counts the
    keys to attend to (append first).  Returns (o [B,Q,Hq,Dv], lse [B,Q,Hq] or
    None)."""
    i = q.get_device()
    (kp, vp, ks, vs, table, lens), (P, page, block, Hkv, D, Dv, B, M), code = _cache(
        k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, i)
    if q.dim() != 4 or q.shape[0] != B or q.shape[3] != D:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [{B}, Q, Hq, {D}]")
    dtype = _DTYPE_CODE.get(q.dtype)
    if dtype is None:
        raise TypeError(f"q: dtype {q.dtype}, expected float32, float16 or bfloat16")
    Q, Hq = q.shape[1], q.shape[2]
    if not _here(i, stream):
        with _elsewhere(q, stream):
            return attn_fwd_paged_q8(q, k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k,
                                     o, lse, seqlens_q=seqlens_q, window=window, scale=scale,
                                     algo=algo, mask=mask, want_lse=want_lse)
    qx = _tensor("q", q, q.dtype, (B, Q, Hq, D), i)
    if o is None:
        o = (torch.empty_like(q) if D == Dv else
             torch.empty((B, Q, Hq, Dv), dtype=q.dtype, device=q.device))
    if lse is None and want_lse:
        lse = torch.empty((B, Q, Hq), dtype=torch.float32, device=q.device)
    ox = _tensor("o", o, q.dtype, (B, Q, Hq, Dv), i)
    lx = None if lse is None else _tensor("lse", lse, torch.float32, (B, Q, Hq), i)
    sq = None if seqlens_q is None else _tensor("seqlens_q", seqlens_q, torch.int32, (B,), i)
    _check(load_library().attn_fwd_paged_q8(
        qx, kp, vp, ks, vs, ox, lx, B, Hq, Hkv, Q, D, Dv, table, M, page, P, block, code, sq, lens,
        int(window), 1.0 / math.sqrt(D) if scale is None else float(scale), MASKS[mask], dtype,
        ALGOS[algo], _raw_stream(i)))
    return o, lse


def _pool_arrays(pools, pages, i, what):
    """Pointers and page bytes of pools (of device ``i``) whose first axis counts
    ``pages`` pages, as 64-bit arrays."""
    if not (all(map(_is_contiguous, pools)) and all(map(i.__eq__, map(_get_device, pools))) and
            all(map((pages,).__eq__, [t.shape[:1] for t in pools]))):
        for k, t in enumerate(pools):
            if t.dim() < 1 or t.shape[0] != pages:
                raise ValueError(f"{what}[{k}]: shape {tuple(t.shape)}, expected {pages} pages "
                                 "first")
            if not t.is_contiguous():
                raise ValueError(f"{what}[{k}] must be contiguous")
            if t.get_device() != i:
                raise ValueError(f"{what}[{k}] is on {t.device}, unlike the tables")
    sizes = array.array("q", map(_nbytes, pools))
    if pages > 1:
        sizes = array.array("q", [x // pages for x in sizes])
    return array.array("Q", map(_data_ptr, pools)), sizes


def _at(a):
    """The address of an array's first element (it lives as long as the array)."""
    return a.buffer_info()[0]


def attn_pages_copy(src_pools, dst_pools, src, dst, *, stream=None):
    """Copies page ``src[i]`` of each of ``src_pools`` to page ``dst[i]`` of the
    pool at the same place of ``dst_pools`` (the same list to copy within it).
    ``src``, ``dst``: int32 [n]; the dst pages are distinct, and none of them is
    a src page of the same pool.  Pairs with a page that does not exist are
    skipped."""
    i = src.get_device()
    if len(src_pools) != len(dst_pools):
        raise ValueError(f"{len(src_pools)} source pools and {len(dst_pools)} destinations")
    n = src.numel()
    sx = _tensor("src", src, torch.int32, (n,), i)
    dx = _tensor("dst", dst, torch.int32, (n,), i)
    sp = src_pools[0].shape[0] if len(src_pools) else 0
    dp = dst_pools[0].shape[0] if len(dst_pools) else 0
    sptr, sbytes = _pool_arrays(src_pools, sp, i, "src_pools")
    if dst_pools is src_pools:
        dptr = sptr
    else:
        dptr, dbytes = _pool_arrays(dst_pools, dp, i, "dst_pools")
        if sbytes != dbytes:
            raise ValueError("the pages of a source pool and of its destination differ in size")
    if not _here(i, stream):
        with _elsewhere(src, stream):
            return attn_pages_copy(src_pools, dst_pools, src, dst)
    _check(load_library().attn_pages_copy(_at(sptr), _at(dptr), _at(sbytes), len(sptr), sp, dp, sx,
                                          dx, n, _raw_stream(i)))


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
    i = block_table.get_device()
    S, M = block_table.shape
    P, N = refcount.numel(), parents.numel()
    tx = _tensor("block_table", block_table, torch.int32, (S, M), i)
    lx = _tensor("seqlens", seqlens, torch.int32, (S,), i)
    rx = _tensor("refcount", refcount, torch.int32, (P,), i)
    px = _tensor("parents", parents, torch.int32, (N,), i)
    nx = None if new_tokens is None else _tensor("new_tokens", new_tokens, torch.int32, (N,), i)
    ptrs, sizes = _pool_arrays(pools, P, i, "pools")
    if not _here(i, stream):
        with _elsewhere(block_table, stream):
            return attn_pages_fork(pools, block_table, seqlens, refcount, parents, page_size,
                                   new_tokens=new_tokens)
    # one allocation: the new version's table, lengths, counts, and the status
    out = torch.empty((N * M + N + P + 4,), dtype=torch.int32, device=block_table.device)
    at, l0, r0, s0 = out.data_ptr(), N * M, N * M + N, N * M + N + P
    _check(load_library().attn_pages_fork(
        _at(ptrs), _at(sizes), len(ptrs), tx, lx, rx, S, M, P, int(page_size), px, nx, N, at,
        at + 4 * l0, at + 4 * r0, at + 4 * s0, _raw_stream(i)))
    table_out, lens_out, refs_out, status = out.split_with_sizes((l0, N, P, 4))
    return table_out.view(N, M), lens_out, refs_out, status


def attn_pages_compact(pools, block_table, refcount, *, stream=None):
    """Moves the live pages (``refcount`` [P] int32 > 0) to the front of every
    pool, in place, and renumbers them: returns (block_table, refcount, remap
    [P], n_live []), new tensors; remap: a live page's new number, -1 for a free
    one."""
    i = block_table.get_device()
    S, M = block_table.shape
    P = refcount.numel()
    tx = _tensor("block_table", block_table, torch.int32, (S, M), i)
    rx = _tensor("refcount", refcount, torch.int32, (P,), i)
    ptrs, sizes = _pool_arrays(pools, P, i, "pools")
    if not _here(i, stream):
        with _elsewhere(block_table, stream):
            return attn_pages_compact(pools, block_table, refcount)
    out = torch.empty((S * M + 2 * P + 1,), dtype=torch.int32, device=block_table.device)
    at, r0, m0, n0 = out.data_ptr(), S * M, S * M + P, S * M + 2 * P
    _check(load_library().attn_pages_compact(
        _at(ptrs), _at(sizes), len(ptrs), tx, rx, S, M, P, at, at + 4 * r0, at + 4 * m0,
        at + 4 * n0, _raw_stream(i)))
    table_out, refs_out, remap, n_live = out.split_with_sizes((r0, P, P, 1))
    return table_out.view(S, M), refs_out, remap, n_live.view(())
