"""The position rotation: of queries and keys and of their gradients
(``attn_rope``, ``attn_rope_bwd``), and of the rows of a serving step on their way
into a paged cache (``attn_rope_append``: the pages of ``attn_fwd_paged``;
``attn_rope_append_q8``: the 8-bit cache of ``attn_fwd_paged_q8``).

``cos`` and ``sin`` are float32 [positions, rot / 2]: the first ``rot`` columns of a
head are rotated, as pairs of columns i and i + rot / 2 (``pairs="half"``) or 2 i and
2 i + 1 (``"adjacent"``).  A training step::

    q, k = attn_rope(q, k, cos, sin)
    o, lse = attn_fwd(q, k, v)
    dq, dk, dv = attn_bwd(q, k, v, o, lse, dout)
    dq, dk = attn_rope_bwd(dq, dk, cos, sin)

A decoding step over pages that hold ``lens`` rows a sequence::

    q = attn_rope_append(q, k, v, cos, sin, k_pages, v_pages, table, lens)
    o, lse = attn_fwd_paged(q, k_pages, v_pages, table, lens + 1)

q, k and v may be views whose rows of heads are equally spaced (the parts of a fused
projection).  As the rest of the package this is argument marshalling only.
"""
from __future__ import annotations

import torch

from .binding import _DTYPE_CODE, _check, load_library
from .cache import _cache, _elsewhere, _here, _raw_stream, _tensor

PAIRS = {"half": 0, "adjacent": 1}


def _rows(name, x, shape, dtype, i):
    """Checks a tensor of rows [.., H, D] whose rows of heads are equally spaced;
    returns its address and that spacing in elements."""
    if x.dtype is not dtype:
        raise TypeError(f"{name}: dtype {x.dtype}, expected {dtype}")
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.get_device() != i:
        raise ValueError(f"{name} is on {x.device}, unlike the other tensors")
    H, D = shape[-2:]
    if x.is_contiguous():
        return x.data_ptr(), H * D
    s = x.stride()
    if (D > 1 and s[-1] != 1) or (H > 1 and s[-2] != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous (strides {s})")
    row = H * D
    if len(shape) == 3:
        row = s[0] if shape[0] > 1 else row
    elif shape[1] > 1:
        row = s[1]
        if shape[0] > 1 and s[0] != shape[1] * row:
            raise ValueError(f"{name}: rows must be equally spaced (strides {s})")
    elif shape[0] > 1:
        row = s[0]
    return x.data_ptr(), row


def _angles(cos, sin, i):
    """Checks a table of angles; returns (cos, sin, positions, rotated columns)."""
    if cos is None and sin is None:
        return None, None, 0, 0
    if cos is None or sin is None or cos.dim() != 2:
        raise ValueError("cos and sin are [positions, rot / 2], or both None")
    P, half = cos.shape
    return (_tensor("cos", cos, torch.float32, (P, half), i),
            _tensor("sin", sin, torch.float32, (P, half), i), P, 2 * half)


def _dtype(name, x):
    code = _DTYPE_CODE.get(x.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {x.dtype}, expected float32, float16 or bfloat16")
    return code


def _rope(q, k, cos, sin, q_out, k_out, positions, pairs, stream, inverse):
    i = q.get_device()
    if q.dim() not in (3, 4):
        raise ValueError(f"q: shape {tuple(q.shape)}, expected [B, N, Hq, D] or [N, Hq, D]")
    lead, (Hq, D) = tuple(q.shape[:-2]), q.shape[-2:]
    dtype = _dtype("q", q)
    if PAIRS.get(pairs) is None:
        raise ValueError(f"pairs: {pairs!r}, expected one of {sorted(PAIRS)}")
    qx, qs = _rows("q", q, q.shape, q.dtype, i)
    kx, ks, Hkv = None, 0, 0
    if k is not None:
        if k.dim() != q.dim():
            raise ValueError(f"k: shape {tuple(k.shape)}, expected {lead + ('Hkv', D)}")
        Hkv = k.shape[-2]
        kx, ks = _rows("k", k, lead + (Hkv, D), q.dtype, i)
    elif k_out is not None:
        raise ValueError("k_out without k")
    cx, sx, P, rot = _angles(cos, sin, i)
    px = None if positions is None else _tensor("positions", positions, torch.int32, lead, i)
    if not _here(i, stream):
        with _elsewhere(q, stream):
            return _rope(q, k, cos, sin, q_out, k_out, positions, pairs, None, inverse)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    ox = _tensor("q_out", q_out, q.dtype, q.shape, i)
    kox = None
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        kox = _tensor("k_out", k_out, q.dtype, k.shape, i)
    B, N = lead if len(lead) == 2 else (1, lead[0])
    if q.numel() + (k.numel() if k is not None else 0):
        _check(load_library().attn_rope(qx, kx, ox, kox, cx, sx, B, N, Hq, Hkv, D, rot, P, qs, ks,
                                        px, PAIRS[pairs], inverse, dtype, _raw_stream(i)))
    return q_out, k_out


def attn_rope(q, k, cos, sin, q_out=None, k_out=None, *, positions=None, pairs="half",
              stream=None):
    """Rotates q [B,N,Hq,D] and k [B,N,Hkv,D] (fp32, fp16 or bf16; or [N,H,D]; k may
    be None) by position: row i of a sequence is at position i, or at
    ``positions`` int32 [B,N] (outside the table: NaN).  ``q_out`` and ``k_out``
    may be contiguous q and k themselves.  Returns (q_out, k_out)."""
    return _rope(q, k, cos, sin, q_out, k_out, positions, pairs, stream, 0)


def attn_rope_bwd(dq, dk, cos, sin, dq_out=None, dk_out=None, *, positions=None, pairs="half",
                  stream=None):
    """Gradients of attn_rope's inputs for the gradients dq [B,N,Hq,D] and dk
    [B,N,Hkv,D] of its outputs, with the same angles, positions and pairs."""
    return _rope(dq, dk, cos, sin, dq_out, dk_out, positions, pairs, stream, 1)


def _append(q, k, v, cu, max_new, cos, sin, sizes, addresses, q_out, new, positions, pairs,
            stream, code):
    """The call behind the four appends.  sizes and addresses: what the checks of the
    cache gave; cu None: padded rows."""
    i = k.get_device()
    kp, vp, ks, vs, table, lens = addresses = tuple(addresses)
    P, page, block, Hkv, D, Dv, B, M = sizes
    dtype = _dtype("k", k)
    packed = cu is not None
    if k.dim() != (3 if packed else 4) or (not packed and k.shape[0] != B):
        raise ValueError(f"k: shape {tuple(k.shape)}, expected "
                         f"{'[T' if packed else f'[{B}, N'}, {Hkv}, {D}]")
    lead = tuple(k.shape[:-2])
    if PAIRS.get(pairs) is None:
        raise ValueError(f"pairs: {pairs!r}, expected one of {sorted(PAIRS)}")
    kx, kst = _rows("k", k, lead + (Hkv, D), k.dtype, i)
    vx, vst = _rows("v", v, lead + (Hkv, Dv), k.dtype, i)
    qx, qst, Hq, ox = None, 0, 0, None
    if q is not None:
        if q.dim() != k.dim():
            raise ValueError(f"q: shape {tuple(q.shape)}, expected {lead + ('Hq', D)}")
        Hq = q.shape[-2]
        qx, qst = _rows("q", q, lead + (Hq, D), k.dtype, i)
    cx, sx, npos, rot = _angles(cos, sin, i)
    px = None if positions is None else _tensor("positions", positions, torch.int32, lead, i)
    nx = None if new is None else _tensor("seqlens_new", new, torch.int32, (B,), i)
    cux = None if cu is None else _tensor("cu_seqlens_new", cu, torch.int32, (B + 1,), i)
    if not _here(i, stream):
        with _elsewhere(k, stream):
            return _append(q, k, v, cu, max_new, cos, sin, sizes, addresses, q_out, new, positions,
                           pairs, None, code)
    N, total = (int(max_new), lead[0]) if packed else (lead[1], 0)
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ox = _tensor("q_out", q_out, q.dtype, q.shape, i)
        if q.numel() == 0:
            qx = ox = None
            Hq = 0
    elif q_out is not None:
        raise ValueError("q_out without q")
    lib, at = load_library(), _raw_stream(i)
    rows = (cx, sx, B, N, total, Hq, Hkv, D, Dv, rot, npos, qst, kst, vst, nx, cux, px,
            PAIRS[pairs], lens, table, M, page, P)
    if code is None:
        _check(lib.attn_rope_append(qx, kx, vx, ox, kp, vp, *rows, dtype, at))
    else:
        _check(lib.attn_rope_append_q8(qx, kx, vx, ox, kp, vp, ks, vs, *rows, block, code, dtype, at))
    return q_out


def _pages(k, k_pages, v_pages, block_table, seqlens_k):
    """Checks 16- or 32-bit pages as attn_cache's are checked: (addresses, sizes)."""
    i = k.get_device()
    if k_pages.dim() != 4 or v_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("pages are [P, page, Hkv, D] and the block table [B, max_pages]")
    P, page, Hkv, D = k_pages.shape
    Dv = v_pages.shape[3]
    B, M = block_table.shape
    return (_tensor("k_pages", k_pages, k.dtype, (P, page, Hkv, D), i),
            _tensor("v_pages", v_pages, k.dtype, (P, page, Hkv, Dv), i), None, None,
            _tensor("block_table", block_table, torch.int32, (B, M), i),
            _tensor("seqlens_k", seqlens_k, torch.int32, (B,), i)), (P, page, 0, Hkv, D, Dv, B, M)


def attn_rope_append(q, k, v, cos, sin, k_pages, v_pages, block_table, seqlens_k, q_out=None, *,
                     seqlens_new=None, positions=None, pairs="half", stream=None):
    """Rotates q [B,N,Hq,D] (or None) and k [B,N,Hkv,D], and writes k and v
    [B,N,Hkv,Dv] into pages of their type behind the ``seqlens_k`` rows each
    sequence has; ``seqlens_new`` int32 [B]: how many of the N are there (default:
    all).  Row i's position is ``seqlens_k + i``, or ``positions`` int32 [B,N]; cos
    and sin None: no rotation.  The pages that rows go to are in ``block_table``
    already; ``seqlens_k`` is not changed.  Returns the rotated q (``q_out``, which
    may be a contiguous q itself; +0 in rows past ``seqlens_new``)."""
    at, sizes = _pages(k, k_pages, v_pages, block_table, seqlens_k)
    return _append(q, k, v, None, 0, cos, sin, sizes, at, q_out, seqlens_new, positions,
                   pairs, stream, None)


def attn_rope_append_varlen(q, k, v, cu_seqlens_new, max_new, cos, sin, k_pages, v_pages,
                            block_table, seqlens_k, q_out=None, *, positions=None, pairs="half",
                            stream=None):
    """attn_rope_append with the new rows packed: q [T,Hq,D], k [T,Hkv,D], v
    [T,Hkv,Dv], sequence b's rows [cu_seqlens_new[b], cu_seqlens_new[b + 1]), at
    most ``max_new`` of them.  Rows of ``q_out`` outside every sequence are not
    written."""
    at, sizes = _pages(k, k_pages, v_pages, block_table, seqlens_k)
    return _append(q, k, v, cu_seqlens_new, max_new, cos, sin, sizes, at, q_out, None,
                   positions, pairs, stream, None)


def attn_rope_append_q8(q, k, v, cos, sin, k_pages, v_pages, k_scale, v_scale, block_table,
                        seqlens_k, q_out=None, *, seqlens_new=None, positions=None, pairs="half",
                        stream=None):
    """attn_rope_append into an 8-bit cache (scales and codes as attn_cache_append
    writes them, of the rotated keys in fp32)."""
    at, sizes, code = _cache(k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, k.get_device())
    return _append(q, k, v, None, 0, cos, sin, sizes, at, q_out, seqlens_new, positions,
                   pairs, stream, code)


def attn_rope_append_q8_varlen(q, k, v, cu_seqlens_new, max_new, cos, sin, k_pages, v_pages,
                               k_scale, v_scale, block_table, seqlens_k, q_out=None, *,
                               positions=None, pairs="half", stream=None):
    """attn_rope_append_q8 with the new rows packed, as attn_rope_append_varlen."""
    at, sizes, code = _cache(k_pages, v_pages, k_scale, v_scale, block_table, seqlens_k, k.get_device())
    return _append(q, k, v, cu_seqlens_new, max_new, cos, sin, sizes, at, q_out, None,
                   positions, pairs, stream, code)
