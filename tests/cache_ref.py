"""Plain restatement (numpy, 64 bits) of the 8-bit paged cache for the tests:
codes and scales, appending rows, the next version of a block table, and
compaction -- one element, slot or page at a time, as the definitions read."""
import math

import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
TORCH_CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def e4m3_values():
    """Values of the codes 0..255 (the NaN codes 127 and 255 as NaN)."""
    v = np.empty(256)
    for c in range(128):
        e, m = c >> 3, c & 7
        v[c] = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    v[127] = math.nan
    v[128:] = -v[:128]
    return v


E4M3 = e4m3_values()


def code_values(codes, kind):
    """Values of an array of uint8 bit patterns."""
    return codes.view(np.int8).astype(np.float64) if kind == "int8" else E4M3[codes]


def round_codes(y, kind):
    """uint8 bit patterns of round-to-nearest-even(y); NaN and infinities give 0."""
    y = np.where(np.isfinite(y), y, 0.0)
    if kind == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    mags = E4M3[:127]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(mags, a), 0, 126)  # mags[hi] >= a
    lo = np.clip(hi - 1, 0, 126)
    dh, dl = mags[hi] - a, a - mags[lo]
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(a >= mags[126], 126, pick)
    return (pick | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def scale_for(a, kind):
    """The smallest 2^e >= 2^-100 with a <= qmax * 2^e; NaN for a non-finite a."""
    if not np.isfinite(a):
        return math.nan
    e = -100
    while a > QMAX[kind] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(rows, lens, new, table, codes, scales, kind):
    """rows: list of [n, Hkv, D] arrays (one a sequence) written behind lens[b]
    rows; codes uint8 [P, page, Hkv, D] and scales [P, nblk, Hkv] (float64) in
    place."""
    P, page, Hkv, D = codes.shape
    blk = page // scales.shape[1]
    M = table.shape[1]
    for b, x in enumerate(rows):
        pos, end = int(lens[b]), min(int(lens[b]) + int(new[b]), M * page)
        while pos < end:
            start = pos // blk * blk
            stop = min(end, start + blk)
            pg = int(table[b, start // page])
            if 0 <= pg < P:
                r0, sub = start % page, start % page // blk
                for h in range(Hkv):
                    v = x[pos - lens[b]: stop - lens[b], h].astype(np.float64)
                    s = scale_for(np.max(np.abs(v)) if not np.isnan(v).any() else math.nan, kind)
                    if start < pos:
                        old = scales[pg, sub, h]
                        s = math.nan if math.isnan(old) or math.isnan(s) else max(old, s)
                        if not s == old:
                            held = codes[pg, r0: r0 + pos - start, h]
                            held[...] = round_codes(code_values(held, kind) * (old / s), kind)
                    scales[pg, sub, h] = s
                    with np.errstate(invalid="ignore"):
                        codes[pg, pos % page: pos % page + stop - pos, h] = round_codes(v / s, kind)
            pos = stop


def as_values(codes, scales, kind):
    """[P, page, Hkv, D] float64 of codes (uint8) and scales."""
    P, page, Hkv, D = codes.shape
    nb = scales.shape[1]
    v = code_values(codes, kind).reshape(P, nb, page // nb, Hkv, D)
    return (v * scales.astype(np.float64)[:, :, None, :, None]).reshape(P, page, Hkv, D)


def gather(values, table, lens, K):
    """[B, K, H, D] keys or values of sequences laid out in pages (zeros past lens)."""
    page = values.shape[1]
    out = np.zeros((table.shape[0], K) + values.shape[2:])
    for b in range(table.shape[0]):
        for j in range(min(int(lens[b]), K)):
            pg = min(max(int(table[b, j // page]), 0), values.shape[0] - 1)
            out[b, j] = values[pg, j % page]
    return out


def fork(table, lens, refs, parents, new, page):
    """(table, lens, refs, status, copies) of the next version; copies: (src, dst)."""
    S, M = table.shape
    P, N = len(refs), len(parents)
    ok = lambda c: 0 <= c < P  # noqa: E731
    was = np.zeros(P, int)
    for c in table.reshape(-1):
        if ok(c):
            was[c] += 1
    slots = []
    for i in range(N):
        p = int(parents[i])
        if not 0 <= p < S:
            slots.append(None)
            continue
        n = min(max(int(lens[p]), 0), M * page)
        slots.append((p, n, -(-(n + max(int(new[i]), 0)) // page)))
    full = {int(table[p, j]) for s in slots if s for p, n, _ in [s] for j in range(n // page)}
    owner = {}
    for i, s in enumerate(slots):
        if s:
            for j in range(s[1] // page, min(s[2], M)):
                owner.setdefault(int(table[s[0], j]), (i, j))
    out = np.full((N, M), -1, np.int32)
    free = [p for p in range(P) if refs[p] == 0]
    taken, copies, need = [], [], 0
    for i, s in enumerate(slots):
        if not s:
            continue
        p, n, want = s
        for j in range(min(want, M)):
            c = int(table[p, j])
            if j < n // page:
                out[i, j] = c if ok(c) else -1
                continue
            if ok(c) and refs[c] > 0 and c not in full and refs[c] <= was[c] and owner[c] == (i, j):
                out[i, j] = c
                continue
            if need < len(free):
                out[i, j] = free[need]
                if ok(c) and j == n // page and n % page:
                    copies.append((c, free[need]))
            need += 1
    wide = sum(1 for s in slots if s and s[2] > M)
    missing = max(0, need - len(free))
    if wide or missing:
        return (np.full((N, M), -1, np.int32), np.zeros(N, np.int32), refs.copy(),
                np.array([missing, wide, 0, 0], np.int32), [])
    left = refs - was
    for c in out.reshape(-1):
        if ok(c):
            left[c] += 1
    lens_out = np.array([s[1] if s else 0 for s in slots], np.int32)
    return out, lens_out, left.astype(np.int32), np.array([0, 0, need, len(copies)], np.int32), copies


def compact(table, refs):
    """(table, refs, remap, n, moves)."""
    P = len(refs)
    n = int(np.sum(refs > 0))
    holes = [p for p in range(n) if refs[p] <= 0]
    movers = [p for p in range(n, P) if refs[p] > 0]
    remap = np.array([p if refs[p] > 0 else -1 for p in range(P)], np.int32)
    for s, d in zip(movers, holes):
        remap[s] = d
    left = np.zeros(P, np.int32)
    for p in range(P):
        if refs[p] > 0:
            left[remap[p]] = refs[p]
    out = np.full(table.shape, -1, np.int32)
    for i in np.ndindex(table.shape):
        if 0 <= table[i] < P:
            out[i] = remap[table[i]]
    return out, left, remap, n, list(zip(movers, holes))
