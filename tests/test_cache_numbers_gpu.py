"""Attention over the 8-bit cache where its numbers are at their ends -- value
scales of any size, scales and codes that are no numbers -- on every path of the
kernel that reads the codes, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn
from tests import cache_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}      # half a step of the type, relative
LEAST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}   # half of its smallest step
PAGE, D = 64, 64

# one cluster a sequence and head; shares of a long sequence that a merge joins; many
# sequences a share, whole and cut; the same with row groups of 16
PATHS = {
    "cluster": dict(lens=[500, 129], Q=1, Hq=4, Hkv=2),
    "merge": dict(lens=[20000, 300], Q=1, Hq=4, Hkv=2),
    "whole": dict(lens=[700, 0, 65] + [100 + 9 * i for i in range(57)], Q=1, Hq=8, Hkv=4),
    "groups": dict(lens=[500, 129], Q=12, Hq=4, Hkv=2),
    "groups merge": dict(lens=[9000, 77], Q=12, Hq=4, Hkv=2),
}


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Problem:
    """Random codes in shuffled pages, scales that a test may change, random queries."""

    def __init__(self, g, path, block=32, kind="int8", dtype="bf16", window=0, **more):
        self.__dict__.update({**PATHS[path], **more})
        self.kind, self.dtype, self.window, self.block = kind, dtype, window, block
        need = [-(-n // PAGE) for n in self.lens]
        P = sum(need) + 2
        order = iter(g.permutation(P))
        self.table = np.full((len(self.lens), max(need)), -1, np.int32)
        for b, n in enumerate(need):
            for j in range(n):
                self.table[b, j] = next(order)
        self.codes = [g.integers(0, 256, (P, PAGE, self.Hkv, D), dtype=np.uint8) for _ in "kv"]
        for c in self.codes:
            c[(c == 128) if kind == "int8" else (c & 127) == 127] = 1
        s = 2.0 ** g.integers(-8, -5, (2, P, PAGE // block, self.Hkv))
        self.scales = list((s if kind == "int8" else s / 4).astype(np.float32))
        q = g.standard_normal((len(self.lens), self.Q, self.Hq, D)).astype(np.float32)
        self.q = torch.from_numpy(q).to(DT[dtype])

    def at(self, b, j):
        """Index of key j of sequence b among the pages' rows, and among their blocks."""
        pg = int(self.table[b, j // PAGE])
        return (pg, j % PAGE), (pg, j % PAGE // self.block)

    def run(self, **kw):
        t = cache_ref.TORCH_CODE[self.kind]
        pages = [torch.from_numpy(c.copy()).to(DEV).view(t) for c in self.codes]
        scales = [torch.from_numpy(s.copy()).to(DEV) for s in self.scales]
        kw.setdefault("algo", "decode")
        o, lse = attn.attn_fwd_paged_q8(self.q.to(DEV), *pages, *scales, i32(self.table),
                                        i32(self.lens), window=self.window, **kw)
        torch.cuda.synchronize()
        return o.double().cpu().numpy(), lse.double().cpu().numpy()

    def keys(self, b, i):
        """The keys that row i of sequence b attends to, [lo, hi)."""
        n = self.lens[b]
        hi = max(0, n - self.Q + i + 1)
        return (max(0, hi - self.window) if self.window else 0), hi

    def exact(self):
        """(o, lse, how far o and lse may be off).

        Over the keys a row attends to, with p relative to its largest and w = p times
        the value's scale: a score's fp32 accumulation is off by at most (D + 8) 2^-24 of
        scale * sum |q||k|, which moves p by twice that relative to it; sums over n keys
        are off by n 2^-24 each, ex2 by 2^-22; w is rounded to fp16 under the row's own
        unit, in which its largest is 2^8 or more -- by 2^-11 of itself, or by half of a step
        of 2^-24, which is 2^-33 of the largest -- and to fp32 before that (2^-150 at the
        least); o once at the end."""
        B, Q, Hq, G = len(self.lens), self.Q, self.Hq, self.Hq // self.Hkv
        codes = [cache_ref.code_values(c, self.kind) for c in self.codes]
        q = self.q.double().numpy()
        o = np.zeros((B, Q, Hq, D))
        lse = np.full((B, Q, Hq), -math.inf)
        to, tl = np.zeros(o.shape), np.zeros(lse.shape)
        for b in range(B):
            n = self.lens[b]
            if not n:
                continue
            pg, r = self.table[b, np.arange(n) // PAGE], np.arange(n) % PAGE
            kc, vc = (c[pg, r] for c in codes)
            ks, vs = (s.astype(np.float64)[pg, r // self.block] for s in self.scales)
            for h in range(Hq):
                k, sv, cv = kc[:, h // G] * ks[:, h // G, None], vs[:, h // G], vc[:, h // G]
                for i in range(Q):
                    lo, hi = self.keys(b, i)
                    if lo >= hi:
                        continue
                    s = k[lo:hi] @ q[b, i, h] / math.sqrt(D)
                    big = np.max(np.abs(k[lo:hi]) @ np.abs(q[b, i, h])) / math.sqrt(D)
                    m = s.max()
                    p = np.exp(s - m)
                    w, c = p * sv[lo:hi], cv[lo:hi]
                    total = p.sum()
                    o[b, i, h] = w @ c / total
                    lse[b, i, h] = m + math.log(total)
                    ds = (D + 8) * 2.0 ** -24 * big
                    rel = 2 * ds + 2 * (hi - lo) * 2.0 ** -24 + 2.0 ** -20
                    small = np.abs(c).sum(0) * (2.0 ** -33 * w.max() + 2.0 ** -150)
                    to[b, i, h] = ((2.0 ** -11 + rel) * (w @ np.abs(c)) + small) / total
                    tl[b, i, h] = ds + (hi - lo) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * abs(lse[b, i, h])
        to += HALF[self.dtype] * (np.abs(o) + to) + LEAST[self.dtype]
        return o, lse, to, tl

    def check(self, **kw):
        o, lse = self.run(**kw)
        ro, rl, to, tl = self.exact()
        empty = rl == -math.inf
        assert np.isfinite(o).all() and np.isfinite(lse[~empty]).all()
        assert (o[empty] == 0).all() and (lse[empty] == -math.inf).all()
        eo, el = np.abs(o - ro)[~empty] / to[~empty], np.abs(lse[~empty] - rl[~empty]) / tl[~empty]
        assert eo.max() <= 1, f"o off by {eo.max():.3g} of the bound"
        assert el.max() <= 1, f"lse off by {el.max():.3g} of the bound"
        return o, lse


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("small", [2.0 ** -149, 2.6e-41, 2.0 ** -127, 0.0])
@pytest.mark.parametrize("mixed", [False, True])
def test_value_scales_next_to_zero(path, small, mixed):
    """Scales whose reciprocal is no fp32 number: everywhere, or in the first half of
    each sequence (what every warp meets first) and here and there behind it."""
    g = np.random.default_rng(1)
    x = Problem(g, path)
    for b, n in enumerate(x.lens):
        for j in range(0, n, x.block):
            if not mixed or j < n // 2 or g.random() < 0.3:
                x.scales[1][x.at(b, j)[1]] = small
    x.check()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("which", ["key", "value"])
def test_scales_that_are_no_numbers_poison_the_rows_that_attend(path, bad, which):
    """One block of one head: every row of its heads is not finite, across the merge of
    shares and the joins of a cluster too, and all others have the bits they had."""
    g = np.random.default_rng(2)
    x = Problem(g, path)
    before = x.run()
    x.scales[which == "value"][x.at(0, 40)[1] + (1,)] = bad
    o, lse = x.run()
    G = x.Hq // x.Hkv
    hit = np.zeros(lse.shape, bool)
    hit[0, :, G:2 * G] = True
    assert not np.isfinite(o[hit]).any()
    if which == "value":
        assert np.array_equal(lse[hit], before[1][hit])
    elif math.isnan(bad):
        assert np.isnan(lse[hit]).all()
    assert np.array_equal(o[~hit], before[0][~hit]) and np.array_equal(lse[~hit], before[1][~hit])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("path", PATHS)
def test_value_scales_of_any_spread(path, kind):
    """Blocks of 2^-100 to 2^100 in any order: what a row weighs least does not cost what
    it weighs most its bits."""
    g = np.random.default_rng(3)
    x = Problem(g, path, block=8, kind=kind)
    x.scales[1][...] = 2.0 ** g.integers(-100, 101, x.scales[1].shape)
    x.check()


# rows that end (or begin, under the window) inside a block's last (first) key
RAGGED = {"cluster": dict(lens=[500, 132], Q=4), "merge": dict(lens=[20004, 300], Q=4),
          "whole": dict(lens=[100 + 8 * i for i in range(57)], Q=2), "groups": dict(lens=[500, 132]),
          "groups merge": dict(lens=[9004, 84])}


@pytest.mark.parametrize("huge", [2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("path", PATHS)
def test_a_value_scale_counts_only_where_its_key_does(path, huge):
    """The last key, which the last row alone attends to, and the keys that only the first
    row's window still holds, are in blocks of very large scales: the bounds of the
    other rows know nothing of them."""
    g = np.random.default_rng(4)
    x = Problem(g, path, block=8, **{**RAGGED[path], "lens": [n - 3 for n in RAGGED[path]["lens"]]})
    for b, n in enumerate(x.lens):     # n = 1 mod 8
        x.scales[1][x.at(b, n - 1)[1]] *= huge
    x.check()
    x = Problem(g, path, block=8, **RAGGED[path])
    x.window = 54 - x.Q                # row 0 begins at n - 53 = 7 mod 8: at a block's last key
    for b, n in enumerate(x.lens):
        lo, _ = x.keys(b, 0)
        x.scales[1][x.at(b, lo - lo % 8)[1]] *= huge
    x.check()


@pytest.mark.parametrize("path", PATHS)
def test_a_large_value_scale_of_a_key_that_hardly_counts(path):
    """A block in the first tile (and one in the middle) whose probability is about 2^-73
    and whose values are 2^67 times the others': 2^-6 of the whole, and no reason for the
    others to lose bits."""
    g = np.random.default_rng(5)
    x = Problem(g, path, block=8)
    sign = np.where(g.random(D) < 0.5, -1.0, 1.0)
    x.q = (x.q.float().abs() * torch.from_numpy(sign).float()).to(x.q.dtype)
    away = np.where(sign > 0, -127, 127).astype(np.int8).view(np.uint8)
    for b, n in enumerate(x.lens):
        for j in {0, n // 2 // 8 * 8} if n else ():
            row, blk = x.at(b, j)
            x.codes[0][row[0], row[1]:row[1] + 8] = away
            x.scales[0][blk] = 2.0 ** -4
            x.scales[1][blk] = 2.0 ** 60
    x.check()


@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("path", PATHS)
def test_a_value_code_that_is_no_number_reaches_only_rows_that_attend(path, spread):
    """e4m3's NaN code in a value column: rows that attend to the key are NaN there (and
    only there), all others keep their bits.  Keys: the last one, which only the last row
    attends to; the first one of the first row's window; one that all attend to."""
    g = np.random.default_rng(6)
    x = Problem(g, path, block=8, kind="e4m3", **RAGGED[path])
    x.window = 54 - x.Q
    if spread:
        x.scales[1][...] = 2.0 ** g.integers(-20, 20, x.scales[1].shape)
    before = x.run()
    codes = x.codes[1].copy()
    for column, code in ((0, 127), (37, 255)):
        for where in ("last", "first", "all"):
            x.codes[1] = codes.copy()
            hit = np.zeros(before[0].shape, bool)
            for b, n in enumerate(x.lens):
                j = {"last": n - 1, "first": x.keys(b, 0)[0], "all": x.keys(b, x.Q - 1)[0] + 3}[where]
                x.codes[1][x.at(b, j)[0] + (1, column)] = code
                G = x.Hq // x.Hkv
                for i in range(x.Q):
                    lo, hi = x.keys(b, i)
                    hit[b, i, G:2 * G, column] = lo <= j < hi
            o, lse = x.run()
            assert np.isnan(o[hit]).all() and hit.any()
            assert np.array_equal(o[~hit], before[0][~hit]) and np.array_equal(lse, before[1])


@pytest.mark.parametrize("algo", ["decode", "generic"])
@pytest.mark.parametrize("big", [2.0 ** 14, 2.0 ** 24, 2.0 ** 50, 2.0 ** 108])
@pytest.mark.parametrize("path", PATHS)
def test_scores_up_to_the_largest_numbers(path, big, algo):
    """One key with a scale of 2^14 to 2^108: a score of about +2^10 times that leaves the key
    alone, a negative one drops it as a scale of 2^10 does, to the bit.  All keys with such
    scores, but one with half of their size: it is left alone."""
    g = np.random.default_rng(7)
    x = Problem(g, path, block=1)
    sign = np.where(g.random(D) < 0.5, -1, 1)
    x.q = (x.q.float().abs() * torch.from_numpy(sign).float()).to(x.q.dtype)
    at = {b: x.at(b, n // 3) for b, n in enumerate(x.lens) if n}

    def put(code, scale):
        for row, blk in at.values():
            x.codes[0][row] = (code * sign).astype(np.int8).view(np.uint8)
            x.scales[0][blk] = scale

    put(-127, 2.0 ** 10)
    below = x.run(algo=algo)
    put(-127, big)
    o, lse = x.run(algo=algo)
    assert np.array_equal(o, below[0]) and np.array_equal(lse, below[1])
    q = x.q.double().numpy()

    def check_alone(code):
        o, lse = x.run(algo=algo)
        for b, (row, blk) in at.items():
            v = cache_ref.code_values(x.codes[1][row], x.kind) * x.scales[1][blk].astype(np.float64)[:, None]
            v = v.repeat(x.Hq // x.Hkv, axis=0)[None]
            # (the probability is 1, the others 0: o is a value, rounded once)
            assert (np.abs(o[b] - v) <= HALF[x.dtype] * np.abs(v) + LEAST[x.dtype]).all()
            s = np.abs(q[b]).sum(-1) * code * big / math.sqrt(D)
            assert (np.abs(lse[b] - s) <= ((D + 8) * 2.0 ** -24 + 2.0 ** -20) * np.abs(s)).all()

    put(127, big)
    check_alone(127)
    x.codes[0][...] = (-127 * sign).astype(np.int8).view(np.uint8)
    x.scales[0][...] = big
    put(-64, big)
    check_alone(-64)


@pytest.mark.parametrize("algo", ["tcgen05", "mma", "generic"])
@pytest.mark.parametrize("what", ["key scale", "value scale", "value code"])
def test_numbers_that_are_none_over_expanded_keys(what, algo):
    """The kernels over expanded keys give what attn_fwd gives over the same keys and values,
    NaN among them, to the bit."""
    g = np.random.default_rng(8)
    x = Problem(g, "groups", block=8, kind="e4m3", lens=[497, 129])
    if what == "value code":
        x.codes[1][x.at(0, 496)[0] + (1, 3)] = 127
    else:
        x.scales[what == "value scale"][x.at(0, 496)[1] + (1,)] = math.nan
    o, lse = x.run(algo=algo)
    K = x.table.shape[1] * PAGE
    dense = [cache_ref.gather(cache_ref.as_values(c, s, x.kind), x.table, x.lens, K)
             for c, s in zip(x.codes, x.scales)]
    k, v = (torch.from_numpy(d).to(DEV).to(DT[x.dtype]) for d in dense)
    assert torch.isnan(v if what[0] == "v" else k).any()
    ro, rl = attn.attn_fwd(x.q.to(DEV), k, v, seqlens_k=i32(x.lens), algo=algo)
    assert np.array_equal(o, ro.double().cpu().numpy(), equal_nan=True)
    assert np.array_equal(lse, rl.double().cpu().numpy(), equal_nan=True)


@pytest.mark.parametrize("path", PATHS)
def test_a_table_far_wider_than_the_sequences(path):
    """A table for 131072 keys, as a serving program keeps one: the kernels are chosen by its
    width, and the expanded keys of one to eight sequences at a time take the workspace."""
    g = np.random.default_rng(9)
    x = Problem(g, path)
    fitted = x.run(algo="tcgen05")
    wide = np.full((len(x.lens), 131072 // PAGE), -1, np.int32)
    wide[:, :x.table.shape[1]] = x.table
    x.table = wide
    x.check()
    o, lse = x.run(algo="tcgen05")
    assert np.array_equal(o, fitted[0]) and np.array_equal(lse, fitted[1])
