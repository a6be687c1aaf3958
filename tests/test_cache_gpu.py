"""The 8-bit paged cache on the GPU against its plain restatement in 64 bits
(tests/cache_ref.py) and the oracle: appended codes and scales exactly,
attention within a bound derived from the roundings, pages exactly."""
import concurrent.futures
import math

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn
import oracle
from tests import cache_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# half a step of a rounding to the type, relative to the value
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def bits(t):
    return t.view(torch.uint8).cpu().numpy()


class Cache:
    """A cache of random codes whose unused places hold hostile values: NaN
    scales, and any codes."""

    def __init__(self, g, lens, page, block, Hkv, D, Dv, kind, max_pages=None, spare=3,
                 pow2=True):
        B = len(lens)
        need = [-(-int(n) // page) for n in lens]
        self.M = max_pages or max(1, max(need))
        P = sum(need) + spare
        order = g.permutation(P)
        self.table = np.full((B, self.M), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens, self.kind, self.page = np.asarray(lens, np.int32), kind, page
        self.codes, self.scales = [], []
        for W in (D, Dv):
            c = g.integers(0, 256, (P, page, Hkv, W), dtype=np.uint8)
            if kind == "int8":
                c[c == 128] = 129
            else:
                c[(c & 127) == 127] = 126
                # e4m3's values spread over 17 binades: keep most of them near one
                c = np.where(g.random(c.shape) < 0.9, (c & 0x87) | (6 + (c & 8)) << 3, c)
                c = c.astype(np.uint8)
            s = 2.0 ** g.integers(-8, -4, (P, page // block, Hkv))
            if kind == "e4m3":
                s = s * 16
            if not pow2:
                s = s * g.uniform(0.6, 1.0, s.shape)
            self.codes.append(c)
            self.scales.append(s.astype(np.float32))
        # blocks that hold no token get NaN scales
        used = np.zeros((P, page // block), bool)
        for b in range(B):
            for j in range(0, int(lens[b]), block):
                used[self.table[b, j // page], j % page // block] = True
        for s in self.scales:
            s[~used] = np.nan

    def gpu(self):
        t = cache_ref.TORCH_CODE[self.kind]
        pages = [torch.from_numpy(c.copy()).to(DEV).view(t) for c in self.codes]
        scales = [torch.from_numpy(s.copy()).to(DEV) for s in self.scales]
        return pages[0], pages[1], scales[0], scales[1]

    def finest(self, K):
        """[B, H, D]: 2^-39 of the sequence's largest value scale times its codes'
        magnitudes -- half a step of the decode kernel's smallest probabilities
        (fp16 steps of 2^-24 under 2^14 at the row's largest, relative to the
        largest scale), added up over the keys."""
        ones = np.ones_like(self.scales[1])
        c = cache_ref.gather(np.abs(cache_ref.as_values(self.codes[1], ones, self.kind)), self.table,
                             self.lens, K)
        B, _, H, _ = c.shape
        nb = self.scales[1].shape[1]
        s = np.nan_to_num(self.scales[1]).repeat(self.page // nb, axis=1)
        s = cache_ref.gather(s[..., None], self.table, self.lens, K).max(1)
        return 2.0 ** -39 * c.sum(1) * s

    def dense(self, K):
        """[B, K, H, D] float32 values (exact for powers of two) of the valid keys."""
        out = []
        for c, s in zip(self.codes, self.scales):
            v = cache_ref.as_values(c, np.nan_to_num(s), self.kind)
            out.append(cache_ref.gather(v, self.table, self.lens, K))
        return out


def attention_bounds(q, k, v, B, Hq, Hkv, Q, K, D, Dv, lens, sq, window, scale, mask, dtype, finest=0):
    """Oracle outputs and how far the kernels may be from them.

    With A = sum p |v| of a row: a score's fp32 accumulation is off by at most
    (D + 8) 2^-24 S, S = scale * max_k sum |q||k|, and moves p by twice that
    relative to it; the sums over K keys of p and of p v are off by at most
    K 2^-24 each, ex2 by 2^-22; p is rounded to q's type (or finer) for the
    second product, O once at the end.  Below 2^-14 an fp16 p (at most 1 at the
    row's largest score, so that sum p >= 1) has steps of 2^-24: off by 2^-25,
    which times |v| adds up over the keys; the decode kernel's probabilities reach
    further down (``finest``)."""
    kw = dict(B=B, Hq=Hq, Hkv=Hkv, Q=Q, K=K, D=D, Dv=Dv, seqlens_q=sq, seqlens_k=lens,
              window=window, scale=scale, mask=mask)
    f = lambda x: np.ascontiguousarray(x, np.float32)  # noqa: E731
    o, lse = oracle.attn_padded(f(q), f(k), f(v), **kw)
    a, _ = oracle.attn_padded(f(q), f(k), f(np.abs(v)), **kw)
    G = Hq // Hkv
    s = np.zeros((B, Q, Hq))
    for b in range(B):
        n = int(lens[b])
        if n:
            ka = np.abs(k[b, :n]).repeat(G, axis=1)  # [n, Hq, D]
            s[b] = abs(scale) * np.einsum("qhd,khd->qhk", np.abs(q[b]), ka).max(-1)
    ds = (D + 8) * 2.0 ** -24 * s
    rel = 2 * ds + 2 * K * 2.0 ** -24 + 2.0 ** -20
    half = HALF[dtype]
    tol_o = half * np.abs(o) + (half + rel[..., None]) * a + 1e-30
    if dtype == "f16":  # subnormal outputs and probabilities
        tol_o = tol_o + 2.0 ** -25 * (1 + np.abs(v).sum(1).repeat(G, axis=1)[:, None])
    if not np.isscalar(finest):
        tol_o = tol_o + finest.repeat(G, axis=1)[:, None]
    tol_l = ds + K * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
    return o, lse, tol_o, tol_l


def check_attention(g, dtype, kind, B, Hq, Hkv, Q, D, Dv, lens, page, block, *, window=0,
                    mask="causal", sq=None, algo="auto", max_pages=None, scale=None, qscale=1.0):
    c = Cache(g, lens, page, block, Hkv, D, Dv, kind, max_pages)
    K = c.M * page
    q = torch.from_numpy(g.standard_normal((B, Q, Hq, D)).astype(np.float32) * qscale).to(DT[dtype])
    scale = 1 / math.sqrt(D) if scale is None else scale
    kp, vp, ks, vs = c.gpu()
    o = torch.full((B, Q, Hq, Dv), math.nan, dtype=DT[dtype], device=DEV)
    lse = torch.full((B, Q, Hq), math.nan, device=DEV)
    before = [bits(t) for t in (kp, vp, ks, vs)]
    attn.attn_fwd_paged_q8(q.to(DEV), kp, vp, ks, vs, i32(c.table), i32(c.lens), o, lse,
                           seqlens_q=None if sq is None else i32(sq), window=window, scale=scale,
                           algo=algo, mask=mask)
    torch.cuda.synchronize()
    assert all(np.array_equal(x, bits(t)) for x, t in zip(before, (kp, vp, ks, vs)))
    kd, vd = c.dense(K)
    ro, rl, to, tl = attention_bounds(
        q.float().numpy().astype(np.float64), kd, vd, B, Hq, Hkv, Q, K, D, Dv, c.lens,
        None if sq is None else np.asarray(sq, np.int32), window, scale,
        {"causal": 0, "causal_top_left": 1, "none": 2}[mask], dtype, c.finest(K))
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    empty = rl == -math.inf
    assert np.all(o[empty] == 0) and not np.signbit(o[empty]).any() and np.all(lse[empty] == -math.inf)
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(lse[~empty]))
    eo = np.abs(o - ro) / to
    el = np.abs(lse[~empty] - rl[~empty]) / tl[~empty] if (~empty).any() else np.zeros(1)
    assert eo.max() <= 1, f"o off by {eo.max():.3g} of the bound"
    assert el.max() <= 1, f"lse off by {el.max():.3g} of the bound"


ATTEND = [
    # dtype, kind, Hq, Hkv, Q, D, Dv, lens, page, block, options
    ("bf16", "e4m3", 8, 2, 1, 128, 128, [1, 0, 63, 64, 65, 700], 64, 64, {}),
    ("bf16", "int8", 32, 8, 1, 128, 128, [127, 128, 129, 1025], 64, 16, {}),
    ("f16", "int8", 8, 1, 1, 64, 64, [2053, 1, 500], 128, 32, {}),
    ("f16", "e4m3", 16, 4, 4, 64, 64, [3, 900, 2, 0], 32, 8, {}),           # fewer keys than rows
    ("bf16", "int8", 4, 4, 1, 256, 256, [333, 40], 16, 16, {}),
    ("bf16", "e4m3", 6, 2, 5, 128, 128, [1000, 31], 256, 128, {}),          # 15 rows, G = 3
    ("bf16", "int8", 12, 2, 1, 96, 96, [77, 400], 64, 32, {}),
    ("f16", "e4m3", 3, 3, 2, 80, 80, [150, 9], 8, 2, {}),
    ("bf16", "int8", 8, 2, 1, 128, 64, [300, 300], 64, 64, {}),             # D != Dv
    ("bf16", "e4m3", 8, 2, 3, 64, 128, [300, 12], 64, 64, {}),
    ("bf16", "e4m3", 8, 2, 1, 128, 128, [900, 100, 5], 64, 64, dict(window=70)),
    ("f16", "int8", 8, 2, 4, 64, 64, [900, 100, 5], 64, 64, dict(window=1)),
    ("bf16", "int8", 8, 2, 4, 128, 128, [300, 2, 0], 64, 16, dict(mask="causal_top_left")),
    ("bf16", "int8", 8, 2, 4, 128, 128, [300, 2, 0], 64, 16, dict(mask="none")),
    ("bf16", "e4m3", 8, 2, 4, 128, 128, [300, 70, 9], 64, 64, dict(sq=[2, 0, 4])),
    ("bf16", "int8", 4, 2, 1, 40, 24, [50, 7], 4, 4, {}),                   # odd widths, tiny pages
    ("f16", "e4m3", 4, 2, 2, 33, 7, [50, 7, 0], 16, 1, {}),
    ("f32", "int8", 4, 2, 3, 64, 48, [90, 0, 2], 16, 16, {}),
    ("f32", "e4m3", 4, 1, 1, 72, 72, [200], 1, 1, {}),                      # one-token pages
    ("bf16", "e4m3", 8, 2, 20, 128, 128, [700, 33, 20], 64, 64, {}),        # more rows than 16
    ("bf16", "int8", 8, 2, 7, 128, 128, [700, 3], 64, 64, {}),              # 28 rows
    ("bf16", "e4m3", 8, 2, 150, 128, 128, [700, 33, 0, 150], 64, 32, {}),
    ("f16", "int8", 4, 2, 130, 64, 64, [1000, 130], 128, 16, dict(window=100)),
    ("bf16", "int8", 4, 2, 64, 256, 256, [300, 64], 64, 64, {}),
    ("bf16", "e4m3", 8, 2, 1, 128, 128, [64, 1], 64, 64, dict(max_pages=40)),  # a wide table
    ("bf16", "int8", 8, 2, 1, 128, 128, [500], 64, 64, dict(scale=-0.05)),
    ("bf16", "int8", 8, 2, 1, 128, 128, [500], 64, 64, dict(scale=0.0)),
    ("bf16", "e4m3", 8, 2, 1, 128, 128, [500], 64, 64, dict(qscale=1e-20, scale=1e19)),
    ("bf16", "int8", 8, 2, 1, 128, 128, [500], 64, 64, dict(qscale=1e20, scale=1e-21)),
    ("f16", "int8", 64, 8, 1, 128, 128, [9000, 4097], 64, 64, {}),          # many splits
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
def test_attention_over_the_cache(i):
    dtype, kind, Hq, Hkv, Q, D, Dv, lens, page, block, kw = ATTEND[i]
    check_attention(np.random.default_rng(100 + i), dtype, kind, len(lens), Hq, Hkv, Q, D, Dv,
                    lens, page, block, **kw)


@pytest.mark.parametrize("algo", ["generic", "tcgen05", "mma", "decode"])
def test_attention_with_a_chosen_kernel(algo):
    check_attention(np.random.default_rng(7), "bf16", "int8", 2, 8, 2, 3, 128, 128, [300, 41], 64,
                    16, algo=algo)


def test_attention_ignores_scales_of_pages_behind_the_window():
    # a page that every row's window has left may be anyone's: its scales (finite
    # and huge, or NaN) take no part
    g = np.random.default_rng(8)
    for bad in (1e30, math.nan):
        c = Cache(g, [200, 120], 64, 64, 2, 128, 128, "int8")
        for b, n in enumerate((200, 120)):
            for s in c.scales:  # keys up to n - 41 are outside
                s[c.table[b, (n - 40) // 64 - 1]] = 2.0 ** -5
        q = torch.from_numpy(g.standard_normal((2, 1, 8, 128)).astype(np.float32)).bfloat16().to(DEV)
        kp, vp, ks, vs = c.gpu()
        good = attn.attn_fwd_paged_q8(q, kp, vp, ks, vs, i32(c.table), i32(c.lens), window=40)
        for b, n in enumerate((200, 120)):
            for s in (ks, vs):
                s[int(c.table[b, (n - 40) // 64 - 1])] = bad
        got = attn.attn_fwd_paged_q8(q, kp, vp, ks, vs, i32(c.table), i32(c.lens), window=40)
        assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])


def test_attention_without_pages():
    # an empty table: every row is empty
    c = Cache(np.random.default_rng(0), [0, 0], 16, 16, 2, 64, 64, "int8")
    kp, vp, ks, vs = c.gpu()
    q = torch.randn((2, 1, 4, 64), device=DEV, dtype=torch.bfloat16)
    o, lse = attn.attn_fwd_paged_q8(q, kp, vp, ks, vs, torch.zeros((2, 0), dtype=torch.int32, device=DEV),
                                    i32([0, 0]))
    assert (o == 0).all() and (lse == -math.inf).all()


def test_attention_scales_that_are_no_powers_of_two():
    # code * scale: the decode kernels multiply scores and probabilities by the
    # scales in fp32; a copy in q's type would round every key and value once
    g = np.random.default_rng(5)
    c = Cache(g, [300, 77], 64, 16, 2, 128, 128, "int8", pow2=False)
    q = torch.from_numpy(g.standard_normal((2, 1, 8, 128)).astype(np.float32)).bfloat16()
    kp, vp, ks, vs = c.gpu()
    o, lse = attn.attn_fwd_paged_q8(q.to(DEV), kp, vp, ks, vs, i32(c.table), i32(c.lens))
    kd, vd = c.dense(c.M * 64)
    ro, rl, to, tl = attention_bounds(q.double().numpy(), kd, vd, 2, 8, 2, 1, c.M * 64, 128, 128,
                                      c.lens, None, 0, 128 ** -0.5, 0, "bf16")
    # (one rounding of a key moves a score by at most half a step of S, and p by twice that)
    s = np.stack([128 ** -0.5 * np.einsum("qhd,khd->qhk", np.abs(q[b].double().numpy()),
                                          np.abs(kd[b]).repeat(4, 1)).max(-1) for b in range(2)])
    a = (to - HALF["bf16"] * np.abs(ro))  # at least half a step of sum p |v|
    to = to + a + 2 * HALF["bf16"] * s[..., None] * a / HALF["bf16"]
    assert (np.abs(o.float().cpu().numpy() - ro) <= to).all()
    assert (np.abs(lse.cpu().numpy() - rl) <= tl + HALF["bf16"] * s).all()


def test_attention_over_a_poisoned_block_is_not_a_number_or_empty():
    # a NaN scale is a NaN key: the rows that attend to it are not finite values
    g = np.random.default_rng(6)
    c = Cache(g, [300, 300], 64, 64, 2, 128, 128, "int8")
    kp, vp, ks, vs = c.gpu()
    ks[int(c.table[1, 2]), 0, 1] = math.nan
    q = torch.randn((2, 1, 8, 128), device=DEV, dtype=torch.bfloat16)
    o, lse = attn.attn_fwd_paged_q8(q, kp, vp, ks, vs, i32(c.table), i32(c.lens))
    bad = ~torch.isfinite(o.float()).all(-1)
    assert not bad[0].any() and not bad[1, :, :4].any()
    assert bad[1, :, 4:].all()


@pytest.mark.parametrize("i", range(8))
def test_attention_of_ragged_batches(i):
    """Shares of the tiles that begin and end anywhere in units of any length:
    empty sequences, single tiles, units over many shares."""
    g = np.random.default_rng(600 + i)
    B = int(g.integers(1, 70))
    most = int([20, 130, 600, 5000][i % 4] if B < 8 or i % 4 < 3 else 600)
    lens = [int(n) if g.random() < 0.8 else 0 for n in g.integers(0, most + 1, B)]
    Hkv, G, Q = int(g.integers(1, 5)), int(g.integers(1, 5)), int(g.integers(1, 4))
    check_attention(g, ["bf16", "f16"][i % 2], ["int8", "e4m3"][i // 2 % 2], B, Hkv * G, Hkv, Q, 64,
                    64, lens, 64, 32, window=int(g.integers(0, 300)) if i % 3 == 0 else 0)


@pytest.mark.parametrize("i", range(12))
def test_attention_of_small_problems(i):
    """Few tiles a sequence: one to eight CTAs share them in a cluster, some
    without a tile; empty sequences, windows, fewer keys than rows."""
    g = np.random.default_rng(700 + i)
    page = int([8, 16, 64, 128][i % 4])
    M = int(g.integers(1, max(2, 4000 // page // (1 + i % 5))))
    B = int(g.integers(1, 5)) if i < 9 else 90
    lens = [int(n) if g.random() < 0.85 else 0 for n in g.integers(0, M * page + 1, B)]
    Hkv, G, Q = int(g.integers(1, 5)), int(g.integers(1, 5)), int(g.integers(1, 4))
    D = int(g.choice([64, 96, 128, 256]))
    check_attention(g, ["bf16", "f16"][i % 2], ["int8", "e4m3"][i // 2 % 2], B, Hkv * G, Hkv, Q, D,
                    D, lens, page, 8, window=int(g.integers(1, 200)) if i % 3 == 0 else 0,
                    max_pages=M, algo="decode")


ROWS = [
    # dtype, kind, Hq, Hkv, Q, D, Dv, lens, page, block, options: row groups of 16
    ("bf16", "e4m3", 17, 1, 1, 128, 128, [700, 0, 1, 129], 64, 64, {}),
    ("f16", "int8", 16, 2, 3, 64, 64, [2053, 2, 500], 128, 32, {}),              # 24 rows
    ("bf16", "int8", 32, 4, 4, 128, 128, [300, 7000, 64], 64, 16, {}),           # 32
    ("bf16", "e4m3", 6, 2, 11, 96, 80, [900, 10, 333], 64, 64, {}),              # 33: a group of one row
    ("f16", "e4m3", 12, 4, 16, 256, 256, [400, 16], 32, 8, {}),                  # 48
    ("bf16", "int8", 8, 1, 8, 64, 128, [3000, 5], 64, 64, dict(window=200)),     # 64
    ("bf16", "e4m3", 8, 2, 9, 128, 128, [300, 2, 0, 9], 16, 16, dict(mask="causal_top_left")),
    ("bf16", "int8", 8, 2, 9, 128, 128, [300, 2, 0, 9], 16, 16, dict(mask="none")),
    ("f16", "int8", 8, 2, 40, 64, 64, [900, 100, 5], 64, 64, dict(window=1)),
    ("bf16", "e4m3", 8, 2, 20, 128, 128, [700, 33, 20, 90], 64, 64, dict(sq=[3, 0, 20, 17])),
    ("f16", "e4m3", 4, 1, 250, 64, 64, [1000, 3], 64, 32, {}),                   # 1000
    ("bf16", "int8", 4, 1, 256, 80, 80, [256, 2000, 0], 128, 128, dict(window=100)),
    ("bf16", "int8", 40, 20, 9, 128, 128, [300, 500, 41, 77, 1, 0, 64] * 3, 64, 64, {}),
    ("bf16", "int8", 36, 36, 30, 64, 64, [30, 600, 0, 64] * 2, 64, 64, {}),       # 72 groups
]


@pytest.mark.parametrize("i", range(len(ROWS)))
def test_attention_of_many_rows_over_the_codes(i):
    dtype, kind, Hq, Hkv, Q, D, Dv, lens, page, block, kw = ROWS[i]
    check_attention(np.random.default_rng(900 + i), dtype, kind, len(lens), Hq, Hkv, Q, D, Dv,
                    lens, page, block, algo="decode", **kw)


@pytest.mark.parametrize("algo", ["tcgen05", "mma"])
@pytest.mark.parametrize("i", [i for i, c in enumerate(ATTEND) if c[4] >= 20])
def test_attention_of_many_rows_over_expanded_keys(i, algo):
    dtype, kind, Hq, Hkv, Q, D, Dv, lens, page, block, kw = ATTEND[i]
    if algo == "mma" and D > 128:
        pytest.skip("wider than the kernel takes")
    check_attention(np.random.default_rng(950 + i), dtype, kind, len(lens), Hq, Hkv, Q, D, Dv,
                    lens, page, block, algo=algo, **kw)


# -------------------------------------------------------------------- append

def run_append(g, dtype, kind, lens, new, N, Hkv, D, Dv, page, block, packed=False, extra_pages=0,
               spread=6.0, table_edit=None):
    B = len(lens)
    end = [a + b for a, b in zip(lens, new)]
    c = Cache(g, end, page, block, Hkv, D, Dv, kind, max_pages=max(1, max(-(-e // page) for e in end)) + extra_pages)
    # only the rows before the new ones count as held: blocks behind them NaN
    held = np.zeros((len(c.codes[0]), page // block), bool)
    for b in range(B):
        for j in range(0, lens[b], block):
            held[c.table[b, j // page], j % page // block] = True
    for s in c.scales:
        s[~held] = np.nan
    if table_edit:
        table_edit(c.table)
    rows = []
    for W in (D, Dv):
        x = g.standard_normal((B, N, Hkv, W)) * 2.0 ** g.uniform(-spread, spread, (B, N, Hkv, 1))
        rows.append(torch.from_numpy(x.astype(np.float32)).to(DT[dtype]))
    kp, vp, ks, vs = c.gpu()
    if packed:
        cu = np.concatenate([[0], np.cumsum(new)])
        flat = [torch.cat([r[b, :new[b]] for b in range(B)]).to(DEV) for r in rows]
        attn.attn_cache_append_varlen(*flat, i32(cu), N, kp, vp, ks, vs, i32(c.table), i32(lens))
    else:
        attn.attn_cache_append(rows[0].to(DEV), rows[1].to(DEV), kp, vp, ks, vs, i32(c.table),
                               i32(lens), seqlens_new=i32(new))
    torch.cuda.synchronize()
    for r, codes, scales, got_c, got_s in zip(rows, c.codes, c.scales, (kp, vp), (ks, vs)):
        s64 = scales.astype(np.float64)
        cache_ref.append([r[b, :new[b]].double().numpy() for b in range(B)], lens, new, c.table,
                         codes, s64, kind)
        got = got_s.cpu().numpy().astype(np.float64)
        assert np.array_equal(got, s64, equal_nan=True), "scales"
        assert np.array_equal(bits(got_c).reshape(codes.shape), codes), "codes"


APPEND = [
    # dtype, kind, lens, new, N, Hkv, D, Dv, page, block
    ("bf16", "int8", [0, 1, 63, 64, 100], [1, 1, 1, 1, 0], 1, 8, 128, 128, 64, 64),
    ("bf16", "e4m3", [0, 1, 63, 64, 100], [1, 1, 1, 1, 1], 1, 2, 64, 64, 64, 16),
    ("f16", "int8", [5, 0, 30], [200, 77, 3], 200, 2, 128, 64, 64, 32),
    ("bf16", "e4m3", [5, 0, 200], [130, 256, 1], 256, 3, 96, 80, 128, 128),
    ("f32", "int8", [2, 9], [40, 11], 40, 2, 64, 64, 16, 8),
    ("f32", "e4m3", [2, 9], [40, 0], 41, 1, 33, 7, 16, 1),       # odd widths: element by element
    ("f16", "e4m3", [0, 3], [5, 4], 5, 2, 12, 20, 4, 2),
    ("bf16", "int8", [10], [700], 700, 1, 256, 512, 256, 256),   # more than a thread keeps
    ("bf16", "int8", [7], [300], 300, 1, 33, 24, 256, 256),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append(i, packed):
    run_append(np.random.default_rng(200 + i), *APPEND[i], packed=packed)


def test_append_drops_rows_without_a_place():
    def edit(t):
        t[0, 1] = -1          # no page
        t[1, 0] = 1 << 20     # no such page
    run_append(np.random.default_rng(1), "bf16", "int8", [10, 0, 20], [40, 30, 3], 40, 2, 64, 64, 16,
               16, table_edit=edit)
    # past the table's last page
    g = np.random.default_rng(2)
    c = Cache(g, [32, 32], 16, 16, 2, 64, 64, "e4m3")
    kp, vp, ks, vs = c.gpu()
    before = [bits(t) for t in (kp, vp, ks, vs)]
    x = torch.randn((2, 5, 2, 64), device=DEV)
    attn.attn_cache_append(x, x, kp, vp, ks, vs, i32(c.table), i32([32, 1000]))
    attn.attn_cache_append(x, x, kp, vp, ks, vs, i32(c.table), i32([32, 32]), seqlens_new=i32([-3, 0]))
    assert all(np.array_equal(a, bits(t)) for a, t in zip(before, (kp, vp, ks, vs)))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_token_by_token_is_near_the_rows(kind):
    """A block filled one token at a time, each larger than the last by up to 4:
    int8 codes are off by at most one step of the final scale in all (half a
    step a rounding, the earlier ones' steps at most halves of the next), e4m3
    codes by half a step of the value, or of the subnormals under the final scale
    once more."""
    g = np.random.default_rng(11)
    page = block = 16
    kp = torch.zeros((2, page, 1, 64), dtype=torch.int8, device=DEV).view(cache_ref.TORCH_CODE[kind])
    vp = kp.clone()
    ks = torch.full((2, 1, 1), math.nan, device=DEV)
    vs = ks.clone()
    x = g.standard_normal((1, page, 1, 64)) * np.cumprod(2.0 ** g.uniform(-0.5, 2, page))[None, :, None, None]
    x = torch.from_numpy(x.astype(np.float32)).bfloat16()
    for t in range(page):
        xt = x[:, t:t + 1].to(DEV)
        attn.attn_cache_append(xt, xt, kp, vp, ks, vs, i32([[1]]), i32([t]))
    want = x[0, :, 0].double().numpy()
    s = float(ks[1, 0, 0])
    assert s == cache_ref.scale_for(np.abs(want).max(), kind) and float(vs[1, 0, 0]) == s
    got = cache_ref.as_values(bits(kp).reshape(2, page, 1, 64), ks.cpu().numpy(), kind)[1, :, 0]
    assert np.array_equal(bits(kp), bits(vp))
    if kind == "int8":
        assert np.abs(got - want).max() <= s
    else:
        assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * s).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_of_values_that_are_not_finite_poisons_their_block(kind, bad):
    g = np.random.default_rng(12)
    c = Cache(g, [40], 32, 16, 2, 64, 64, kind)
    kp, vp, ks, vs = c.gpu()
    pg = int(c.table[0, 0])
    x = torch.randn((1, 20, 2, 64), device=DEV)
    x[0, 1, 1, 5] = bad
    attn.attn_cache_append(x[:, :4].contiguous(), x[:, :4].contiguous(), kp, vp, ks, vs,
                           i32(c.table), i32([3]))
    assert torch.isnan(ks[pg, 0, 1]) and torch.isfinite(ks[pg, 0, 0])
    assert (bits(kp)[pg, :7, 1] & 127 == 0).all()   # earlier rows and new ones
    # it stays poisoned until the block is begun afresh
    x[0, 1, 1, 5] = 0
    attn.attn_cache_append(x[:, :1].contiguous(), x[:, :1].contiguous(), kp, vp, ks, vs, i32(c.table), i32([7]))
    assert torch.isnan(ks[pg, 0, 1])
    attn.attn_cache_append(x[:, :1].contiguous(), x[:, :1].contiguous(), kp, vp, ks, vs, i32(c.table), i32([0]))
    assert torch.isfinite(ks[pg, 0]).all()


# --------------------------------------------------------------------- pages

def random_pools(g, P, shapes):
    return [torch.from_numpy(g.integers(0, 256, (P, n), dtype=np.uint8)).to(DEV) for n in shapes]


@pytest.mark.parametrize("shapes", [(4096,), (16, 32768, 48), (7, 4100, 1, 4099), (64,) * 70])
@pytest.mark.parametrize("n", [0, 1, 9])
def test_page_copy(shapes, n):
    g = np.random.default_rng(20)
    pools = random_pools(g, 21, shapes)
    want = [p.cpu().numpy().copy() for p in pools]
    order = g.permutation(21)
    src, dst = order[:n], order[n:2 * n]
    attn.attn_pages_copy(pools, pools, i32(src), i32(dst))
    for w, p in zip(want, pools):
        w[dst] = w[src]
        assert np.array_equal(w, p.cpu().numpy())


def test_page_copy_between_pools_and_of_pages_that_do_not_exist():
    g = np.random.default_rng(21)
    a, b = random_pools(g, 9, (512, 6)), random_pools(g, 5, (512, 6))
    want = [p.cpu().numpy().copy() for p in b]
    for w, p in zip(want, a):
        w[[4, 0]] = p.cpu().numpy()[[8, 3]]
    attn.attn_pages_copy(a, b, i32([8, 3, -1, 9, 2, 2]), i32([4, 0, 1, 2, 5, -7]))
    assert all(np.array_equal(w, p.cpu().numpy()) for w, p in zip(want, b))


def random_table(g, S, M, page, P, share=0.6, pins=2):
    """A consistent random version: slots that share prefixes of full pages."""
    table = np.full((S, M), -1, np.int32)
    lens = np.zeros(S, np.int32)
    free = list(g.permutation(P))
    for i in range(S):
        n = int(g.integers(0, M * page // 2 + 1))
        at = 0
        if i and g.random() < share:  # share the full pages of an earlier slot
            j = int(g.integers(0, i))
            at = min(lens[j] // page, n // page)
            table[i, :at] = table[j, :at]
        for e in range(at, -(-n // page)):
            if not free:
                n = e * page
                break
            table[i, e] = free.pop()
        lens[i] = n
    refs = np.zeros(P, np.int32)
    for c in table[table >= 0]:
        refs[c] += 1
    for c in g.permutation(P)[:pins]:  # somebody else's
        refs[c] += 1
    return table, lens, refs


def check_fork(g, table, lens, refs, parents, new, page, shapes=(160, 5000)):
    P = len(refs)
    pools = random_pools(g, P, shapes)
    want = [p.cpu().numpy().copy() for p in pools]
    out = attn.attn_pages_fork(pools, i32(table), i32(lens), i32(refs), i32(parents), page,
                               new_tokens=None if new is None else i32(new))
    ref = cache_ref.fork(table, lens, refs, parents, [0] * len(parents) if new is None else new, page)
    for name, x, r in zip(("table", "lens", "refs", "status"), out, ref):
        assert np.array_equal(x.cpu().numpy(), r), (name, x.cpu().numpy(), r)
    for w, p in zip(want, pools):
        src = w.copy()
        for s, d in ref[4]:
            w[d] = src[s]
        assert np.array_equal(w, p.cpu().numpy()), "pages"
    return ref


# pages of a few bytes (one cluster does everything), of so many that the copies take
# a launch of their own, and of so many more that the plan keeps lists
BIG, HUGE = (1 << 18, 5000), (1 << 20, 1 << 20, 5000)


@pytest.mark.parametrize("shapes", [(160, 5000), BIG, HUGE, ()])
@pytest.mark.parametrize("seed", range(12))
def test_fork(seed, shapes):
    g = np.random.default_rng(300 + seed)
    S, M, page = int(g.integers(1, 40)), int(g.integers(1, 50)), int(2 ** g.integers(0, 7))
    table, lens, refs = random_table(g, S, M, page, S * M + 5)
    N = int(g.integers(1, 50))
    parents = g.integers(-1, S + 1, N)
    new = np.minimum(g.integers(-2, 3 * page, N), M * page // 2)
    if len(refs) * sum(shapes) > 1 << 30:
        shapes = (1 << 30) // len(refs) // 16 * 16, 48
    check_fork(g, table, lens, refs, parents, None if seed % 4 == 0 else new, page, shapes)


def test_fork_of_many_slots_and_wide_growth():
    g = np.random.default_rng(31)
    table, lens, refs = random_table(g, 300, 80, 16, 9000, pins=20)
    ref = check_fork(g, table, lens, refs, g.integers(0, 300, 1100), g.integers(0, 64, 1100), 16,
                     shapes=(64,))
    assert ref[3][0] == 0 and ref[3][3] > 300


@pytest.mark.parametrize("room", [True, False])
def test_fork_in_a_pool_of_very_many_pages(room):
    """200 thousand pages: the counts are kept in a workspace."""
    g = np.random.default_rng(37)
    table, lens, refs = random_table(g, 40, 60, 8, 200003, pins=5)
    if not room:
        refs[refs == 0] = 1
    parents = g.integers(-1, 40, 70)
    check_fork(g, table, lens, refs, parents, g.integers(0, 30, 70), 8, shapes=(48, 1000))


def test_fork_of_a_wide_table():
    """More entries than one cluster writes, and more slots than a block lists."""
    g = np.random.default_rng(38)
    table, lens, refs = random_table(g, 20, 30, 8, 9000, pins=5)
    wide = np.full((20, 700), -1, np.int32)
    wide[:, :30] = table
    check_fork(g, wide, lens, refs, g.integers(0, 20, 300), np.ones(300, int), 8, shapes=(64,))
    check_fork(g, table, lens, refs, g.integers(-1, 20, 4200), np.ones(4200, int), 8, shapes=(64,))


@pytest.mark.parametrize("shapes", [(160, 5000), BIG])
def test_fork_makes_a_rolled_back_page_private(shapes):
    # slot 0 rolled back into page 3, which slot 1 still holds as a full page
    table = np.array([[3, -1], [3, 1]], np.int32)
    refs = np.array([0, 1, 0, 2], np.int32)
    ref = check_fork(np.random.default_rng(0), table, np.array([2, 5]), refs, [0, 1], [1, 1], 4, shapes)
    assert ref[0].tolist() == [[0, -1], [3, 1]] and ref[4] == [(3, 0)]
    # the same page held by nobody else but a pin: copied, too
    ref = check_fork(np.random.default_rng(0), table[:1], np.array([2]), np.array([0, 0, 0, 2]), [0],
                     [1], 4, shapes)
    assert ref[4] == [(3, 0)]


@pytest.mark.parametrize("shapes", [(160, 5000), BIG])
def test_fork_without_room_changes_nothing(shapes):
    g = np.random.default_rng(33)
    table, lens, refs = random_table(g, 6, 8, 4, 14, pins=0)
    ref = check_fork(g, table, lens, refs, [0, 1, 2, 3, 4, 5] * 3, [9] * 18, 4, shapes)
    assert ref[3][0] > 0
    ref = check_fork(g, table, lens, refs, [0, -1], [100, 0], 4, shapes)
    assert ref[3][1] == 1
    ref = check_fork(g, table, lens, refs, [0, -1], [2 ** 31 - 1, 0], 4, shapes)
    assert ref[3][1] == 1


@pytest.mark.parametrize("small", [True, False])
def test_fork_of_an_inconsistent_table_stays_in_bounds(small):
    # entries out of range, lengths past the table, counts that do not fit: wrong pages
    # at worst; the guard bytes behind every buffer stay
    g = np.random.default_rng(34)
    S, M, P, N = 7, 6, 20, 30
    table = g.integers(-5, P + 5, (S, M)).astype(np.int32)
    lens = g.integers(-10, 10 * M, S).astype(np.int32)
    pools = random_pools(g, P, (100,) if small else (1 << 19,))
    for refs in (np.zeros(P), np.full(P, 3), g.integers(-1, 3, P)):
        out = attn.attn_pages_fork(pools, i32(table), i32(lens), i32(refs), i32(g.integers(-3, S + 3, N)), 4,
                                   new_tokens=i32(g.integers(-5, 9, N)))
        t = out[0].cpu().numpy()
        assert ((t >= -1) & (t < P)).all()


def test_fork_without_slots_frees_everything():
    g = np.random.default_rng(35)
    table, lens, refs = random_table(g, 5, 6, 8, 40, pins=0)
    ref = check_fork(g, table, lens, refs, [], [], 8)
    assert (ref[2] == 0).all()


@pytest.mark.parametrize("P", [1, 2, 31, 1024, 5000, 40001, 200003])
@pytest.mark.parametrize("share", [0.0, 0.1, 0.5, 0.95, 1.0])
@pytest.mark.parametrize("total", [81, 1 << 25, 1 << 28])
def test_compact(P, share, total):
    """Pools of 81 bytes a page (one cluster does everything), of 32 MB (a copy
    launch) and of 256 MB (lists in a workspace)."""
    g = np.random.default_rng(P + int(100 * share))
    if total > 81 and not 1024 <= P <= 40001:
        pytest.skip("the same path as with small pages")
    refs = np.where(g.random(P) < share, g.integers(1, 4, P), 0).astype(np.int32)
    table = g.integers(-3, P + 3, (9, 33)).astype(np.int32)
    pools = random_pools(g, P, (total // P // 16 * 16, 33) if total > 81 else (48, 33))
    want = [p.cpu().numpy().copy() for p in pools]
    out = attn.attn_pages_compact(pools, i32(table), i32(refs))
    ref = cache_ref.compact(table, refs)
    for name, x, r in zip(("table", "refs", "remap", "n"), out, ref):
        assert np.array_equal(x.cpu().numpy(), r), name
    for w, p in zip(want, pools):
        src = w.copy()
        for s, d in ref[4]:
            w[d] = src[s]
        assert np.array_equal(w, p.cpu().numpy())


def test_pages_of_many_pools():
    # more pools than one launch takes
    g = np.random.default_rng(36)
    table, lens, refs = random_table(g, 9, 8, 8, 120, pins=1)
    check_fork(g, table, lens, refs, [0, 0, 1, 1, 2, 2, 3, 3], [1] * 8, 8, shapes=(96,) * 130)
    P = 50
    refs = (g.random(P) < 0.5).astype(np.int32)
    pools = random_pools(g, P, (40,) * 70)
    want = [p.cpu().numpy().copy() for p in pools]
    attn.attn_pages_compact(pools, i32(np.zeros((0, 4))), i32(refs))
    moves = cache_ref.compact(np.zeros((0, 4), np.int32), refs)[4]
    for w, p in zip(want, pools):
        src = w.copy()
        for s, d in moves:
            w[d] = src[s]
        assert np.array_equal(w, p.cpu().numpy())


# ------------------------------------------------------------- as they are used

def serve(steps, dtype="bf16", kind="int8", graph=False, stream=None):
    """A small beam search: prompts, then steps of fork, append, attention; one
    compaction on the way.  Returns what is needed to check it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    B, Hq, Hkv, D, page, block, M, P = 6, 8, 2, 128, 16, 8, 12, 90
    pages = lambda: torch.zeros((P, page, Hkv, D), dtype=torch.int8, device=DEV).view(  # noqa: E731
        cache_ref.TORCH_CODE[kind])
    scales = lambda: torch.full((P, page // block, Hkv), math.nan, device=DEV)  # noqa: E731
    kp, vp, ks, vs = pages(), pages(), scales(), scales()
    pools = [kp, vp, ks, vs]
    table = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    history = [[] for _ in range(B)]  # rows of each slot
    outs = []
    for t in range(steps):
        n = 37 if t == 0 else 1
        parents = torch.arange(B, device=DEV, dtype=torch.int32)
        if t:
            parents = torch.randint(0, B, (B,), generator=g, device=DEV, dtype=torch.int32)
        new = torch.full((B,), n, dtype=torch.int32, device=DEV)
        if t == 0:
            new -= torch.arange(B, dtype=torch.int32, device=DEV) * 5
        k = torch.randn((B, n, Hkv, D), generator=g, device=DEV).to(DT[dtype])
        v = torch.randn((B, n, Hkv, D), generator=g, device=DEV).to(DT[dtype])
        q = torch.randn((B, 1, Hq, D), generator=g, device=DEV).to(DT[dtype])
        table, lens, refs, status = attn.attn_pages_fork(pools, table, lens, refs, parents, page,
                                                         new_tokens=new, stream=stream)
        if t == steps // 2:
            table, refs, remap, live = attn.attn_pages_compact(pools, table, refs, stream=stream)
        attn.attn_cache_append(k, v, kp, vp, ks, vs, table, lens, seqlens_new=new, stream=stream)
        with torch.cuda.stream(stream) if stream else torch.cuda.device(0):
            lens = lens + new
        outs.append((q, *attn.attn_fwd_paged_q8(q, kp, vp, ks, vs, table, lens, stream=stream)))
        history = [list(history[p]) + [(k[i, :m], v[i, :m])] for i, (p, m) in
                   enumerate(zip(parents.tolist(), new.tolist()))]
        yield outs[-1], history, lens, (kp, vp, ks, vs, table, refs, status)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_serving_steps_together(kind):
    for (q, o, lse), history, lens, (kp, vp, ks, vs, table, refs, status) in serve(20, kind=kind):
        assert status[:2].tolist() == [0, 0]
        page = kp.shape[1]
        live = torch.bincount(table[table >= 0].long(), minlength=len(refs)).to(torch.int32)
        assert torch.equal(live, refs)
        k = cache_ref.gather(cache_ref.as_values(bits(kp).reshape(kp.shape), np.nan_to_num(ks.cpu().numpy()), kind),
                             table.cpu().numpy(), lens.cpu().numpy(), table.shape[1] * page)
        v = cache_ref.gather(cache_ref.as_values(bits(vp).reshape(vp.shape), np.nan_to_num(vs.cpu().numpy()), kind),
                             table.cpu().numpy(), lens.cpu().numpy(), table.shape[1] * page)
        for b, rows in enumerate(history):
            n = int(lens[b])
            for got, i in ((k, 0), (v, 1)):
                want = torch.cat([r[i] for r in rows]).double().cpu().numpy()
                assert want.shape[0] == n
                # a value is within one step of its block's scale (int8) or half a step of its own
                # (e4m3: 2^-4) and of the subnormals; scales are at most 2 / qmax of the largest |x|
                big = np.abs(want).max() * (2 / cache_ref.QMAX[kind] if kind == "int8" else 2.0 ** -16)
                slack = 0 if kind == "int8" else 2.0 ** -4
                assert (np.abs(got[b, :n] - want) <= big + slack * np.abs(want)).all()
        ro, rl, to, tl = attention_bounds(q.double().cpu().numpy(), k, v, q.shape[0], q.shape[2], kp.shape[2],
                                          1, k.shape[1], 128, 128, lens.cpu().numpy(), None, 0,
                                          128 ** -0.5, 0, "bf16")
        assert (np.abs(o.double().cpu().numpy() - ro) <= to).all()
        assert (np.abs(lse.double().cpu().numpy() - rl) <= tl).all()


def test_serving_steps_on_a_stream():
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    a = [(o.clone(), lse.clone()) for (_, o, lse), *_ in serve(8)]
    torch.cuda.synchronize()
    b = []
    with torch.cuda.stream(st):
        b = [(o, lse) for (_, o, lse), *_ in serve(8, stream=st)]
    st.synchronize()
    for (x, y), (z, w) in zip(a, b):
        assert torch.equal(x, z) and torch.equal(y, w)


def test_two_captured_graphs_replay_as_the_eager_calls():
    """One decoding step captured twice (two graphs, each with its workspaces)
    and replayed in turn on fresh inputs gives the eager calls' bits."""
    g = np.random.default_rng(40)

    def make(seed):
        g = np.random.default_rng(seed)
        c = Cache(g, [500, 33, 200], 16, 16, 2, 128, 128, "int8", max_pages=40, spare=40)
        refs = np.bincount(c.table[c.table >= 0], minlength=len(c.codes[0])).astype(np.int32)
        pools = list(c.gpu())
        x = [torch.from_numpy(g.standard_normal((3, 1, h, 128)).astype(np.float32)).bfloat16().to(DEV)
             for h in (2, 2, 8)]
        return pools, i32(c.table), i32(c.lens), i32(refs), x

    one = i32([1, 1, 1])

    def step(pools, table, lens, refs, x, parents):
        t, n, r, s = attn.attn_pages_fork(pools, table, lens, refs, parents, 16, new_tokens=one)
        attn.attn_cache_append(x[0], x[1], *pools, t, n)
        o, lse = attn.attn_fwd_paged_q8(x[2], *pools, t, n + 1)
        t2, r2, m, live = attn.attn_pages_compact(pools, t, r)
        return t, r, s, o, lse, t2, r2, m, live

    par = i32([2, 0, 0])
    states = [make(50), make(51)]
    want = []
    for seed in (50, 51):
        args = make(seed)
        want.append([x.clone() for x in step(*args, par)] + [p.clone() for p in args[0]])
    fresh = [make(50), make(51)]
    step(*make(52), par)  # first calls happen outside a capture
    torch.cuda.synchronize()
    graphs, outs = [], []
    for args in states:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(*args, par))
        graphs.append(gr)
    for _ in range(2):
        for k in (0, 1):
            for a, b in zip(states[k][0], fresh[k][0]):
                a.copy_(b)
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in (0, 1):
            for a, b in zip(list(outs[k]) + states[k][0], want[k]):
                assert torch.equal(a.view(torch.uint8) if a.dim() else a, b.view(torch.uint8) if b.dim() else b)


def test_offsets_past_32_bits():
    """Pools of more than 4 GB: pages at their end are read and written as those of a
    small pool are (attention by both paths, appending, copying, forking)."""
    g = np.random.default_rng(41)
    page, Hkv, D, P = 64, 8, 256, 33000          # 131072 bytes a page
    c = Cache(g, [500, 64, 130], page, 16, Hkv, D, D, "int8", max_pages=9)
    small = list(c.gpu())
    n = small[0].shape[0]
    big = [torch.empty((P,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV) for t in small]
    off = P - n
    for t, b in zip(small, big):
        b[off:] = t
    table = i32(c.table)
    far = torch.where(table >= 0, table + off, table)
    lens, new = i32(c.lens), i32([5, 64, 3])
    refs = torch.bincount(table[table >= 0].long(), minlength=n).to(torch.int32)
    far_refs = torch.cat([torch.ones(off, dtype=torch.int32, device=DEV), refs])
    # a fork that copies pages (and finds its free ones at the end), rows behind them
    par = i32([0, 0, 1, 2])
    t1, l1, r1, s1 = attn.attn_pages_fork(small, table, lens, refs, par, page)
    t2, l2, r2, s2 = attn.attn_pages_fork(big, far, lens, far_refs, par, page)
    assert torch.equal(torch.where(t1 >= 0, t1 + off, t1), t2) and s1[3] > 0 and torch.equal(s1, s2)
    x = [torch.randn((4, 7, Hkv, D), device=DEV).bfloat16() for _ in range(2)]
    room = i32([7, 3, 0, 5])
    attn.attn_cache_append(*x, *small, t1, l1, seqlens_new=room)
    attn.attn_cache_append(*x, *big, t2, l2, seqlens_new=room)
    for Q in (1, 40):
        q = torch.randn((4, Q, 2 * Hkv, D), device=DEV).bfloat16()
        a = attn.attn_fwd_paged_q8(q, *small, t1, l1 + room)
        b = attn.attn_fwd_paged_q8(q, *big, t2, l2 + room)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    src, dst = i32([0, 2]), i32([n - 1, n - 2])
    attn.attn_pages_copy(small, small, src, dst)
    attn.attn_pages_copy(big, big, src + off, dst + off)
    for t, b in zip(small, big):
        assert torch.equal(t.view(torch.uint8), b[off:].contiguous().view(torch.uint8))


def test_attention_at_the_last_key_that_32_bits_count():
    """A sequence of 2^31 - 64 keys (a table that names one page again and again):
    the last tile ends behind the keys and, counted in 32 bits, behind 2^31.  Every
    score is -30 and every value 3, so the output is 3.  A thread adds up the terms
    of 2^24 tiles over at least 256 shares in fp32, 2^16 additions: its sum of
    probabilities is off by 2^16 * 2^-24 = 2^-8 of itself at most (the sums of values
    are of equal powers of two, and exact), the merge of a few hundred terms by
    2^-14, and fp16 rounds by 2^-11.  Keys that do not exist would score 0, e^30
    above the others."""
    page, D, K = 64, 16, (1 << 31) - 64
    kp = torch.full((1, page, 1, D), 2, dtype=torch.int8, device=DEV)
    vp = torch.full((1, page, 1, D), 3, dtype=torch.int8, device=DEV)
    one = torch.ones((1, 1, 1), device=DEV)
    table = torch.zeros((1, K // page), dtype=torch.int32, device=DEV)
    q = torch.full((1, 1, 1, D), -1., dtype=torch.float16, device=DEV)   # score -32, x scale
    scale = 30. / 32.
    for lens, window in ((K, 0), (K, 1000), (K - 37, 0)):
        o, lse = attn.attn_fwd_paged_q8(q, kp, vp, one, one, table, i32([lens]), window=window,
                                        scale=scale)
        n = min(lens, window or lens)
        off = 2. ** -8 + 2. ** -14
        assert abs(o.double().mean().item() - 3.) <= 3 * (off + 2. ** -11) and o.std() == 0
        assert abs(lse.item() - (math.log(n) - 30.)) <= 1.01 * off + 1e-4   # (fp32 near 30: 2e-6)


def test_calls_from_two_threads():
    """Two threads, a stream each, append, attend and fork at the same time, each on
    a cache of its own: what the calls give one after the other."""
    def work(seed, stream):
        g = np.random.default_rng(seed)
        c = Cache(g, [300, 64, 0, 1000 + seed], 64, 16, 4, 128, 128, "int8", max_pages=20)
        x = [torch.from_numpy(g.standard_normal((4, 9, 4, 128), np.float32)).to(DEV).bfloat16()
             for _ in range(2)]
        q = torch.from_numpy(g.standard_normal((4, 9, 8, 128), np.float32)).to(DEV).bfloat16()
        pools, table, lens = list(c.gpu()), i32(c.table), i32(c.lens)
        refs = torch.zeros(pools[0].shape[0], dtype=torch.int32, device=DEV)
        refs[table[table >= 0].long()] = 1
        parents, new = i32([0, 1, 2, 3]), i32([1, 0, 3, 2])
        torch.cuda.current_stream().synchronize()
        out = []
        with torch.cuda.stream(stream):
            for _ in range(20):
                t, n, r, s = attn.attn_pages_fork(pools, table, lens, refs, parents, 64, new_tokens=new)
                attn.attn_cache_append(*x, *pools, t, n, seqlens_new=new)
                for Q in (1, 9):
                    out += attn.attn_fwd_paged_q8(q[:, :Q].contiguous(), *pools, t, n + new)
                out += [t, n, r, s]
        stream.synchronize()
        return out

    streams = [torch.cuda.Stream() for _ in range(2)]
    alone = [work(seed, streams[0]) for seed in (50, 51)]
    with concurrent.futures.ThreadPoolExecutor(2) as pool:
        both = list(pool.map(work, (50, 51), streams))
    for a, b in zip(alone, both):
        assert len(a) == len(b) and all(np.array_equal(bits(x), bits(y)) for x, y in zip(a, b))


def test_attention_without_lse():
    g = np.random.default_rng(42)
    c = Cache(g, [300, 7], 64, 16, 2, 128, 128, "e4m3")
    args = (torch.randn((2, 1, 8, 128), device=DEV).half(), *c.gpu(), i32(c.table), i32(c.lens))
    o, lse = attn.attn_fwd_paged_q8(*args)
    o2, none = attn.attn_fwd_paged_q8(*args, want_lse=False)
    assert none is None and torch.equal(o, o2)


def test_launch_count_moves():
    n = attn.kernel_launches()
    for _ in serve(1):
        pass
    assert attn.kernel_launches() - n >= 4
    assert attn.device_status() == (0, 0)
