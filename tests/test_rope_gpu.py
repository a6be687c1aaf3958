"""The position rotation and the rotated appends on the GPU against their plain
restatement (tests/rope_ref.py, tests/cache_ref.py): bit for bit where the roundings
are defined (fp32, one by one), and within derived bounds of 64 bits."""
import math

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn
from tests import cache_ref, rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}  # half a step; fp32 results are not rounded again


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def rows(g, shape, dtype):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(DT[dtype])


def as_np(t):
    return t.float().cpu().numpy()


def rounded(y, dtype):
    return torch.from_numpy(np.ascontiguousarray(y, dtype=np.float32)).to(DT[dtype])


def same(got, want):
    """Bit for bit, NaN as NaN."""
    a, b = got.cpu(), want.cpu()
    nan = torch.isnan(b.float())
    assert torch.equal(torch.isnan(a.float()), nan)
    u = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[a.element_size()]
    assert torch.equal(a.contiguous().view(u)[~nan], b.contiguous().view(u)[~nan])


# (B, N, Hq, Hkv, D, rot): single rows, odd sizes, widths of every vector size, wide heads
SHAPES = [(1, 1, 1, 1, 2, 2), (2, 3, 4, 2, 64, 64), (1, 129, 6, 2, 80, 40), (3, 5, 5, 1, 112, 56),
          (2, 33, 8, 8, 128, 128), (1, 7, 3, 3, 33, 14), (1, 2, 40, 8, 256, 64), (2, 4, 2, 1, 512, 512),
          (1, 65, 64, 4, 96, 48), (2, 9, 3, 1, 72, 0), (1, 3, 2, 2, 511, 510)]


@pytest.mark.parametrize("pairs", ["half", "adjacent"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope(shape, dtype, pairs):
    B, N, Hq, Hkv, D, rot = shape
    g = np.random.default_rng(sum(shape))
    q, k = rows(g, (B, N, Hq, D), dtype), rows(g, (B, N, Hkv, D), dtype)
    cos, sin = rope_ref.angles(N + 3, rot)
    pos = g.integers(-1, N + 4, (B, N))  # some outside the table
    for positions in (None, pos):
        at = (np.broadcast_to(np.arange(N), (B, N)) if positions is None else pos).reshape(-1)
        for inverse, call in ((False, attn.attn_rope), (True, attn.attn_rope_bwd)):
            got = call(q.to(DEV), k.to(DEV), torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV),
                       positions=None if positions is None else i32(pos), pairs=pairs)
            for y, x, H in ((got[0], q, Hq), (got[1], k, Hkv)):
                flat = as_np(x).reshape(-1, H, D)
                same(y.view(-1, H, D), rounded(rope_ref.rotate(flat, cos, sin, at, pairs, inverse, np.float32), dtype))
                # 64 bits: a product and a sum round by 2^-24 of the terms each, the type by half a step
                ref = rope_ref.rotate(flat, cos, sin, at, pairs, inverse)
                terms = np.abs(flat).astype(np.float64)
                a, b = rope_ref.columns(D, rot, pairs)
                terms[..., a] = terms[..., b] = terms[..., a] + terms[..., b]
                bound = 2.0 ** -23 * terms * (1 + 2.0 ** -20) + HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -10) + 2.0 ** -25
                err = np.abs(as_np(y).reshape(-1, H, D) - ref)
                assert np.all((err <= bound) | np.isnan(ref))


def test_rope_special_values():
    x = torch.tensor([[[float("inf"), 1.0, float("nan"), 2.0, 0.0, -0.0, 1e38, 3e38]]]).to(DEV)
    cos, sin = rope_ref.angles(4, 8)
    y, none = attn.attn_rope(x, None, torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV),
                             positions=i32([3]), pairs="adjacent")
    assert none is None
    with np.errstate(invalid="ignore", over="ignore"):
        same(y, torch.from_numpy(rope_ref.rotate(as_np(x), cos, sin, [3], "adjacent", dtype=np.float32)))


def test_rope_without_a_table_row():
    x = torch.ones((2, 1, 4), device=DEV)
    none = torch.empty((0, 1), device=DEV)
    y, _ = attn.attn_rope(x, None, none, none)
    assert torch.isnan(y[..., :2]).all() and (y[..., 2:] == 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_of_views_in_place_and_on_streams(dtype):
    B, N, Hq, Hkv, D = 2, 37, 6, 2, 64
    g = np.random.default_rng(3)
    cos, sin = (torch.from_numpy(t).to(DEV) for t in rope_ref.angles(N, D))
    for odd in (0, 3):  # the second: rows that are no multiple of a vector apart, and unaligned
        fused = rows(g, (B, N, (Hq + 2 * Hkv) * D + odd), dtype).to(DEV)
        q = fused[..., odd: odd + Hq * D].unflatten(-1, (Hq, D))
        k = fused[..., odd + Hq * D: odd + (Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        was = fused.clone()
        want = attn.attn_rope(q.contiguous(), k.contiguous(), cos, sin)
        got = attn.attn_rope(q, k, cos, sin)
        same(got[0], want[0]), same(got[1], want[1])
        assert torch.equal(fused, was)
        p, r = q.contiguous(), k.contiguous()
        back = attn.attn_rope(p, r, cos, sin, p, r)
        assert back[0] is p and back[1] is r
        same(p, want[0]), same(r, want[1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = attn.attn_rope(q, k, cos, sin, stream=side)
        side.synchronize()
        same(got[0], want[0]), same(got[1], want[1])
    with pytest.raises(attn.AttnError, match="overlaps"):  # k's output in q's rows
        attn.attn_rope(p, r, cos, sin, None, p.view(-1)[: r.numel()].view(r.shape))


def test_rope_gradient_against_differences():
    # the rotation is linear: a central difference of sum(dy * rope(x)) along d is its
    # derivative but for roundings, each 2^-23 of the terms; steps of 1 keep them that size
    B, N, H, D = 2, 19, 3, 48
    g = np.random.default_rng(8)
    x, dy, d = (torch.from_numpy(g.integers(-8, 9, (B, N, H, D)).astype(np.float32)).to(DEV) for _ in range(3))
    cos, sin = (torch.from_numpy(t).to(DEV) for t in rope_ref.angles(N, 32))
    for pairs in ("half", "adjacent"):
        dx, _ = attn.attn_rope_bwd(dy, None, cos, sin, pairs=pairs)
        up, _ = attn.attn_rope(x + d, None, cos, sin, pairs=pairs)
        down, _ = attn.attn_rope(x - d, None, cos, sin, pairs=pairs)
        want = float((dy.double() * (up.double() - down.double())).sum()) / 2
        got = float((dx.double() * d.double()).sum())
        terms = float((dy.abs().double() * (x.abs() + d.abs()).double()).sum())
        assert abs(got - want) <= 2.0 ** -21 * terms


# ------------------------------------------------------------------ appends

class Step:
    """New rows of a batch, a table of their pages, and what lies there."""

    def __init__(self, g, lens, new, page, Hq, Hkv, D, Dv, rot, dtype, packed, positions=False, fused=False,
                 slack=0, max_pages=None, N=None):
        self.B, self.N = len(lens), N or max(1, max(new))
        self.lens, self.new, self.page, self.packed, self.dtype = lens, new, page, packed, dtype
        need = [-(-(a + b) // page) for a, b in zip(lens, new)]
        self.M = max_pages or max(1, max(need))
        P = sum(need) + 2
        order = g.permutation(P)
        self.table = np.full((self.B, self.M), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, : min(n, self.M)] = order[at: at + min(n, self.M)]
            at += n
        self.P, self.Hkv, self.D, self.Dv = P, Hkv, D, Dv
        lead = (sum(new) + slack,) if packed else (self.B, self.N)
        if fused:
            x = rows(g, lead + ((Hq + Hkv) * D + Hkv * Dv,), dtype)
            self.q, self.k, self.v = (t.unflatten(-1, (-1, w)) for t, w in zip(
                x.split([Hq * D, Hkv * D, Hkv * Dv], -1), (D, D, Dv)))
        else:
            self.q, self.k, self.v = (rows(g, lead + (h, w), dtype) for h, w in ((Hq, D), (Hkv, D), (Hkv, Dv)))
        total = max(a + b for a, b in zip(lens, new)) + 5
        self.cos, self.sin = rope_ref.angles(total, rot)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.positions = g.integers(0, total, lead).astype(np.int32) if positions else None

    def row(self, b, i):
        return int(self.cu[b]) + i if self.packed else (b, i)

    def turned(self, pairs):
        """[n, H, D] fp32 rows of q and of k, and v, of each sequence."""
        for b, n in enumerate(self.new):
            at = slice(int(self.cu[b]), int(self.cu[b]) + n) if self.packed else (b, slice(0, n))
            pos = self.lens[b] + np.arange(n) if self.positions is None else self.positions[at]
            yield (*(rope_ref.rotate(as_np(t[at]), self.cos, self.sin, pos, pairs, dtype=np.float32)
                     for t in (self.q, self.k)), as_np(self.v[at]))

    def angles(self):
        if self.cos.shape[1] == 0:
            return None, None
        return torch.from_numpy(self.cos).to(DEV), torch.from_numpy(self.sin).to(DEV)

    def call(self, cache, pairs, q=True, **kw):
        """The framework's call over `cache` (2 pools, or 4 tensors of an 8-bit one)."""
        dev = lambda t: t.to(DEV) if t.is_contiguous() else t._base.to(DEV).as_strided(t.shape, t.stride(), t.storage_offset())  # noqa: E731
        x = [dev(self.q) if q else None, dev(self.k), dev(self.v)]
        kw = dict(kw, pairs=pairs, positions=None if self.positions is None else i32(self.positions))
        where = (*cache, i32(self.table), i32(self.lens))
        eight = "_q8" if len(cache) == 4 else ""
        if self.packed:
            f = getattr(attn, f"attn_rope_append{eight}_varlen")
            return f(*x, i32(self.cu), self.N, *self.angles(), *where, **kw)
        return getattr(attn, f"attn_rope_append{eight}")(*x, *self.angles(), *where, seqlens_new=i32(self.new), **kw)

    def check_q(self, got, pairs):
        for b, (y, _, _) in enumerate(self.turned(pairs)):
            n = self.new[b]
            if self.packed:
                same(got[int(self.cu[b]): int(self.cu[b]) + n], rounded(y, self.dtype))
            else:
                same(got[b, :n], rounded(y, self.dtype))
                assert not got[b, n:].float().any() and not torch.signbit(got[b, n:].float()).any()


APPENDS = [
    # lens, new, page, Hq, Hkv, D, Dv, rot
    ([0], [1], 1, 1, 1, 16, 16, 16),
    ([5, 0, 63, 64, 200], [1, 1, 1, 1, 1], 64, 8, 2, 64, 64, 64),
    ([0, 17, 3], [40, 0, 129], 16, 6, 2, 128, 128, 128),
    ([7, 8, 9], [9, 8, 7], 8, 3, 1, 80, 48, 40),
    ([31, 0], [2, 70], 32, 5, 5, 33, 20, 14),
    ([100, 1], [3, 3], 128, 16, 4, 112, 112, 56),
    ([0, 4], [6, 5], 4, 2, 2, 256, 512, 0),
]


@pytest.mark.parametrize("variant", ["plain", "packed", "positions", "fused", "packed fused"])
@pytest.mark.parametrize("dtype,pairs", [("bf16", "half"), ("f16", "adjacent"), ("f32", "half")])
@pytest.mark.parametrize("case", APPENDS)
def test_append(case, dtype, pairs, variant):
    lens, new, page, Hq, Hkv, D, Dv, rot = case
    g = np.random.default_rng(len(lens) + D)
    st = Step(g, lens, new, page, Hq, Hkv, D, Dv, rot, dtype, "packed" in variant, variant == "positions",
              "fused" in variant)
    kp = torch.full((st.P, page, Hkv, D), math.nan, dtype=DT[dtype], device=DEV)
    vpg = torch.full((st.P, page, Hkv, Dv), math.nan, dtype=DT[dtype], device=DEV)
    got = st.call((kp, vpg), pairs)
    st.check_q(got, pairs)
    want_k, want_v = torch.full(kp.shape, math.nan, dtype=kp.dtype), torch.full(vpg.shape, math.nan, dtype=kp.dtype)
    for b, (_, k, v) in enumerate(st.turned(pairs)):
        for i in range(new[b]):
            j = lens[b] + i
            want_k[st.table[b, j // page], j % page] = rounded(k[i], dtype)
            want_v[st.table[b, j // page], j % page] = rounded(v[i], dtype)
    same(kp, want_k), same(vpg, want_v)
    # without q the same rows go in
    kp2, vp2 = torch.full_like(kp, math.nan), torch.full_like(vpg, math.nan)
    assert st.call((kp2, vp2), pairs, q=False) is None
    same(kp2, want_k), same(vp2, want_v)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kind", ["none", "int8", "e4m3"])
def test_rows_without_a_place_are_dropped(kind, packed):
    g = np.random.default_rng(1)
    lens, new, page, H, D = [3, 14, 0, 9], [20, 6, 4, 2], 8, 2, 32
    st = Step(g, lens, new, page, 2, H, D, D, D, "bf16", packed, max_pages=2, slack=3)
    st.table[2, 0] = -1          # no page
    st.table[3, 1] = st.P        # past the pool
    P = st.P
    if kind == "none":
        cache = [torch.zeros((P, page, H, D), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        want = [torch.zeros((P, page, H, D)) for _ in "kv"]
    else:
        cache = [torch.zeros((P, page, H, D), dtype=cache_ref.TORCH_CODE[kind], device=DEV) for _ in "kv"]
        cache += [torch.ones((P, 2, H), device=DEV) for _ in "kv"]
        want = [(np.zeros((P, page, H, D), np.uint8), np.ones((P, 2, H))) for _ in "kv"]
    canary = torch.full(st.q.shape, 7.0, dtype=st.q.dtype, device=DEV)
    got = st.call(cache, "half", q_out=canary)
    st.check_q(got, "half")
    if packed:  # rows behind the last sequence
        assert (got[sum(new):] == 7).all()
    turned = list(st.turned("half"))
    if kind == "none":
        for b in range(4):
            for i in range(new[b]):
                j = lens[b] + i
                pg = st.table[b, j // page] if j < 2 * page else -1
                if 0 <= pg < P:
                    for w in (0, 1):
                        want[w][pg, j % page] = torch.from_numpy(turned[b][1 + w][i])
        for x, y in zip(cache, want):
            same(x, y.to(torch.bfloat16))
    else:
        for w in (0, 1):
            cache_ref.append([t[1 + w] for t in turned], lens, new, st.table, *want[w], kind)
            assert np.array_equal(cache[w].view(torch.uint8).cpu().numpy(), want[w][0])
            assert np.array_equal(cache[2 + w].cpu().numpy(), want[w][1].astype(np.float32))


@pytest.mark.parametrize("variant", ["plain", "packed", "positions", "fused"])
@pytest.mark.parametrize("kind,dtype,pairs", [("int8", "bf16", "half"), ("e4m3", "f16", "adjacent"),
                                              ("int8", "f32", "adjacent"), ("e4m3", "bf16", "half")])
@pytest.mark.parametrize("case", [c for c in APPENDS if c[0] != [0, 4]] + [([0, 61], [200, 70], 128, 4, 2, 128, 128, 128)])
def test_append_q8(case, kind, dtype, pairs, variant):
    lens, new, page, Hq, Hkv, D, Dv, rot = case
    g = np.random.default_rng(len(lens) + D)
    st = Step(g, lens, new, page, Hq, Hkv, D, Dv, rot, dtype, variant == "packed", variant == "positions",
              variant == "fused")
    for block in sorted({1, max(1, page // 4), page}):
        nb = page // block
        codes, scales = [], []
        for W in (D, Dv):
            c = g.integers(0, 256, (st.P, page, Hkv, W), dtype=np.uint8)
            c[(c & 127) == 127] = 126  # no NaN code
            c[c == 128] = 129
            codes.append(c)
            scales.append(2.0 ** g.integers(-12, -2, (st.P, nb, Hkv)))
        cache = [torch.from_numpy(c).to(DEV).view(cache_ref.TORCH_CODE[kind]) for c in codes]
        cache += [torch.from_numpy(s).float().to(DEV) for s in scales]
        st.check_q(st.call(cache, pairs), pairs)
        turned = list(st.turned(pairs))
        for w in (0, 1):
            cache_ref.append([t[1 + w] for t in turned], lens, new, st.table, codes[w], scales[w], kind)
            assert np.array_equal(cache[w].view(torch.uint8).cpu().numpy(), codes[w])
            assert np.array_equal(cache[2 + w].cpu().numpy(), scales[w].astype(np.float32))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_q8_poisoned_blocks(kind):
    # an infinite key, a NaN value and a position past the table each poison their block, and no other
    page, H, D = 16, 1, 16
    cos, sin = (torch.from_numpy(t).to(DEV) for t in rope_ref.angles(30, D))
    x = torch.ones((3, 1, 1, D), device=DEV)
    v = torch.ones((3, 1, 1, D), device=DEV)
    x[0, 0, 0, 3], v[1, 0, 0, 2] = math.inf, math.nan
    cache = [torch.zeros((3, page, H, D), dtype=cache_ref.TORCH_CODE[kind], device=DEV) for _ in "kv"]
    cache += [torch.ones((3, 1, H), device=DEV) for _ in "kv"]
    attn.attn_rope_append_q8(None, x, v, cos, sin, *cache, i32([[0], [1], [2]]), i32([0, 0, 0]),
                             positions=i32([[1], [2], [30]]))
    assert torch.isnan(cache[2]).flatten().tolist() == [True, False, True]
    assert torch.isnan(cache[3]).flatten().tolist() == [False, True, False]
    assert not cache[0][0].float().any() and not cache[1][1].float().any()


def test_append_without_rotation_is_the_plain_append():
    # rot 0 into the 8-bit cache: what attn_cache_append writes, for every vector size
    g = np.random.default_rng(9)
    for D in (64, 56, 33):
        st = Step(g, [5, 30], [40, 3], 32, 2, 2, D, D, 0, "bf16", False)
        caches = []
        for _ in range(2):
            caches.append([torch.zeros((st.P, 32, 2, D), dtype=torch.int8, device=DEV) for _ in "kv"] +
                          [torch.full((st.P, 4, 2), 2.0 ** -9, device=DEV) for _ in "kv"])
        st.call(caches[0], "half", q=False)
        attn.attn_cache_append(st.k.to(DEV), st.v.to(DEV), *caches[1], i32(st.table), i32(st.lens),
                               seqlens_new=i32(st.new))
        for a, b in zip(*caches):
            assert torch.equal(a, b)


def test_append_past_32_bits_of_offsets():
    # pools of more than 2^31 elements: rows go to their last page
    page, H, D = 64, 8, 128
    P = (1 << 31) // (page * H * D) + 2
    kp, vpg = (torch.zeros((P, page, H, D), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    g = np.random.default_rng(4)
    q, k, v = (rows(g, (1, 2, h, D), "bf16").to(DEV) for h in (H, H, H))
    cos, sin = (torch.from_numpy(t).to(DEV) for t in rope_ref.angles(100, D))
    attn.attn_rope_append(q, k, v, cos, sin, kp, vpg, i32([[P - 1]]), i32([62]))
    same(vpg[P - 1, 62:], v[0])
    at = rope_ref.rotate(as_np(k[0]), as_np(cos), as_np(sin), [62, 63], "half", dtype=np.float32)
    same(kp[P - 1, 62:], rounded(at, "bf16"))
    assert int(torch.count_nonzero(kp)) == int(torch.count_nonzero(kp[P - 1])) and not vpg[: P - 1].any()


def test_append_in_a_graph():
    # captured once, replayed over changed lengths and rows
    g = np.random.default_rng(2)
    B, H, D, page = 3, 2, 64, 16
    q, k, v = (rows(g, (B, 1, h, D), "bf16").to(DEV) for h in (4, H, H))
    cos, sin = (torch.from_numpy(t).to(DEV) for t in rope_ref.angles(64, D))
    table, lens = i32(np.arange(6).reshape(3, 2)), i32([0, 5, 14])
    pools = [torch.zeros((6, page, H, D), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        attn.attn_rope_append(q, k, v, cos, sin, *pools, table, lens, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.attn_rope_append(q, k, v, cos, sin, *pools, table, lens, out)
    for step in range(3):
        lens += 1
        k.copy_(rows(g, (B, 1, H, D), "bf16"))
        other = [p.clone() for p in pools]
        graph.replay()
        want = attn.attn_rope_append(q, k, v, cos, sin, *other, table, lens)
        same(out, want)
        for a, b in zip(pools, other):
            same(a, b)


# Many rows go through shared memory, by other kernels than few.  Each must give what the
# calls for a few of its rows at a time give, bit for bit.

MANY = [(4, 1501, 8, 4, 96, 48), (1, 4099, 3, 1, 64, 64), (2, 1301, 40, 8, 256, 64), (1, 401, 100, 4, 512, 512),
        (3, 2001, 6, 2, 80, 40), (1, 6007, 14, 2, 72, 24), (3, 4001, 8, 4, 96, 48),
        (1, 20011, 3, 1, 128, 128)]


@pytest.mark.parametrize("dtype,pairs", [("bf16", "half"), ("f16", "adjacent"), ("f32", "half"), ("f32", "adjacent")])
@pytest.mark.parametrize("shape", MANY)
def test_rope_of_many_rows(shape, dtype, pairs):
    B, N, Hq, Hkv, D, rot = shape
    g = np.random.default_rng(sum(shape))
    x = rows(g, (B, N, (Hq + Hkv) * D), dtype).to(DEV)
    q, k = (t.unflatten(-1, (-1, D)) for t in x.split([Hq * D, Hkv * D], -1))
    cos, sin = (torch.from_numpy(t).to(DEV) for t in rope_ref.angles(N, rot))
    pos = i32(g.integers(-1, N + 1, (B, N)))
    for f in (attn.attn_rope, attn.attn_rope_bwd):
        got = f(q, k, cos, sin, positions=pos, pairs=pairs)
        only = f(q, None, cos, sin, positions=pos, pairs=pairs)
        same(only[0] if isinstance(only, tuple) else only, got[0])
        for a in range(0, N, 700):
            for b in range(B):
                at = (slice(b, b + 1), slice(a, min(N, a + 700, a + 311000 // (Hq * D) + 1)))
                want = f(q[at], k[at], cos, sin, positions=pos[at].contiguous(), pairs=pairs)
                same(got[0][at], want[0]), same(got[1][at], want[1])
    # in place
    q, k = q.contiguous(), k.contiguous()
    want = attn.attn_rope(q, k, cos, sin, positions=pos, pairs=pairs)
    attn.attn_rope(q, k, cos, sin, q, k, positions=pos, pairs=pairs)
    same(q, want[0]), same(k, want[1])


# lens, new, page, Hq, Hkv, D, Dv, rot
MANY_APPENDS = [([0, 70, 3000, 5], [3001, 0, 1400, 1], 64, 32, 8, 128, 128, 128),
                ([1, 16, 99], [2001, 2000, 3], 16, 4, 3, 96, 64, 48),
                ([7] * 40, [301] * 20 + [17] * 20, 128, 8, 2, 128, 256, 64)]


def one_sequence(st, b, n0, n1):
    """Rows n0 .. n1 of sequence b as a batch of their own."""
    one = Step.__new__(Step)
    one.__dict__.update(st.__dict__)
    at = slice(int(st.cu[b]) + n0, int(st.cu[b]) + n1) if st.packed else (b, slice(n0, n1))
    one.q, one.k, one.v = (t[at].contiguous()[None] for t in (st.q, st.k, st.v))
    one.positions = None if st.positions is None else st.positions[at][None]
    one.packed, one.B, one.N = False, 1, n1 - n0
    one.lens, one.new, one.table = [st.lens[b] + n0], [n1 - n0], st.table[b: b + 1]
    return one


@pytest.mark.parametrize("variant", ["plain", "packed", "positions", "fused", "packed fused"])
@pytest.mark.parametrize("kind,dtype,pairs", [("none", "bf16", "half"), ("none", "f16", "adjacent"), ("none", "f32", "half"),
                                              ("int8", "bf16", "adjacent"), ("e4m3", "f16", "half"), ("int8", "f32", "half")])
@pytest.mark.parametrize("case", range(len(MANY_APPENDS)))
def test_append_of_many_rows(case, kind, dtype, pairs, variant):
    lens, new, page, Hq, Hkv, D, Dv, rot = MANY_APPENDS[case]
    g = np.random.default_rng(case)
    st = Step(g, lens, new, page, Hq, Hkv, D, Dv, rot, dtype, "packed" in variant, variant == "positions",
              "fused" in variant, slack=9 if "packed" in variant else 0)
    st.table[0, 2] = -1  # a page that is not there
    st.cos, st.sin = st.cos[:-40], st.sin[:-40]  # the longest sequence runs past the angles
    for block in ((0,) if kind == "none" else (16, page)):
        pools = []
        for _ in range(2):
            if kind == "none":
                pools.append([torch.full((st.P, page, Hkv, w), 3.0, dtype=DT[dtype], device=DEV) for w in (D, Dv)])
            else:
                pools.append([torch.full((st.P, page, Hkv, w), 5, dtype=torch.uint8, device=DEV).view(
                    cache_ref.TORCH_CODE[kind]) for w in (D, Dv)])
                pools[-1] += [torch.full((st.P, page // block, Hkv), 2.0 ** -9, device=DEV) for _ in "kv"]
        canary = torch.full(st.q.shape, 7.0, dtype=st.q.dtype, device=DEV)
        got = st.call(pools[0], pairs, q_out=canary)
        for b, n in enumerate(new):
            # (8-bit blocks take all their new rows at once)
            step = max(n, 1) if kind != "none" else max(1, 300000 // ((Hq + Hkv) * max(D, Dv)))
            for a in range(0, n, step):
                e = min(n, a + step)
                want = one_sequence(st, b, a, e).call(pools[1], pairs)
                c = int(st.cu[b])
                same(got[c + a: c + e] if st.packed else got[b, a:e], want[0])
            if not st.packed:
                assert not got[b, n:].float().any() and not torch.signbit(got[b, n:].float()).any()
        if st.packed:
            assert (got[sum(new):] == 7).all()
        for x, y in zip(*pools):
            same(x, y)
        again = [p.clone() for p in pools[0]]  # and without q, over what is there now
        st.call(pools[0], pairs, q=False)
        for b, n in enumerate(new):
            if n:
                one_sequence(st, b, 0, n).call(again, pairs, q=False)
        for x, y in zip(pools[0], again):
            same(x, y)


@pytest.mark.parametrize("kind", ["none", "e4m3"])
def test_many_rows_in_two_graphs_at_once(kind):
    # two captured appends over pools of their own, replayed on two streams at once, with rows
    # and lengths that change between replays
    g = np.random.default_rng(6)
    lens, new, page = [0] * 6, [2001, 300, 1, 777, 0, 1290], 64
    steps = [Step(g, lens, new, page, 16, 4, 128, 128, 128, "bf16", False) for _ in range(2)]
    keep, graphs = [], []
    for st in steps:
        if kind == "none":
            pools = [torch.zeros((st.P, page, 4, 128), dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        else:
            pools = [torch.zeros((st.P, page, 4, 128), dtype=cache_ref.TORCH_CODE[kind], device=DEV) for _ in "kv"]
            pools += [torch.zeros((st.P, 1, 4), device=DEV) for _ in "kv"]
        x = [t.to(DEV) for t in (st.q, st.k, st.v)]
        n, out = i32(new), torch.empty_like(x[0])
        f = attn.attn_rope_append if kind == "none" else attn.attn_rope_append_q8
        args = (*x, *st.angles(), *pools, i32(st.table), i32(lens))
        call = lambda f=f, args=args, out=out, n=n: f(*args, out, seqlens_new=n)  # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
        keep.append((x, n, out, pools, args, f))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        for x, n, out, pools, args, f in keep:
            n.copy_(i32(np.minimum(new, g.integers(0, 2002, 6))))
            x[1].copy_(torch.randn_like(x[1]))
            out.fill_(3)
            for p in pools:
                p.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for x, n, out, pools, args, f in keep:
            other = [torch.zeros_like(p) for p in pools]
            want = f(*x, *args[3:5], *other, *args[-2:], seqlens_new=n)
            same(out, want)
            for a, b in zip(pools, other):
                same(a, b)


@pytest.mark.parametrize("kind", ["none", "int8"])
def test_outputs_side_by_side(kind):
    # outputs that touch, without a byte in common, are taken
    g = np.random.default_rng(11)
    q, k, v = (rows(g, (2, 5, h, 64), "bf16").to(DEV) for h in (4, 2, 2))
    cos, sin = (torch.from_numpy(t).to(DEV) for t in rope_ref.angles(9, 64))
    want = attn.attn_rope(q, k, cos, sin)
    x = torch.empty(q.numel() + k.numel(), dtype=q.dtype, device=DEV)
    got = attn.attn_rope(q, k, cos, sin, x[: q.numel()].view(q.shape), x[q.numel():].view(k.shape))
    same(got[0], want[0]), same(got[1], want[1])
    got = attn.attn_rope(q, k, cos, sin, x[k.numel():].view(q.shape), x[: k.numel()].view(k.shape))
    same(got[0], want[0]), same(got[1], want[1])
    # q's rows, then k's pages, then the scales, v's pages, and q's again
    code = torch.bfloat16 if kind == "none" else torch.int8
    n, size = 2 * 16 * 2 * 64, code.itemsize
    at, parts = 0, []
    mem = torch.zeros(2 * q.numel() * 2 + 2 * n * size + 2 * 32, dtype=torch.uint8, device=DEV)
    for b, t, shape in ((q.numel() * 2, q.dtype, q.shape), (n * size, code, (2, 16, 2, 64)), (32, torch.float32, (2, 2, 2)),
                        (32, torch.float32, (2, 2, 2)), (n * size, code, (2, 16, 2, 64)), (q.numel() * 2, q.dtype, q.shape)):
        parts.append(mem[at: at + b].view(t).view(shape))
        at += b
    for out in (parts[0], parts[5]):
        where = (i32([[1], [0]]), i32([0, 3]))
        if kind == "none":
            y = attn.attn_rope_append(q, k, v, cos, sin, parts[1], parts[4], *where, out)
        else:
            y = attn.attn_rope_append_q8(q, k, v, cos, sin, parts[1], parts[4], *parts[2:4], *where, out)
        same(y, attn.attn_rope(q, None, cos, sin, positions=i32(np.arange(5) + [[0], [3]]))[0])


@pytest.mark.parametrize("kind,with_q", [("rows", True), ("none", True), ("e4m3", True), ("e4m3", False)])
def test_waits_that_run_out_are_reported(kind, with_q):
    # A wait for a copy gives up once the limit has passed.  The first stage of a warp, or of
    # a block, comes from global memory, hundreds of ns away, so with a limit of 1 ns some
    # wait runs out; the launch ends, and the next one is right.
    st = Step(np.random.default_rng(15), [0, 70, 3000, 5], [3001, 0, 1400, 1], 64, 32, 8, 128, 128, 128, "bf16", False)
    cos, sin = st.angles()
    q, k = st.q.to(DEV), st.k.to(DEV)

    def call():
        if kind == "rows":
            return list(attn.attn_rope(q, k, cos, sin))
        code = torch.bfloat16 if kind == "none" else cache_ref.TORCH_CODE[kind]
        pools = [torch.zeros((st.P, 64, 8, 128), dtype=code, device=DEV) for _ in "kv"]
        if kind != "none":
            pools += [torch.zeros((st.P, 1, 8), device=DEV) for _ in "kv"]
        y = st.call(pools, "half", q=with_q)
        return [y, *pools] if with_q else pools

    want = call()
    torch.cuda.synchronize()
    attn.device_status()
    before = attn.set_wait_limit(1)
    try:
        call()
        torch.cuda.synchronize()
        assert attn.device_status() == (4, 0x401)
    finally:
        attn.set_wait_limit(before)
    got = call()
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
    for a, b in zip(got, want):
        same(a, b)


@pytest.mark.parametrize("kind", ["none", "int8"])
def test_max_new_beyond_the_rows(kind):
    # max_new is a bound: one that no sequence can reach runs what a near one runs
    st = Step(np.random.default_rng(16), [0, 70], [1, 1023], 64, 32, 8, 128, 128, 128, "bf16", True)
    got, launches = [], []
    for st.N in (1024, 1 << 20):
        code = torch.bfloat16 if kind == "none" else cache_ref.TORCH_CODE[kind]
        pools = [torch.zeros((st.P, 64, 8, 128), dtype=code, device=DEV) for _ in "kv"]
        if kind != "none":
            pools += [torch.zeros((st.P, 1, 8), device=DEV) for _ in "kv"]
        before = attn.kernel_launches()
        got.append([st.call(pools, "half"), *pools])
        launches.append(attn.kernel_launches() - before)
    st.check_q(got[0][0], "half")
    for a, b in zip(*got):
        same(a, b)
    assert launches[0] == launches[1], launches


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_many_rows_without_a_rotation(dtype, packed):
    # rot 0: rows into pages of their type, and q, as they are
    lens, new, page, D, Dv = [0, 70, 5], [3001, 0, 1400], 64, 128, 64
    st = Step(np.random.default_rng(17), lens, new, page, 16, 8, D, Dv, 0, dtype, packed)
    pools = [torch.full((st.P, page, 8, w), 3.0, dtype=DT[dtype], device=DEV) for w in (D, Dv)]
    want = [p.cpu() for p in pools]
    got = st.call(pools, "half").cpu()
    for b, n in enumerate(new):
        at = slice(int(st.cu[b]), int(st.cu[b]) + n) if packed else (b, slice(0, n))
        same(got[at], st.q[at])
        j = lens[b] + np.arange(n)
        for w, x in zip(want, (st.k, st.v)):
            w[torch.from_numpy(st.table[b][j // page]).long(), torch.from_numpy(j % page)] = x[at]
    for p, w in zip(pools, want):
        same(p, w)
    x, _ = attn.attn_rope(st.q.to(DEV), None, None, None)
    same(x, st.q)
