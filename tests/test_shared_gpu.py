"""Attention over shared beginnings on the GPU, against the definition in 64 bits over
every sequence's own table, within bounds derived from the roundings."""
import concurrent.futures
import math

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}  # half a step of a rounding
GUARD = 4096


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Batch:
    """Groups of sequences over one pool.  Rows that no key is in hold NaN; the partly
    filled page at the end of a shared beginning is copied for every member."""

    def __init__(self, seed, sizes, pre, tails, Q, Hq, Hkv, D, Dv, page, dtype, alone=(), seqlens_q=None, spare=2,
                 short=()):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.sizes, self.pre, self.Q, self.Hq, self.Hkv, self.D, self.Dv = sizes, pre, Q, Hq, Hkv, D, Dv
        self.page, self.dtype = page, dtype
        group = np.repeat(np.arange(len(sizes)), sizes)
        lens = [pre[n] + t for n, t in zip(group, tails)] + list(alone)
        for b, n in short:
            lens[b] = n
        self.lens, self.B = np.asarray(lens, np.int64), len(lens)
        self.M = max(1, max(-(-int(n) // page) for n in [*lens, *pre, 1]))
        rows = []  # table entries: shared full pages by group, then the sequence's own
        at, firsts = 0, []
        for n in range(len(sizes)):
            firsts.append(at)
            at += pre[n] // page
        table = np.full((self.B, self.M), -1, np.int64)
        partial = []
        for b in range(self.B):
            full = pre[group[b]] // page if b < len(group) else 0
            need = -(-int(self.lens[b]) // page)
            table[b, :full] = np.arange(firsts[group[b]], firsts[group[b]] + full) if full else 0
            for e in range(full, need):
                table[b, e] = at
                at += 1
            if b < len(group) and pre[group[b]] % page and need > full:
                partial.append((b, full, pre[group[b]] % page))
        self.P = at + spare
        order = rng.permutation(self.P)
        self.table = np.where(table >= 0, order[np.maximum(table, 0)], -1)
        shape = (self.P, page, Hkv)
        self.k = torch.randn(shape + (D,), generator=g, device=DEV).to(DT[dtype])
        self.v = torch.randn(shape + (Dv,), generator=g, device=DEV).to(DT[dtype])
        # partly filled pages: equal contents for the members of a group
        first = {}
        for b, e, n in partial:
            src = first.setdefault(group[b], self.table[b, e])
            for t in (self.k, self.v):
                t[int(self.table[b, e]), :n] = t[int(src), :n]
        used = torch.zeros((self.P, page), dtype=torch.bool, device=DEV)
        for b in range(self.B):
            for e in range(self.M):
                if self.table[b, e] >= 0:
                    used[int(self.table[b, e]), : max(0, min(page, int(self.lens[b]) - e * page))] = True
        for n in range(len(sizes)):
            for e in range(pre[n] // page):
                used[int(order[firsts[n] + e])] = True
        self.k[~used] = math.nan
        self.v[~used] = math.nan
        self.q = torch.randn((self.B, Q, Hq, D), generator=g, device=DEV).to(DT[dtype])
        self.sq = np.full(self.B, Q) if seqlens_q is None else np.asarray(seqlens_q)
        self.seqlens_q = None if seqlens_q is None else i32(seqlens_q)
        for b in range(self.B):
            self.q[b, int(self.sq[b]):] = math.nan  # padded rows are never used
        self.cu = i32(np.concatenate([[0], np.cumsum(sizes)]))
        self.shared = i32(pre)

    def call(self, o=None, lse=None, **kw):
        return attn.attn_fwd_paged_shared(self.q, self.k, self.v, i32(self.table), i32(self.lens), self.cu,
                                          self.shared, o, lse, seqlens_q=self.seqlens_q, **kw)

    def check(self, scale=None, **kw):
        """The call between guards, with canaries; against 64 bits."""
        B, Q, Hq, Dv = self.B, self.Q, self.Hq, self.Dv
        no, nl = B * Q * Hq * Dv, B * Q * Hq
        ob = torch.full((no + GUARD,), math.nan, dtype=DT[self.dtype], device=DEV)
        lb = torch.full((nl + GUARD,), math.nan, dtype=torch.float32, device=DEV)
        ob[no:], lb[nl:] = 5, 5
        o, lse = ob[:no].view(B, Q, Hq, Dv), lb[:nl].view(B, Q, Hq)
        was = [t.clone() for t in (self.q, self.k, self.v)]
        self.call(o, lse, scale=scale, **kw)
        torch.cuda.synchronize()
        assert attn.device_status()[0] == 0
        assert (ob[no:] == 5).all() and (lb[nl:] == 5).all()
        for a, b in zip(was, (self.q, self.k, self.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        self.compare(o, lse, scale)
        return o, lse

    def compare(self, o, lse, scale=None):
        G, page, D = self.Hq // self.Hkv, self.page, self.D
        sc = 1 / math.sqrt(D) if scale is None else scale
        u = HALF[self.dtype]
        for b in range(self.B):
            n, qb = int(self.lens[b]), int(self.sq[b])
            j = torch.arange(n, device=DEV)
            pg = torch.from_numpy(self.table[b]).to(DEV)[j // page]
            k, v = self.k[pg, j % page].double(), self.v[pg, j % page].double()      # [n, Hkv, *]
            q = self.q[b].double().view(self.Q, self.Hkv, G, D)
            hi = torch.arange(self.Q, device=DEV) + n - qb + 1
            hi[qb:] = 0
            empty = hi <= 0
            s = torch.einsum("ihgd,khd->ihgk", q, k) * sc
            s = s.masked_fill(j >= hi[:, None, None, None], -math.inf)
            m = s.amax(-1, keepdim=True) if n else s.sum(-1, keepdim=True) - math.inf
            m = torch.where(m == -math.inf, torch.zeros_like(m), m)
            m[empty] = 0
            e = torch.exp(s - m)
            e[empty] = 0
            l = e.sum(-1, keepdim=True)
            p = e / torch.where(l > 0, l, torch.ones_like(l))
            ref = torch.einsum("ihgk,khd->ihgd", p, v)
            size = torch.einsum("ihgk,khd->ihgd", p, v.abs())
            # a score: D products, each sum rounded by 2^-23 of the terms; 2^x and the sums: 2^-20
            terms = torch.einsum("ihgd,khd->ihgk", q.abs(), k.abs()) * abs(sc)
            terms = torch.where(s == -math.inf, torch.zeros_like(s), terms).nan_to_num(0)
            ds = (terms.amax(-1, keepdim=True) if n else terms.sum(-1, keepdim=True)) * D * 2.0 ** -23
            de = 2 * ds + 2.0 ** -20
            # P and O round to the type; fp16 P below 2^-14 of the maximum by 2^-25
            bound = (u * 1.02 + de) * size + u * 1.02 * ref.abs() + 2.0 ** -24
            if self.dtype == "f16":
                bound = bound + 2.0 ** -25 * v.abs().sum(0)[None, :, None]
            got = o[b].double().view(self.Q, self.Hkv, G, self.Dv)
            real = ~empty
            err = (got - ref).abs()
            assert (err[real] <= bound[real]).all(), (b, float((err[real] / bound[real]).max()))
            gl = lse[b].double().view(self.Q, self.Hkv, G)
            rl = (m + torch.log(l)).squeeze(-1)
            lb = (ds + 2.0 ** -20 + 2.0 ** -22 * rl.abs()[..., None]).squeeze(-1)
            assert ((gl - rl).abs()[real] <= lb[real]).all()
            # rows without a key and padded rows: +0 and -inf
            assert not o[b][empty].float().any() and not torch.signbit(o[b][empty].float()).any()
            assert (lse[b][empty] == -math.inf).all()


# sizes, shared keys, own keys, Q, Hq, Hkv, D, Dv, page
CASES = {
    "one beam step": ([4, 4], [320, 256], [1, 40, 7, 64, 65, 3, 2, 1], 1, 8, 2, 128, 128, 64),
    "one key": ([2], [1], [0, 0], 1, 1, 1, 64, 64, 8),
    "one key each": ([3], [0], [1, 1, 1], 1, 2, 1, 64, 64, 16),
    "nothing": ([2, 1], [0, 0], [0, 0, 0], 1, 2, 2, 64, 64, 8),
    "tile edges": ([5], [128], [127, 128, 129, 1, 0], 1, 4, 1, 64, 64, 128),
    "partial pages": ([3, 2], [200, 77], [60, 1, 130, 55, 9], 1, 6, 2, 80, 112, 16),
    "pages of 8": ([3], [133], [5, 260, 1], 2, 4, 2, 128, 64, 8),
    "pages of 256": ([2, 2], [512, 300], [7, 100, 513, 1], 1, 6, 1, 64, 128, 256),
    "drafted tokens": ([6], [500], [4, 5, 9, 130, 4, 31], 4, 15, 5, 96, 96, 32),
    "64 samples": ([64], [1000], [i * 7 % 50 + 1 for i in range(64)], 1, 8, 2, 128, 128, 64),
    "more rows than two tiles": ([70], [260], [i % 9 + 1 for i in range(70)], 1, 14, 2, 64, 64, 64),
    "wide groups": ([3], [300], [1, 2, 3], 1, 128, 1, 128, 128, 64),
    "heads of three": ([50], [140], [1 + i % 3 for i in range(50)], 1, 9, 3, 112, 80, 32),
    "chunks": ([3, 2], [384, 128], [130, 170, 131, 200, 140], 130, 6, 2, 128, 128, 64),
    "long chunk": ([2], [200], [300, 517], 300, 4, 1, 64, 64, 128),
    "alone": ([1, 1], [64, 100], [20, 30], 1, 4, 2, 128, 128, 16),
    "long": ([4], [20000], [3, 700, 129, 1], 1, 8, 2, 128, 128, 64),
    "long tails": ([3, 1], [128, 70], [3001, 1, 64, 1500], 1, 8, 2, 128, 128, 64),
    "long tails, two tokens": ([2], [77], [2500, 2], 2, 16, 2, 128, 64, 128),
    "long tails of small pages": ([3], [90], [900, 3, 258], 4, 4, 1, 64, 128, 16),
    "many rows": ([14], [300], [130 + 3 * i for i in range(14)], 130, 6, 2, 64, 64, 64),
    "many rows and partials": ([2, 12], [30000, 64], [131 + i for i in range(14)], 130, 6, 2, 128, 80, 64),
    "many rows of one token": ([600], [257], [i % 5 + 1 for i in range(600)], 1, 20, 2, 64, 64, 16),
    "many groups": ([2] * 40, [64 * (n % 5) for n in range(40)], [n % 70 for n in range(80)], 1, 4, 2, 64, 64, 64),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", list(CASES))
def test_cases(name, dtype):
    b = Batch(len(name), *CASES[name], dtype)
    b.check(algo="tcgen05")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sequences_outside_groups_short_members_and_padded_rows(dtype):
    # 2 sequences behind the groups; members shorter than the shared part, the first one too;
    # rows past the queries, rows without keys
    b = Batch(3, [3, 2], [200, 130], [5, 9, 300, 4, 1], 3, 6, 2, 64, 64, 16, dtype, alone=(90, 0),
              seqlens_q=[3, 2, 0, 1, 3, 3, 3], short=((1, 70), (3, 129), (4, 2)))
    b.check()
    b.cu, b.shared = i32([1, 3, 3, 5]), i32([70, 5, 10])  # groups that begin behind the first, an empty one
    b.check()
    b.cu, b.shared = i32([0]), i32([])
    b.check(algo="tcgen05")
    b.cu, b.shared = i32([0, 3, 5]), i32([2 ** 31 - 1, -5])  # clamped to the first member's length, to none
    b.lens[:3] = 70
    b.check()


@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
def test_scales(scale):
    Batch(7, [3], [150], [5, 140, 1], 1, 4, 2, 64, 64, 64, "bf16").check(scale=scale)


@pytest.mark.parametrize("dtype,algo,D,page", [("f32", "auto", 64, 16), ("bf16", "auto", 72, 16), ("f16", "auto", 64, 4),
                                               ("bf16", "decode", 128, 64), ("bf16", "generic", 64, 64)])
def test_other_kernels(dtype, algo, D, page):
    # what the tcgen05 kernel does not take reads each sequence's own table
    Batch(5, [3, 2], [64, 32], [5, 30, 1, 2, 9], 1, 4, 2, D, D, page, dtype).check(algo=algo)


def test_against_attention_without_sharing():
    b = Batch(9, [5, 3], [640, 256], [9, 100, 64, 1, 33, 7, 8, 200], 1, 8, 2, 128, 128, 64, "bf16")
    o, lse = b.call()
    po, plse = attn.attn_fwd_paged(b.q, b.k, b.v, i32(np.maximum(b.table, 0)), i32(b.lens))
    assert float((o.float() - po.float()).abs().max()) <= 4 * HALF["bf16"] * float(po.float().abs().max())
    assert float((lse - plse).abs().max()) <= 1e-4


def test_scores_that_are_nan_or_infinite():
    b = Batch(4, [3], [256], [20, 20, 20], 1, 2, 1, 64, 64, 64, "bf16")
    # a NaN key of one sequence alone: its rows are NaN, no other sequence's
    j = 256 + 5
    b.k[int(b.table[1, j // 64]), j % 64, 0, 3] = math.nan
    o, lse = b.call(algo="tcgen05")
    assert torch.isnan(o[1].float()).all() and torch.isnan(lse[1]).all()
    assert torch.isfinite(o[[0, 2]].float()).all() and torch.isfinite(lse[[0, 2]]).all()
    # a NaN among the shared keys: every row
    b.k[int(b.table[0, 1]), 7] = math.nan
    o, lse = b.call(algo="tcgen05")
    assert torch.isnan(o.float()).all() and torch.isnan(lse).all()
    # scores of -inf weigh nothing
    b = Batch(4, [3], [256], [20, 20, 20], 1, 2, 1, 64, 64, 64, "f16")
    b.q[..., 0] = 1
    b.q[..., 1:] = 0
    b.k[..., 0] = torch.where(torch.isnan(b.k[..., 0]), b.k[..., 0], torch.zeros_like(b.k[..., 0]))
    pg = int(b.table[0, 0])
    b.k[pg, :, 0, 0] = -math.inf
    b.k[pg, :, 0, 1:] = 0
    o, lse = b.call(algo="tcgen05")
    n = 256 - 64 + 20
    assert float((lse - math.log(n)).abs().max()) <= 1e-5
    keep = [int(x) for x in b.table[0, 1:4]]
    own = b.v[int(b.table[0, 4]), :20].double()
    mean = (b.v[keep].double().sum((0, 1)) + own.sum(0)) / n
    assert float((o[0, 0].double() - mean).abs().max()) <= 3 * HALF["f16"]


def test_same_bits_every_time_and_in_graphs():
    b = Batch(12, [17, 4], [900, 128], [i * 11 % 90 for i in range(21)], 1, 8, 2, 128, 128, 32, "bf16")
    table, lens = i32(b.table), i32(b.lens)
    f = lambda o=None, lse=None: attn.attn_fwd_paged_shared(b.q, b.k, b.v, table, lens, b.cu, b.shared, o, lse)  # noqa: E731
    want = f()
    for _ in range(5):
        got = f()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # two captured graphs, replayed one behind the other and on two streams at once
    outs = [tuple(torch.empty_like(t) for t in want) for _ in range(2)]
    graphs = []
    for o, lse in outs:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f(o, lse)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f(o, lse)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    lens -= 1  # the captured calls read lengths when they run
    b.lens = b.lens - 1
    want = f()
    for _ in range(3):
        for o, lse in outs:
            o.fill_(7), lse.fill_(7)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o, lse in outs:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_streams_threads_and_no_lse():
    b = Batch(13, [6], [700], [5, 9, 1, 64, 63, 2], 2, 8, 2, 64, 64, 64, "f16")
    want, wl = b.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, none = b.call(stream=side, want_lse=False)
    side.synchronize()
    assert none is None and torch.equal(o, want)

    def work(_):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            got = [b.call() for _ in range(10)]
        s.synchronize()
        return all(torch.equal(o, want) and torch.equal(x, wl) for o, x in got)

    with concurrent.futures.ThreadPoolExecutor(3) as ex:
        assert all(ex.map(work, range(3)))


def test_offsets_past_32_bits():
    # a pool of more than 2^31 elements, with the keys in its last pages
    page, H, D = 128, 8, 128
    P = (1 << 31) // (page * H * D) + 8
    k, v = (torch.empty((P, page, H, D), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    for t in (k, v):
        t[-6:] = torch.randn((6, page, H, D), generator=g, device=DEV).bfloat16()
    q = torch.randn((3, 1, 16, D), generator=g, device=DEV).bfloat16()
    table = i32([[P - 1, P - 2, P - 3], [P - 1, P - 2, P - 4], [P - 1, P - 2, P - 5]])
    lens, cu, pre = i32([300, 257, 384]), i32([0, 3]), i32([256])
    o, lse = attn.attn_fwd_paged_shared(q, k, v, table, lens, cu, pre)
    small = attn.attn_fwd_paged_shared(q, k[-6:].clone(), v[-6:].clone(), table - (P - 6), lens, cu, pre)
    assert torch.equal(o, small[0]) and torch.equal(lse, small[1])


def test_waits_that_run_out_are_reported():
    # A wait gives up after its second try, each of up to 1 us, so some wait has to be
    # longer than 2 us: 60000 keys of 2 heads are 938 tiles, 6 an SM on 152, and the
    # epilogue waits for all of a piece's: 6 x 64 KB at 45 GB/s an SM are 8 us.  (6000
    # keys, one tile a piece, finish within the two tries.)
    b = Batch(14, [8], [60000], [5] * 8, 1, 8, 2, 128, 128, 64, "bf16")
    want = b.call()
    torch.cuda.synchronize()
    before = attn.set_wait_limit(1)
    try:
        b.call()
        torch.cuda.synchronize()
        assert attn.device_status() == (4, 0x107)
    finally:
        attn.set_wait_limit(before)
    got = b.call()
    torch.cuda.synchronize()
    assert attn.device_status()[0] == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("cached", ["bf16", "int8"])
def test_a_serving_run(cached):
    # a prompt, its pages shared by beams, and steps of fork, rotated append and attention
    # over the shared beginning: the same as attention over contiguous rotated keys
    torch.manual_seed(1)
    page, Hq, Hkv, D, P, M = 16, 8, 2, 64, 64, 8
    f = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
    a = torch.arange(200, dtype=torch.float64)[:, None] * f
    cos, sin = a.cos().float().to(DEV), a.sin().float().to(DEV)
    eight = cached == "int8"
    kp, vpg = (torch.zeros((P, page, Hkv, D), dtype=torch.int8 if eight else torch.bfloat16, device=DEV) for _ in "kv")
    scales = [torch.zeros((P, 2, Hkv), device=DEV) for _ in "kv"] if eight else []
    pools = [kp, vpg, *scales]
    new = lambda n, r: [torch.randn((n, r, h, D), device=DEV).bfloat16() for h in (Hq, Hkv, Hkv)]  # noqa: E731
    lens, refs = i32([0, 0]), i32(np.zeros(P))
    table = i32(np.full((2, M), -1))
    table, lens, refs, status = attn.attn_pages_fork(pools, table, lens, refs, i32([0, 1]), page, new_tokens=i32([70, 41]))
    assert status.tolist()[:2] == [0, 0]
    q, k, v = new(2, 70)
    n = i32([70, 41])
    call = attn.attn_rope_append_q8 if eight else attn.attn_rope_append
    call(q, k, v, cos, sin, *pools, table, lens, seqlens_new=n)
    lens = lens + n
    parents = i32([0, 0, 0, 1, 1])
    rows = [[(k[p, : int(n[p])], v[p, : int(n[p])]) for p in parents.tolist()]]
    keys = [torch.cat([t[0]]) for t in rows[0]]
    vals = [torch.cat([t[1]]) for t in rows[0]]
    cu, pre = i32([0, 3, 5]), i32([70, 41])
    for step in range(20):
        table, lens, refs, status = attn.attn_pages_fork(
            pools, table, lens, refs, parents if step == 0 else i32(range(5)), page, new_tokens=i32([1] * 5))
        assert status.tolist()[:2] == [0, 0]
        q, k, v = new(5, 1)
        qr = call(q, k, v, cos, sin, *pools, table, lens)
        lens = lens + 1
        keys = [torch.cat([x, k[b]]) for b, x in enumerate(keys)]
        vals = [torch.cat([x, v[b]]) for b, x in enumerate(vals)]
        if eight:
            o, _ = attn.attn_fwd_paged_q8(qr, *pools, table, lens)
        else:
            o, _ = attn.attn_fwd_paged_shared(qr, *pools, table, lens, cu, pre)
        for b in range(5):
            kk = attn.attn_rope(keys[b][None], None, cos, sin)[0]
            want, _ = attn.attn_fwd(qr[b: b + 1], kk, vals[b][None])
            err = float((o[b].float() - want[0].float()).abs().max())
            # bf16: P and O round by 2^-8 of values up to 4.5; int8: half a step, 2^-7 of
            # the largest, in each element (as in the 8-bit cache's own tests)
            assert err <= (0.1 if eight else 4.5 * 4 * HALF["bf16"])


def c_call(b, N, cu, pre, algo, k=None, v=None, table=None, M=None):
    """The C entry point over b's tensors, with what a C program may pass beside them."""
    o = torch.full((b.B, b.Q, b.Hq, b.Dv), 3.0, dtype=DT[b.dtype], device=DEV)
    lse = torch.full((b.B, b.Q, b.Hq), 3.0, device=DEV)
    lens = i32(b.lens)
    rc = attn.load_library().attn_fwd_paged_shared(
        b.q.data_ptr(), k, v, o.data_ptr(), lse.data_ptr(), b.B, b.Hq, b.Hkv, b.Q, b.D, b.Dv, table, M, b.page, b.P,
        None, lens.data_ptr(), cu, pre, N, 1 / math.sqrt(b.D), {"f32": 0, "f16": 1, "bf16": 2}[b.dtype], algo,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return rc, o, lse


@pytest.mark.parametrize("D,Q", [(128, 1), (80, 1), (64, 30)])
def test_no_groups_without_their_arrays(D, Q):
    # num_groups 0 with NULL in place of cu_groups and shared_lens, own keys by either kernel
    b = Batch(21, [1, 1, 1], [0, 0, 0], [90, 1, 200], Q, 8, 2, D, D, 16, "bf16")
    table = i32(b.table)
    rc, o, lse = c_call(b, 0, None, None, 2, b.k.data_ptr(), b.v.data_ptr(), table.data_ptr(), b.M)
    assert rc == 0, attn.last_error()
    b.compare(o, lse)


@pytest.mark.parametrize("algo", [0, 2])
@pytest.mark.parametrize("D,Q", [(128, 1), (80, 3)])
def test_tables_without_entries(D, Q, algo):
    # max_pages 0: no sequence has a key, and pages and table may be NULL as in attn_fwd_paged
    b = Batch(22, [2, 1], [0, 0], [0, 0, 0], Q, 8, 2, D, D, 16, "bf16")
    b.lens[:] = 7  # clamped to the capacity
    for pages in (None, b.k.data_ptr()):
        rc, o, lse = c_call(b, 2, b.cu.data_ptr(), b.shared.data_ptr(), algo, pages, pages, None, 0)
        assert rc == 0, attn.last_error()
        assert not o.view(torch.int16).any() and (lse == -math.inf).all()


@pytest.mark.parametrize("D", [64, 80])  # own keys by the decode's kernel, and by the tcgen05 one
@pytest.mark.parametrize("sizes,pre", [([700, 1, 1399], [100, 0, 33]), ([1] * 2050, [16 * (n % 4) for n in range(2050)]),
                                       ([2, 3] * 150, [n % 90 for n in range(300)])])
def test_hundreds_and_thousands_of_sequences_and_groups(sizes, pre, D):
    # more of them than are copied to shared memory (2048), or than a block's threads look at
    # in one go (128 groups)
    b = Batch(23, sizes, pre, [1 + i * 7 % 40 for i in range(sum(sizes))], 1, 2, 1, D, D, 16, "bf16")
    b.check(algo="tcgen05")
