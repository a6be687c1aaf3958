"""The page operators through the C entry points, with guard bytes around every output
and pool: nothing outside them is written, whatever the tables hold; and pools of as
many pages as the plans' shared memory just holds, and of one more."""
import array

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn
from tests import cache_ref
from tests.test_cache_gpu import DEV, check_fork, i32, random_pools, random_table

pytestmark = pytest.mark.gpu
GUARD, FILL = 256, 0x5A  # bytes (a multiple of the alignment that the entry points ask for)


class Guarded:
    """`data` (a uint8 array) on the device between guards."""

    def __init__(self, data):
        n = data.size
        self.n, self.buf = n, torch.full((n + 2 * GUARD + 64,), FILL, dtype=torch.uint8, device=DEV)
        self.buf[GUARD:GUARD + n] = torch.from_numpy(data).to(DEV)

    @property
    def ptr(self):
        return self.buf.data_ptr() + GUARD

    def data(self):
        x = self.buf.cpu().numpy()
        assert (x[:GUARD] == FILL).all() and (x[GUARD + self.n:] == FILL).all(), "a guard byte changed"
        return x[GUARD:GUARD + self.n]

    def ints(self):
        return self.data().view(np.int32)


def out_ints(n):
    return Guarded(np.full(4 * n, 0x77, np.uint8))


def addresses(pools):
    ptrs = array.array("Q", [p.ptr for p in pools])
    return ptrs, ptrs.buffer_info()[0]


# pages that the cluster copies by itself, that take a copy launch, and that take lists
SIZES = {"small": (100, 4096), "copies": (1 << 19, 36), "lists": (1 << 24, 36)}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("seed", range(4))
def test_fork_writes_nothing_outside_its_outputs(size, seed):
    """Tables with entries out of range, lengths past the table and counts that do not fit
    (consistent ones for seed 3)."""
    g = np.random.default_rng(800 + seed)
    S, M, P, N, page = 7, 6, 21, 30, 4
    if seed == 3:
        table, lens, refs = random_table(g, S, M, page, P, pins=1)
        N = 8
    else:
        table = g.integers(-5, P + 5, (S, M)).astype(np.int32)
        lens = g.integers(-10, 10 * M, S).astype(np.int32)
        refs = [np.zeros(P), np.full(P, 3), g.integers(-1, 3, P)][seed].astype(np.int32)
    parents, new = i32(g.integers(-3, S + 3, N)), i32(g.integers(-5, 5, N))
    pools = [Guarded(g.integers(0, 256, P * b, dtype=np.uint8)) for b in SIZES[size]]
    ptrs, at = addresses(pools)
    bytes_ = array.array("q", SIZES[size])
    outs = [out_ints(n) for n in (N * M, N, P, 4)]
    lib = attn.load_library()
    t, n, r = i32(table), i32(lens), i32(refs)
    rc = lib.attn_pages_fork(at, bytes_.buffer_info()[0], len(pools), t.data_ptr(), n.data_ptr(), r.data_ptr(), S, M,
                             P, page, parents.data_ptr(), new.data_ptr(), N, *[o.ptr for o in outs],
                             torch.cuda.current_stream().cuda_stream)
    assert rc == 0, attn.last_error()
    torch.cuda.synchronize()
    entries = outs[0].ints()
    assert ((entries >= -1) & (entries < P)).all()
    for x in outs + pools:
        x.data()
    if seed == 3:
        ref = cache_ref.fork(table, lens, refs, parents.cpu().numpy(), new.cpu().numpy(), page)
        for o, want in zip(outs, ref):
            assert np.array_equal(o.ints(), np.asarray(want).reshape(-1))


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("P", [1, 21, 40])
def test_compact_writes_nothing_outside_its_outputs(size, P):
    g = np.random.default_rng(810 + P)
    S, M = 5, 7
    table = g.integers(-5, P + 5, (S, M)).astype(np.int32)
    refs = g.integers(-1, 3, P).astype(np.int32)
    before = [g.integers(0, 256, P * b, dtype=np.uint8) for b in SIZES[size]]
    pools = [Guarded(b) for b in before]
    ptrs, at = addresses(pools)
    bytes_ = array.array("q", SIZES[size])
    outs = [out_ints(n) for n in (S * M, P, P, 1)]
    t, r = i32(table), i32(refs)
    rc = attn.load_library().attn_pages_compact(at, bytes_.buffer_info()[0], len(pools), t.data_ptr(), r.data_ptr(), S,
                                                M, P, *[o.ptr for o in outs], torch.cuda.current_stream().cuda_stream)
    assert rc == 0, attn.last_error()
    torch.cuda.synchronize()
    ref = cache_ref.compact(table, refs)
    for o, want in zip(outs, ref):
        assert np.array_equal(o.ints(), np.asarray(want, np.int32).reshape(-1))
    for b, w, p in zip(SIZES[size], before, pools):
        rows = w.reshape(P, b)
        want = rows.copy()
        for s, d in ref[4]:
            want[d] = rows[s]
        assert np.array_equal(p.data(), want.reshape(-1))


@pytest.mark.parametrize("P", [65535, 65536, 65537, 80000])
def test_fork_at_the_limit_of_the_shared_counts(P):
    """65536 pages are counted in the cluster's shared memory, more in a workspace."""
    g = np.random.default_rng(820)
    table, lens, refs = random_table(g, 60, 40, 8, P, pins=9)
    check_fork(g, table, lens, refs, g.integers(-1, 60, 90), g.integers(0, 30, 90), 8, shapes=(48, 12))


@pytest.mark.parametrize("P", [136528, 136529, 136536, 136537, 140000])
def test_compact_at_the_limit_of_the_shared_lists(P):
    """12 bytes a page of an eighth in 200 KB: 136528 pages fit."""
    g = np.random.default_rng(830)
    refs = np.where(g.random(P) < 0.4, g.integers(1, 4, P), 0).astype(np.int32)
    table = g.integers(-3, P + 3, (20, 33)).astype(np.int32)
    pools = random_pools(g, P, (24, 33))
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
