"""Attention over shared beginnings on the host: refusals of the entry point (before any
GPU call), the checks of the Python binding, and the arithmetic that cuts the work into
shares -- every row meets every key of its own exactly once, partial results never
overlap, and the join finds each of them."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn
from causal_gqa_attention_online_gb300 import build_ext

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "causal_gqa_attention_online_gb300", "csrc")
vp = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return attn.load_library()


def _call(lib, q=64 * MB, kp=128 * MB, vp_=192 * MB, o=256 * MB, lse=320 * MB, B=4, Hq=8, Hkv=2, Q=1, D=64, Dv=64,
          table=MB, M=4, page=64, P=16, sq=0, lens=2 * MB, cu=3 * MB, pre=4 * MB, N=2, scale=0.125, dtype=2, algo=0):
    return lib.attn_fwd_paged_shared(vp(q), vp(kp), vp(vp_), vp(o), vp(lse), B, Hq, Hkv, Q, D, Dv, vp(table), M, page,
                                     P, vp(sq), vp(lens), vp(cu), vp(pre), N, scale, dtype, algo, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(page=48), "page_size"),
    (dict(page=0), "page_size"),
    (dict(P=0), "page counts"),
    (dict(M=-1), "page counts"),
    (dict(M=1 << 26), "page counts"),
    (dict(B=-1), "negative"),
    (dict(Q=-1), "negative"),
    (dict(Hq=7), "multiple"),
    (dict(Hkv=0), "multiple"),
    (dict(D=513), "head widths"),
    (dict(Dv=0), "head widths"),
    (dict(dtype=3), "dtype"),
    (dict(algo=9), "algo"),
    (dict(q=0), "non-null"),
    (dict(o=0), "non-null"),
    (dict(kp=0), "non-null"),
    (dict(vp_=192 * MB + 8), "aligned"),
    (dict(lse=320 * MB + 4), "aligned"),
    (dict(N=-1), "groups"),
    (dict(N=1 << 30), "groups"),
    (dict(scale=float("nan")), "finite"),
    (dict(scale=float("inf")), "finite"),
    (dict(table=0), "block_table"),
    (dict(lens=0), "seqlens_k"),
    (dict(cu=0), "cu_groups"),
    (dict(pre=0), "shared_lens"),
])
def test_refuses(lib, kw, needle):
    assert _call(lib, **kw) == 1
    assert needle in lib.attn_last_error().decode()


@pytest.mark.parametrize("kw", [dict(dtype=0), dict(D=72), dict(D=256, Dv=256), dict(Dv=48), dict(page=4),
                                dict(Hq=258), dict(B=1 << 27, Q=2)])
def test_tcgen05_says_what_it_takes(lib, kw):
    assert _call(lib, algo=2, **kw) == 2
    assert "shared-prefix kernel takes" in lib.attn_last_error().decode()


def test_nothing_is_a_noop(lib):
    for kw in (dict(B=0), dict(Q=0), dict(Hq=0)):
        assert _call(lib, q=0, o=0, lse=0, table=0, lens=0, cu=0, pre=0, **kw) == 0
        assert lib.attn_last_error().decode() == ""


def test_binding_checks():
    q = torch.zeros((4, 1, 8, 64), dtype=torch.bfloat16)
    kp, vpg = (torch.zeros((16, 64, 2, 64), dtype=torch.bfloat16) for _ in "kv")
    table, lens = torch.zeros((4, 4), dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    cu, pre = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    f = attn.attn_fwd_paged_shared
    with pytest.raises(ValueError, match="CUDA"):
        f(q, kp, vpg, table, lens, cu, pre)
    with pytest.raises(TypeError, match="k_pages"):
        f(q, kp.half(), vpg, table, lens, cu, pre)
    with pytest.raises(TypeError, match="q: dtype"):
        f(q.double(), kp, vpg, table, lens, cu, pre)
    with pytest.raises(ValueError, match="cu_groups"):
        f(q, kp, vpg, table, lens, cu[:2].clone(), pre)
    with pytest.raises(TypeError, match="shared_lens"):
        f(q, kp, vpg, table, lens, cu, pre.long())
    with pytest.raises(ValueError, match="block_table"):
        f(q, kp, vpg, table[:3].clone(), lens, cu, pre)
    with pytest.raises(ValueError, match="seqlens_q"):
        f(q, kp, vpg, table, lens, cu, pre, seqlens_q=lens[:1].clone())
    with pytest.raises(ValueError, match="pages are"):
        f(q[0], kp, vpg, table, lens, cu, pre)


# ------------------------------------------------------------------ shares

PROGRAM = r'''
#include <cstdio>
#include <vector>
#include "shared.cuh"
using namespace attn;
int main() {
    int B, Q, Hkv, G, K, page, N, ctas, rows;
    while (scanf("%d %d %d %d %d %d %d %d %d", &B, &Q, &Hkv, &G, &K, &page, &N, &ctas, &rows) == 9) {
        std::vector<int32_t> cu(N + 1), pre(N + 1), lens(B), sq(B);
        for (auto &x : cu) scanf("%d", &x);
        for (int i = 0; i < N; ++i) scanf("%d", &pre[i]);
        for (auto &x : lens) scanf("%d", &x);
        for (auto &x : sq) scanf("%d", &x);
        SharedArgs a = {};
        a.p.B = B; a.p.Q = Q; a.p.Hkv = Hkv; a.p.G = G; a.p.Hq = Hkv * G; a.p.K = K; a.p.page_size = page;
        a.p.seqlens_k = lens.data(); a.p.seqlens_q = sq.data();
        a.cu_groups = cu.data(); a.shared_lens = pre.data(); a.N = N; a.ctas = ctas;
        a.tile_tokens = 128 / G;
        a.tile_align = page < 128 ? page : 128;
        a.cost_one = kCostTile128;
        a.entities = N + B;
        const SharedLens z = shared_lens_of(a);
        std::vector<long long> start(N + B + 1);
        std::vector<int> info(3 * B);
        std::vector<int> span[2] = {std::vector<int>(2 * B * Q * Hkv, -1), std::vector<int>(2 * B * Q * Hkv, -1)};
        long long W = 0;
        for (int e = 0; e < N + B; ++e) {
            const int n = e >= N ? shared_group_of(a, z, e - N) : -1;
            start[e] = W;
            const SharedEntity x = shared_entity(a, z, e, n);
            W += (long long)x.jobs * x.cj;
            if (e >= N) {
                int g0 = x.b0, s = 1;
                if (n >= 0) shared_group(a, z, n, g0, s);
                info[3 * (e - N)] = g0;
                info[3 * (e - N) + 1] = s;
                info[3 * (e - N) + 2] = x.lo;
            }
        }
        start[N + B] = W;
        printf("c %lld %lld\n", W, shared_rows(a.p, ctas));
        const int shares = shared_ctas(W, ctas);
        for (int c = 0; c < ctas; ++c) {
            const long long x0 = shared_bound(W, c, shares), x1 = shared_bound(W, c + 1, shares);
            int e = 0;
            while (x0 < x1 && !(start[e] <= x0 && x0 < start[e + 1])) ++e;
            const int n = e >= N && e < N + B ? shared_group_of(a, z, e - N) : -1;
            SharedBegin begin = {};
            begin.e = e;
            if (e < N + B) begin = shared_begin(a, z, e, n, start[e]);
            SharedWalker wk(a, x0, x1, begin);
            SharedJob k;
            int t0, t1;
            while (wk.next(k, t0, t1)) {
                const int key0 = wk.s.x.kv_start + t0 * 128;
                const int end = k.end < wk.s.x.kv_start + t1 * 128 ? k.end : wk.s.x.kv_start + t1 * 128;
                printf("p %d %d %d %d %d %d %d %d %d %d %lld %d\n", c, wk.s.x.kind, wk.s.x.b0, k.kvh, k.tok0, k.ntok,
                       wk.s.x.lo, wk.s.x.end, key0, end, shared_base(k.at, G, c), t1 - t0);
                if (t0 == 0) span[wk.s.x.kind][2 * k.at] = c;
                if (t1 == k.nt) span[wk.s.x.kind][2 * k.at + 1] = c;
            }
        }
        for (int token = 0; rows && token < B * Q; ++token)
            for (int h = 0; h < Hkv * G; ++h) {
                printf("r %d %d", token, h);
                const int b = token / Q;
                const int len = clamp_len(lens[b], K), Qb = clamp_len(sq[b], Q);
                for (int kind = 0; kind < 2; ++kind) {
                    const SharedRow r = shared_row(a, kind, info[3 * b], info[3 * b + 1], info[3 * b + 2], b, token - b * Q,
                                                   h, len, Qb);
                    if (!r.some) continue;
                    const int *sp = &span[kind][2 * r.at];
                    if (sp[0] < 0 || sp[1] < sp[0]) printf(" bad:0");
                    for (int c = sp[0]; c <= sp[1]; ++c)
                        for (int ch = 0; ch < (r.ntok > a.tile_tokens ? 1 : 2); ++ch)
                            printf(" %d:%lld", kind, shared_base(r.at, G, c) + ch * r.ntok * G + r.lr);
                }
                printf("\n");
            }
        printf("e\n");
    }
}
'''


@pytest.fixture(scope="module")
def prog(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("shared")
    (d / "shared.cu").write_text(PROGRAM)
    r = subprocess.run([nvcc, "-std=c++17", "-I", CSRC, "-o", str(d / "shared"), str(d / "shared.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "shared")


def _cases():
    g = np.random.default_rng(11)
    for i in range(60):
        B, Q = int(g.integers(1, 9)), int(g.choice([1, 1, 2, 5, 40, 140]))
        Hkv, G = int(g.integers(1, 4)), int(g.choice([1, 2, 3, 4, 7, 64, 128])) if Q < 40 else int(g.choice([1, 4, 6]))
        page = int(g.choice([8, 16, 64, 128, 256]))
        M = int(g.integers(1, 1 + 2048 // page))
        K = M * page
        lens = g.integers(0, K + 1, B)
        if i % 5 == 0:
            lens[:] = K
        N = int(g.integers(0, 4))
        cu = np.sort(g.integers(0, B + 1, N + 1))
        if N and i % 2:
            cu[0], cu[-1] = 0, B
        pre = g.integers(0, K + 1, N)
        sq = g.integers(0, Q + 1, B) if i % 3 == 0 else np.full(B, Q)
        yield B, Q, Hkv, G, K, page, N, int(g.choice([1, 2, 7, 152])), cu, pre, lens, sq


def test_shares_cover_every_row_and_key_once(prog):
    cases = list(_cases())
    text = "\n".join(" ".join(str(int(x)) for x in (*c[:8], 1, *c[8], *c[9], *c[10], *c[11])) for c in cases)
    out = subprocess.run([prog], input=text, capture_output=True, text=True, timeout=120).stdout
    blocks = out.split("e\n")
    assert len(blocks) == len(cases) + 1
    for (B, Q, Hkv, G, K, page, N, ctas, cu, pre, lens, sq), text in zip(cases, blocks):
        lines = text.splitlines()
        W, rows = map(int, lines[0].split()[1:])
        tile = 128 // G
        # what each sequence shares, and with whom
        shared = np.zeros(B, int)
        for n in range(N):
            if cu[n + 1] > cu[n]:
                shared[cu[n]: cu[n + 1]] = min(pre[n], lens[cu[n]])
        seen = {}     # (token, head) -> keys met
        where = {}    # partial row -> (token, head) that wrote it
        for ln in lines[1:]:
            f = ln.split()
            if f[0] != "p":
                continue
            c, kind, b0, kvh, tok0, ntok, lo, end, key0, key_end, base, nt = map(int, f[1:])
            two = ntok > tile
            assert 0 < ntok <= 2 * tile and nt >= 1 and key_end > key0 and key_end <= end <= K
            assert (key_end - key0 + 127) // 128 == nt and key0 % min(page, 128) == 0
            if kind == 0:
                assert lo == 0
            for r in range(ntok * G):
                token, h = tok0 + r // G, kvh * G + r % G
                b, i = divmod(token, Q)
                assert lo == 0 or (kind == 1 and lo == shared[b])
                hi = min(lens[b] - sq[b] + i + 1, end) if i < sq[b] else 0
                keys = range(max(lo, key0), max(lo, key0, min(hi, key_end)))
                for chain in range(1 if two else 2):  # (of one tile, the second says that it has none)
                    at = (kind, base + (0 if two else chain * ntok * G) + r)
                    assert at[1] < rows and at not in where
                    where[at] = (token, h)
                if len(keys):
                    seen.setdefault((token, h), []).append(keys)
        for token in range(B * Q):
            b, i = divmod(token, Q)
            hi = max(0, lens[b] - sq[b] + i + 1) if i < sq[b] else 0
            for h in range(Hkv * G):
                got = sorted(seen.get((token, h), []), key=lambda r: r.start)
                at = 0
                for r in got:
                    assert r.start == at
                    at = r.stop
                assert at == hi
        # the join finds exactly the partials of its rows
        found = 0
        for ln in lines[1:]:
            f = ln.split()
            if f[0] == "r":
                for x in f[3:]:
                    kind, at = map(int, x.split(":"))
                    assert where[(kind, at)] == (int(f[1]), int(f[2]))
                    found += 1
        assert found == len(where)


def test_shares_of_large_problems_do_not_overflow(prog):
    # 3 sequences of 2^31 - 128 keys, and 60000 of none: shares stay inside
    K, B = (1 << 31) - 128, 60000
    lens = [K] * 3 + [0] * (B - 3)
    text = " ".join(map(str, [B, 1, 8, 8, K, 128, 1, 152, 0, 0, 3, K - 1000, *lens, *[1] * B]))
    out = subprocess.run([prog], input=text, capture_output=True, text=True, timeout=120).stdout.splitlines()
    pieces = [list(map(int, ln.split()[1:])) for ln in out if ln[0] == "p"]
    assert len({p[0] for p in pieces}) > 140
    for kvh in range(8):
        runs = sorted((p[8], p[9]) for p in pieces if p[1] == 0 and p[3] == kvh)
        assert runs[0][0] == 0 and runs[-1][1] == K - 1000
        assert all(a[1] == b[0] for a, b in zip(runs, runs[1:]))


def test_groups_that_break_the_rules_stay_in_bounds(prog):
    g = np.random.default_rng(6)
    cases = []
    for _ in range(40):
        B, N = int(g.integers(1, 6)), int(g.integers(1, 5))
        cu, pre = g.integers(-3, B + 4, N + 1), g.integers(-50, 900, N)
        lens, sq = g.integers(-10, 700, B), g.integers(-2, 5, B)
        cases.append((B, 3, 2, 4, 512, 64, N, 5, 1, *cu, *pre, *lens, *sq))
    text = "\n".join(" ".join(str(int(x)) for x in c) for c in cases)
    out = subprocess.run([prog], input=text, capture_output=True, text=True, timeout=60).stdout
    blocks = out.split("e\n")
    assert len(blocks) == len(cases) + 1
    for c, text in zip(cases, blocks):
        lines = text.splitlines()
        rows = int(lines[0].split()[2])
        for ln in lines[1:]:
            f = ln.split()
            if f[0] == "p":
                _, kind, b0, kvh, tok0, ntok, lo, end, key0, key_end, base, nt = map(int, f[1:])
                assert 0 <= b0 < c[0] and 0 <= kvh < 2 and 0 <= tok0 and tok0 + ntok <= c[0] * 3
                assert 0 <= key0 < key_end <= 512 and base >= 0
                assert base + ntok * 4 * (1 if ntok > 32 else 2) <= rows


# ------------------------------------------------------------------ a sequence's own keys in parts

OWN = r'''
#include <cstdio>
#include "shared.cuh"
using namespace attn;
int main() {
    int lo, end, splits;
    while (scanf("%d %d %d", &lo, &end, &splits) == 3) {
        printf("%d", end > lo ? own_parts(lo, end, splits) : 0);
        for (int s = 0; s < splits; ++s) {
            int b, e;
            own_split(lo, end, splits, s, b, e);
            printf(" %d %d", b, e);
        }
        printf("\n");
    }
}
'''


def test_parts_of_own_keys(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    (tmp_path / "own.cu").write_text(OWN)
    subprocess.run([nvcc, "-std=c++17", "-I", CSRC, "-o", str(tmp_path / "own"), str(tmp_path / "own.cu")], check=True)
    g = np.random.default_rng(5)
    cases = [(lo, lo + n, s) for lo in (0, 1, 63, 64, 1000) for n in (0, 1, 2, 64, 65, 255, 256, 257, 100001) for s in (1, 2, 5, 64)]
    cases += [(2 ** 31 - 70, 2 ** 31 - 1, 7), (5, 2 ** 31 - 1, 64), (9, 3, 4)]
    cases += [(int(g.integers(0, 5000)), int(g.integers(0, 50000)), int(g.integers(1, 65))) for _ in range(300)]
    out = subprocess.run([str(tmp_path / "own")], input="\n".join(" ".join(map(str, c)) for c in cases),
                         capture_output=True, text=True, timeout=60).stdout.splitlines()
    for (lo, end, splits), line in zip(cases, out, strict=True):
        n, *x = map(int, line.split())
        parts = [(b, e) for b, e in zip(x[::2], x[1::2]) if e > b]
        if end <= lo:
            assert not parts
            continue
        assert all(e - b >= 256 - 63 for b, e in parts[:-1])
        # from lo to end without a gap, the inner bounds on tiles of 64 keys
        assert parts[0][0] == lo and parts[-1][1] == end
        assert all(a[1] == b[0] and a[1] % 64 == 0 for a, b in zip(parts, parts[1:]))
        # the first ones, as many as the join looks for
        assert parts == list(zip(x[::2], x[1::2]))[: len(parts)]
        assert len(parts) == n
