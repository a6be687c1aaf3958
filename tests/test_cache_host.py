"""The 8-bit paged cache on the host: refusals of its entry points (before any
GPU call), the checks of the Python binding, the index arithmetic that decides
which rows an append may write (bad lengths included), the choice of scales, and
the plain restatement that the GPU tests compare with."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn
from causal_gqa_attention_online_gb300 import build_ext
from tests import cache_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "causal_gqa_attention_online_gb300", "csrc")
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return attn.load_library()


def _append(lib, k=1 << 20, v=1 << 21, kp=1 << 22, vp_=1 << 23, ks=1 << 24, vs=1 << 25, B=2, N=3,
            Hkv=2, D=64, Dv=64, new=None, lens=1 << 26, table=1 << 27, M=4, page=64, P=16, block=16,
            code=1, dtype=2):
    return lib.attn_cache_append(vp(k), vp(v), vp(kp), vp(vp_), vp(ks), vp(vs), B, N, Hkv, D, Dv,
                                 vp(new), vp(lens), vp(table), M, page, P, block, code, dtype, None)


BAD_CACHE = [
    (dict(page=48), "page_size"),
    (dict(page=0), "page_size"),
    (dict(block=128), "block_size"),
    (dict(block=24), "block_size"),
    (dict(block=0), "block_size"),
    (dict(P=0), "page counts"),
    (dict(M=-1), "page counts"),
    (dict(M=1 << 26), "page counts"),
    (dict(code=2), "cache dtype"),
    (dict(D=513), "head widths"),
    (dict(Dv=0), "head widths"),
    (dict(Hkv=0), "Hkv"),
    (dict(kp=0), "non-null"),
    (dict(vs=0), "non-null"),
    (dict(vp_=(1 << 23) + 8), "aligned"),
]


@pytest.mark.parametrize("kw,needle", BAD_CACHE + [
    (dict(B=-1), "negative"),
    (dict(N=-2), "negative"),
    (dict(dtype=3), "dtype"),
    (dict(k=0), "non-null"),
    (dict(lens=0), "non-null"),
    (dict(table=0), "non-null"),
    (dict(v=(1 << 21) + 4), "aligned"),
])
def test_append_refuses(lib, kw, needle):
    assert _append(lib, **kw) == 1
    assert needle in lib.attn_last_error().decode()


def test_append_of_nothing_is_a_noop(lib):
    for kw in (dict(B=0), dict(N=0), dict(M=0)):
        assert _append(lib, k=0, v=0, lens=0, table=0, **kw) == 0
        assert lib.attn_last_error().decode() == ""


def test_append_varlen_refuses(lib):
    def call(cu, total, max_new=4):
        return lib.attn_cache_append_varlen(vp(1 << 20), vp(1 << 21), vp(1 << 22), vp(1 << 23),
                                            vp(1 << 24), vp(1 << 25), 2, total, max_new, 2, 64, 64,
                                            vp(cu), vp(1 << 26), vp(1 << 27), 4, 64, 16, 16, 1, 2,
                                            None)
    assert call(0, 5) == 1 and "cu_seqlens_new" in lib.attn_last_error().decode()
    assert call(1 << 28, -1) == 1 and "negative" in lib.attn_last_error().decode()
    assert call(1 << 28, 5, -1) == 1 and "negative" in lib.attn_last_error().decode()
    assert call(1 << 28, 0) == 0


def _fwd(lib, q=1 << 20, kp=1 << 22, vp_=1 << 23, ks=1 << 24, vs=1 << 25, o=1 << 28, B=2, Hq=4,
         Hkv=2, Q=1, D=64, Dv=64, table=1 << 27, M=4, page=64, P=16, block=16, code=1,
         lens=1 << 26, window=0, mask=0, dtype=2, algo=0):
    return lib.attn_fwd_paged_q8(vp(q), vp(kp), vp(vp_), vp(ks), vp(vs), vp(o), None, B, Hq, Hkv,
                                 Q, D, Dv, vp(table), M, page, P, block, code, None, vp(lens),
                                 window, 0.125, mask, dtype, algo, None)


@pytest.mark.parametrize("kw,needle", BAD_CACHE + [
    (dict(B=-1), "negative"),
    (dict(Hq=3), "multiple"),
    (dict(q=0), "non-null"),
    (dict(o=(1 << 28) + 2), "aligned"),
    (dict(dtype=5), "dtype"),
    (dict(algo=7), "algo"),
    (dict(mask=3), "mask"),
    (dict(mask=2, window=4), "window"),
    (dict(table=0), "block_table"),
    (dict(lens=0), "block_table and seqlens_k"),
])
def test_attention_refuses(lib, kw, needle):
    assert _fwd(lib, **kw) == 1
    assert needle in lib.attn_last_error().decode()


@pytest.mark.parametrize("kw", [dict(D=40), dict(Dv=8), dict(D=272, Dv=272), dict(page=4, block=4),
                                dict(Q=513), dict(dtype=0)])
def test_decode_kernel_refuses_what_it_does_not_take(lib, kw):
    assert _fwd(lib, algo=3, **kw) == 2
    assert "8-bit decode kernel" in lib.attn_last_error().decode()


@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("algo", [0, 1, 3])
def test_attention_refuses_a_scale_that_is_no_number(lib, scale, algo):
    p = [vp(x) for x in (1 << 20, 1 << 22, 1 << 23, 1 << 24, 1 << 25, 1 << 28)]
    assert lib.attn_fwd_paged_q8(*p, None, 2, 4, 2, 1, 64, 64, vp(1 << 27), 4, 64, 16, 16, 1, None,
                                 vp(1 << 26), 0, scale, 0, 2, algo, None) == 1
    assert "finite" in lib.attn_last_error().decode()


def test_cache_refuses_rows_of_too_many_elements(lib):
    """A row's elements are counted in 32 bits."""
    heads = (1 << 31) // 64
    assert _append(lib, Hkv=heads) == 1 and "2^31" in lib.attn_last_error().decode()
    assert _fwd(lib, Hq=heads, Hkv=heads) == 1 and "2^31" in lib.attn_last_error().decode()


def test_attention_of_nothing_is_a_noop(lib):
    assert _fwd(lib, B=0, q=0, o=0, table=0, lens=0) == 0
    assert _fwd(lib, Q=0, q=0, o=0, table=0, lens=0) == 0


def _pools(n, null_at=None, size=256, bad_size_at=None):
    p, b = (vp * max(n, 1))(), (ctypes.c_longlong * max(n, 1))()
    for i in range(n):
        p[i] = None if i == null_at else (1 << 20) + 4096 * i
        b[i] = 0 if i == bad_size_at else size
    return p, b


@pytest.mark.parametrize("kw,needle", [
    (dict(npools=-1), "npools"),
    (dict(null_at=1), "pool 1 is null"),
    (dict(bad_size_at=0), "pool 0"),
    (dict(n=-1), "negative"),
    (dict(src=0), "non-null"),
])
def test_page_copy_refuses(lib, kw, needle):
    n = kw.pop("n", 3)
    npools = kw.pop("npools", 2)
    src = kw.pop("src", 1 << 26)
    p, b = _pools(2, **kw)
    assert lib.attn_pages_copy(p, p, b, npools, 8, 8, vp(src), vp(1 << 27), n, None) == 1
    assert needle in lib.attn_last_error().decode()


def test_page_copy_of_nothing_is_a_noop(lib):
    p, b = _pools(2)
    assert lib.attn_pages_copy(p, p, b, 2, 8, 8, None, None, 0, None) == 0
    assert lib.attn_pages_copy(None, None, None, 0, 8, 8, None, None, 4, None) == 0


def _fork(lib, table=1 << 20, lens=1 << 21, refs=1 << 22, S=2, M=4, P=16, page=64, parents=1 << 23,
          N=3, table_out=1 << 24, lens_out=1 << 25, refs_out=1 << 26, status=1 << 27):
    p, b = _pools(1)
    return lib.attn_pages_fork(p, b, 1, vp(table), vp(lens), vp(refs), S, M, P, page, vp(parents),
                               None, N, vp(table_out), vp(lens_out), vp(refs_out), vp(status), None)


@pytest.mark.parametrize("kw,needle", [
    (dict(page=10), "page_size"),
    (dict(S=-1), "bad sizes"),
    (dict(N=-1), "bad sizes"),
    (dict(N=(1 << 30) + 1), "bad sizes"),
    (dict(P=(1 << 30) + 1), "bad sizes"),
    (dict(P=0), "bad sizes"),
    (dict(M=1 << 26), "bad sizes"),
    (dict(refs=0), "null pointer"),
    (dict(parents=0), "null pointer"),
    (dict(lens=0), "null pointer"),
    (dict(table_out=0), "null pointer"),
    (dict(status=0), "null pointer"),
    (dict(refs_out=1 << 22), "alias"),
    (dict(table_out=1 << 20), "alias"),
    (dict(lens_out=1 << 21), "alias"),
])
def test_fork_refuses(lib, kw, needle):
    assert _fork(lib, **kw) == 1
    assert needle in lib.attn_last_error().decode()


@pytest.mark.parametrize("kw,needle", [
    (dict(S=-1), "bad sizes"),
    (dict(P=0), "bad sizes"),
    (dict(P=(1 << 30) + 1), "bad sizes"),
    (dict(refs=0), "null pointer"),
    (dict(table=0), "null pointer"),
    (dict(remap=0), "null pointer"),
    (dict(refs_out=1 << 22), "alias"),
])
def test_compact_refuses(lib, kw, needle):
    a = dict(table=1 << 20, refs=1 << 22, S=2, M=4, P=16, table_out=1 << 24, refs_out=1 << 26,
             remap=1 << 27, n=1 << 28)
    a.update(kw)
    p, b = _pools(1)
    assert lib.attn_pages_compact(p, b, 1, vp(a["table"]), vp(a["refs"]), a["S"], a["M"], a["P"],
                                  vp(a["table_out"]), vp(a["refs_out"]), vp(a["remap"]),
                                  vp(a["n"]), None) == 1
    assert needle in lib.attn_last_error().decode()


# ---------------------------------------------------------------- the binding

def _cpu_cache(P=4, page=16, Hkv=2, D=8, nblk=2, code=torch.int8):
    kp = torch.zeros((P, page, Hkv, D), dtype=torch.int8).view(code)
    ks = torch.ones((P, nblk, Hkv))
    return kp, kp.clone(), ks, ks.clone(), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(
        3, dtype=torch.int32)


def test_binding_has_no_cpu_path():
    kp, vp_, ks, vs, table, lens = _cpu_cache()
    q, k = torch.zeros((3, 1, 4, 8)), torch.zeros((3, 1, 2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_fwd_paged_q8(q, kp, vp_, ks, vs, table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_cache_append(k, k, kp, vp_, ks, vs, table, lens)
    refs = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_pages_fork([kp], table, lens, refs, lens, 16)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_pages_compact([kp], table, refs)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_pages_copy([kp], [vp_], lens, lens)


def test_binding_checks_shapes_and_types():
    kp, vp_, ks, vs, table, lens = _cpu_cache()
    q = torch.zeros((3, 1, 4, 8))
    call = attn.attn_fwd_paged_q8
    with pytest.raises(TypeError, match="k_pages"):
        call(q, kp.float(), vp_, ks, vs, table, lens)
    with pytest.raises(TypeError, match="v_pages"):
        call(q, kp, vp_.view(torch.float8_e4m3fn), ks, vs, table, lens)
    with pytest.raises(ValueError, match="v_pages"):
        call(q, kp, vp_[:, :8].contiguous(), ks, vs, table, lens)
    with pytest.raises(ValueError, match="blocks"):
        call(q, kp, vp_, torch.ones((4, 3, 2)), torch.ones((4, 3, 2)), table, lens)
    with pytest.raises(ValueError, match="v_scale"):
        call(q, kp, vp_, ks, torch.ones((4, 1, 2)), table, lens)
    with pytest.raises(TypeError, match="k_scale"):
        call(q, kp, vp_, ks.double(), vs, table, lens)
    with pytest.raises(TypeError, match="block_table"):
        call(q, kp, vp_, ks, vs, table.long(), lens)
    with pytest.raises(ValueError, match="seqlens_k"):
        call(q, kp, vp_, ks, vs, table, lens[:2])
    with pytest.raises(ValueError, match="contiguous"):
        call(q, kp.transpose(1, 2).contiguous().transpose(1, 2), vp_, ks, vs, table, lens)
    with pytest.raises(ValueError, match="q: shape"):
        call(q[:2], kp, vp_, ks, vs, table, lens)
    with pytest.raises(ValueError, match="q: shape"):
        call(torch.zeros((3, 1, 4, 16)), kp, vp_, ks, vs, table, lens)
    k = torch.zeros((3, 2, 2, 8))
    with pytest.raises(ValueError, match="k: shape"):
        attn.attn_cache_append(k[:, :, :1], k, kp, vp_, ks, vs, table, lens)
    with pytest.raises(TypeError, match="v: dtype"):
        attn.attn_cache_append(k, k.half(), kp, vp_, ks, vs, table, lens)
    with pytest.raises(TypeError, match="k: dtype"):
        attn.attn_cache_append(k.double(), k.double(), kp, vp_, ks, vs, table, lens)
    with pytest.raises(ValueError, match="seqlens_new"):
        attn.attn_cache_append(k, k, kp, vp_, ks, vs, table, lens, seqlens_new=lens[:1])
    refs = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="pages first"):
        attn.attn_pages_fork([kp[:3]], table, lens, refs, lens, 16)
    with pytest.raises(ValueError, match="contiguous"):
        attn.attn_pages_compact([kp.transpose(1, 2)], table, refs)
    with pytest.raises(ValueError, match="differ in size"):
        attn.attn_pages_copy([kp], [ks], lens, lens)
    with pytest.raises(ValueError, match="source pools"):
        attn.attn_pages_copy([kp], [], lens, lens)


# ------------------------------------------------------------ index arithmetic

PROGRAM = r'''
#include <cstdio>
#include <cstring>
#include "q8.cuh"
int main() {
    char what;
    while (std::scanf(" %c", &what) == 1) {
        if (what == 's') {
            int len, n, t, ps, bs;
            long long cap;
            std::scanf("%d %d %lld %d %d %d", &len, &n, &cap, &t, &ps, &bs);
            const attn::AppendSpan s = attn::append_span(len, n, cap, t, ps, bs);
            std::printf("%lld %lld %lld %d %d\n", s.first, s.last, s.start, s.entry, s.sub);
        } else if (what == 'u') {
            int Qb, Kb, w, m, lo, hi;
            std::scanf("%d %d %d %d", &Qb, &Kb, &w, &m);
            attn::unit_keys(Qb, Kb, w, m, lo, hi);
            std::printf("%d %d\n", lo, hi);
        } else {
            unsigned bits;
            int code;
            std::scanf("%x %d", &bits, &code);
            float a;
            std::memcpy(&a, &bits, 4);
            const float s = attn::append_scale(a, code);
            std::memcpy(&bits, &s, 4);
            std::printf("%x\n", bits);
        }
    }
    return 0;
}
'''


@pytest.fixture(scope="module")
def prog(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("span")
    src = d / "span.cu"
    src.write_text(PROGRAM)
    exe = d / "span"
    r = subprocess.run([nvcc, "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(exe)


def test_append_spans_cover_exactly_the_new_rows(prog):
    g = np.random.default_rng(3)
    asked, want = [], []
    for _ in range(200):
        ps = int(g.integers(0, 9))
        bs = int(g.integers(0, ps + 1))
        M = int(g.integers(1, 6))
        cap = M << ps
        length = int(g.integers(0, cap + 1))
        n = int(g.integers(0, cap + 5))  # also past the table
        touch = max(0, n - 1 + (1 << bs) - 1) // (1 << bs) + 1
        asked += [f"s {length} {n} {cap} {t} {ps} {bs}" for t in range(touch)]
        want.append((ps, bs, M, cap, length, n, touch))
    # lengths near 2^31 do not overflow
    big = (1 << 31) - 64
    asked.append(f"s {big - 3} {2 ** 31 - 1} {big} 0 6 4")
    r = subprocess.run([prog], input="\n".join(asked), capture_output=True, text=True, timeout=60)
    lines = [tuple(int(x) for x in ln.split()) for ln in r.stdout.splitlines()]
    assert len(lines) == len(asked)
    at = 0
    for ps, bs, M, cap, length, n, touch in want:
        seen = []
        for first, last, start, entry, sub in lines[at: at + touch]:
            if last > first:
                assert 0 <= entry < M and entry == first >> ps == (last - 1) >> ps
                assert start == first >> bs << bs and last - start <= 1 << bs
                assert sub == (first & ((1 << ps) - 1)) >> bs
                seen += range(first, last)
        at += touch
        assert seen == list(range(length, min(length + n, cap)))
    first, last, start, entry, sub = lines[-1]
    assert (first, last) == (big - 3, big) and entry == (big - 3) >> 6


def test_unit_keys_are_the_union_of_the_rows_legal_keys(prog):
    from tests.oracle_pins import mask_matrix
    cs = [(Qb, Kb, w, m) for Qb in range(0, 8) for Kb in range(0, 9) for m in range(3)
          for w in ((0,) if m == 2 else (0, 1, 2, 5, 9))]
    r = subprocess.run([prog], input="\n".join("u %d %d %d %d" % c for c in cs), capture_output=True,
                       text=True, timeout=60)
    got = [tuple(int(x) for x in ln.split()) for ln in r.stdout.splitlines()]
    assert len(got) == len(cs)
    for (Qb, Kb, w, m), (lo, hi) in zip(cs, got):
        keys = np.flatnonzero(mask_matrix(Qb, Kb, w, m).any(axis=0)) if Qb and Kb else np.zeros(0)
        if keys.size == 0:
            assert hi <= lo, (Qb, Kb, w, m)
        else:
            assert (lo, hi) == (keys[0], keys[-1] + 1), (Qb, Kb, w, m)


@pytest.mark.parametrize("kind,code", [("e4m3", 0), ("int8", 1)])
def test_append_scale_is_the_smallest_power_of_two(prog, kind, code):
    q = cache_ref.QMAX[kind]
    vals = [0.0, 1e-45, 1e-38, 1.0, 3.4028234663852886e38]
    for e in (-110, -101, -100, -99, -30, -1, 0, 1, 20, 117):
        edge = np.float32(q * 2.0 ** e)
        vals += [edge, np.nextafter(edge, np.float32(0)), np.nextafter(edge, np.float32(np.inf))]
    g = np.random.default_rng(4)
    vals += list(np.exp2(g.uniform(-120, 127, 300)))
    vals = np.array(vals, np.float32)
    vals = np.append(vals, np.array([np.inf, np.nan], np.float32))
    r = subprocess.run([prog], input="\n".join(f"a {v:x} {code}" for v in vals.view(np.uint32)),
                       capture_output=True, text=True, timeout=60)
    got = np.array([int(x, 16) for x in r.stdout.split()], np.uint32).view(np.float32)
    assert len(got) == len(vals)
    for a, s in zip(vals, got):
        ref = cache_ref.scale_for(float(a), kind)
        assert (math.isnan(s) and math.isnan(ref)) or float(s) == ref, (a, s, ref)


# -------------------------------------------------- the restatement's own checks

def test_reference_codes_round_to_nearest_even():
    # against torch's conversion, every e4m3 value and the middles between them
    pos = cache_ref.E4M3[:127]
    y = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, np.nextafter((pos[1:] + pos[:-1]) / 2, 1e9)])
    y = np.concatenate([y, -y]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(cache_ref.round_codes(y.astype(np.float64), "e4m3"), want)
    z = np.array([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.4])
    assert list(cache_ref.round_codes(z, "int8").view(np.int8)) == [0, 2, 2, 0, -2, 126, 127]


def test_reference_fork_by_hand():
    # two slots share page 5 (full); slot 0 has 6 tokens (page 2 half full), slot 1 has 4
    table = np.array([[5, 2, -1], [5, -1, -1]], np.int32)
    refs = np.array([0, 0, 1, 0, 0, 2], np.int32)
    out, lens, left, status, copies = cache_ref.fork(table, np.array([6, 4]), refs, [0, 0, 1, -1],
                                                     [1, 3, 1, 9], 4)
    # slot 0 keeps page 2; slot 1 gets a copy in page 0 and page 1 for its third new token;
    # slot 2 page 3; slot 3 is empty
    assert out.tolist() == [[5, 2, -1], [5, 0, 1], [5, 3, -1], [-1, -1, -1]]
    assert lens.tolist() == [6, 6, 4, 0] and copies == [(2, 0)]
    assert left.tolist() == [1, 1, 1, 1, 0, 3] and status.tolist() == [0, 0, 3, 1]
