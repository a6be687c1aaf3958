"""The position rotation on the host: refusals of the entry points (before any GPU
call), the checks of the Python binding, and the plain restatement that the GPU
tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import causal_gqa_attention_online_gb300 as attn
from causal_gqa_attention_online_gb300 import build_ext
from causal_gqa_attention_online_gb300.rope import _rows
from tests import rope_ref

vp = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return attn.load_library()


def _rope(lib, q=64 * MB, k=128 * MB, qo=192 * MB, ko=256 * MB, cos=MB, sin=2 * MB, B=2, N=3, Hq=4, Hkv=2,
          D=64, rot=64, P=10, qs=256, ks=128, pos=0, pairs=0, inverse=0, dtype=2):
    return lib.attn_rope(vp(q), vp(k), vp(qo), vp(ko), vp(cos), vp(sin), B, N, Hq, Hkv, D, rot, P,
                         qs, ks, vp(pos), pairs, inverse, dtype, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(B=-1), "negative size"),
    (dict(N=-1), "negative size"),
    (dict(P=-1), "negative size"),
    (dict(dtype=3), "dtype"),
    (dict(pairs=2), "pairs"),
    (dict(D=513, rot=64), "head widths"),
    (dict(D=0, rot=0), "head widths"),
    (dict(rot=63), "even"),
    (dict(rot=66), "even"),
    (dict(rot=-2), "even"),
    (dict(Hq=1 << 26), "2^31"),
    (dict(qs=-1), "stride"),
    (dict(cos=0), "cos and sin"),
    (dict(sin=0), "cos and sin"),
    (dict(q=64 * MB + 1), "aligned"),
    (dict(cos=MB + 2), "aligned"),
    (dict(pos=3 * MB + 2), "aligned"),
    (dict(q=0), "non-null"),
    (dict(ko=0), "non-null"),
    (dict(qo=64 * MB + 512), "q_out overlaps"),       # its own rows, but shifted
    (dict(qo=64 * MB, qs=300), "q_out overlaps"),     # in place needs dense rows
    (dict(qo=128 * MB), "q_out overlaps"),            # the other input
    (dict(ko=64 * MB), "k_out overlaps"),
    (dict(ko=128 * MB, ks=256), "k_out overlaps"),
])
def test_rope_refuses(lib, kw, needle):
    assert _rope(lib, **kw) == 1
    assert needle in lib.attn_last_error().decode()


Q_BYTES, K_BYTES = 6 * 256 * 2, 6 * 128 * 2  # of q_out and k_out


@pytest.mark.parametrize("ko", [192 * MB, 192 * MB + Q_BYTES - 2, 192 * MB - K_BYTES + 2])
def test_rope_refuses_outputs_that_overlap(lib, ko):
    # the same memory; one element in common, at either end
    assert _rope(lib, ko=ko) == 1
    assert "q_out and k_out overlap" in lib.attn_last_error().decode()


def test_rope_of_nothing_is_a_noop(lib):
    for kw in (dict(B=0), dict(N=0), dict(Hq=0, Hkv=0, q=0, k=0, qo=0, ko=0)):
        assert _rope(lib, **kw) == 0
        assert lib.attn_last_error().decode() == ""


ROWS = dict(q=64 * MB, k=128 * MB, v=192 * MB, qo=256 * MB, kp=512 * MB, vp_=768 * MB, cos=MB, sin=2 * MB, B=2,
            N=3, total=0, Hq=4, Hkv=2, D=64, Dv=64, rot=64, P=10, qs=256, ks=128, vs=128, new=0, cu=0, pos=0,
            pairs=0, lens=3 * MB, table=4 * MB, M=4, page=64, pages=16, dtype=2)


def _append(lib, **kw):
    a = dict(ROWS, **kw)
    return lib.attn_rope_append(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["qo"]), vp(a["kp"]), vp(a["vp_"]), vp(a["cos"]), vp(a["sin"]),
        a["B"], a["N"], a["total"], a["Hq"], a["Hkv"], a["D"], a["Dv"], a["rot"], a["P"], a["qs"], a["ks"], a["vs"],
        vp(a["new"]), vp(a["cu"]), vp(a["pos"]), a["pairs"], vp(a["lens"]), vp(a["table"]), a["M"], a["page"],
        a["pages"], a["dtype"], None)


def _append_q8(lib, ks_=5 * MB, vs_=6 * MB, block=16, code=1, **kw):
    a = dict(ROWS, **kw)
    return lib.attn_rope_append_q8(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["qo"]), vp(a["kp"]), vp(a["vp_"]), vp(ks_), vp(vs_), vp(a["cos"]),
        vp(a["sin"]), a["B"], a["N"], a["total"], a["Hq"], a["Hkv"], a["D"], a["Dv"], a["rot"], a["P"], a["qs"],
        a["ks"], a["vs"], vp(a["new"]), vp(a["cu"]), vp(a["pos"]), a["pairs"], vp(a["lens"]), vp(a["table"]), a["M"],
        a["page"], a["pages"], block, code, a["dtype"], None)


BAD_ROWS = [
    (dict(page=48), "page_size"),
    (dict(pages=0), "page counts"),
    (dict(M=-1), "page counts"),
    (dict(M=1 << 26), "page counts"),
    (dict(kp=0), "non-null"),
    (dict(vp_=768 * MB + 8), "aligned"),
    (dict(B=-1), "negative"),
    (dict(N=-1), "negative"),
    (dict(cu=7 * MB, total=-1), "negative"),
    (dict(dtype=-1), "dtype"),
    (dict(pairs=-1), "pairs"),
    (dict(rot=65), "even"),
    (dict(Dv=513), "head widths"),
    (dict(Hkv=0), "Hkv"),
    (dict(sin=0), "cos and sin"),
    (dict(q=0), "q and q_out"),
    (dict(qo=0), "q and q_out"),
    (dict(Hq=0), "q and q_out"),
    (dict(k=0), "non-null"),
    (dict(v=0), "non-null"),
    (dict(lens=0), "non-null"),
    (dict(table=0), "non-null"),
    (dict(v=192 * MB + 1), "aligned"),
    (dict(vs=-2), "stride"),
    (dict(qo=64 * MB, qs=512), "q_out overlaps"),
    (dict(qo=128 * MB), "q_out overlaps"),
    (dict(qo=192 * MB), "q_out overlaps"),
]


@pytest.mark.parametrize("kw,needle", BAD_ROWS)
def test_append_refuses(lib, kw, needle):
    assert _append(lib, **kw) == 1
    assert needle in lib.attn_last_error().decode()


@pytest.mark.parametrize("kw,needle", BAD_ROWS + [
    (dict(block=24), "block_size"),
    (dict(block=128), "block_size"),
    (dict(code=2), "cache dtype"),
    (dict(ks_=0), "non-null"),
])
def test_append_q8_refuses(lib, kw, needle):
    assert _append_q8(lib, **kw) == 1
    assert needle in lib.attn_last_error().decode()


@pytest.mark.parametrize("call,kw", [(_append, dict(qo=512 * MB)), (_append, dict(qo=512 * MB - Q_BYTES + 2)),
                                     (_append, dict(qo=768 * MB + 262142)), (_append_q8, dict(qo=512 * MB + 131070)),
                                     (_append_q8, dict(qo=768 * MB)), (_append_q8, dict(qo=5 * MB)),
                                     (_append_q8, dict(qo=6 * MB + 510))])
def test_append_refuses_queries_in_the_cache(lib, call, kw):
    # pages of 16 x 64 rows of 2 heads of 64 are 256 KB (8 bits: 128), scales 512 bytes
    assert call(lib, **kw) == 1
    assert "q_out overlaps the cache" in lib.attn_last_error().decode()


@pytest.mark.parametrize("call", [_append, _append_q8])
def test_append_of_nothing_is_a_noop(lib, call):
    for kw in (dict(B=0), dict(N=0), dict(cu=7 * MB, total=0)):
        assert call(lib, k=0, v=0, lens=0, table=0, **kw) == 0
        assert lib.attn_last_error().decode() == ""


# ------------------------------------------------------------------ the Python binding

def _tensors(B=2, N=3, Hq=4, Hkv=2, D=64, dtype=torch.bfloat16):
    q, k, v = (torch.zeros((B, N, h, D), dtype=dtype) for h in (Hq, Hkv, Hkv))
    cos, sin = torch.zeros((10, D // 2)), torch.zeros((10, D // 2))
    kp, vp_ = (torch.zeros((8, 16, Hkv, D), dtype=dtype) for _ in "kv")
    return q, k, v, cos, sin, kp, vp_, torch.zeros((B, 4), dtype=torch.int32), torch.zeros(B, dtype=torch.int32)


def test_binding_needs_a_cuda_device():
    q, k, v, cos, sin, kp, vp_, table, lens = _tensors()
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_rope(q, k, cos, sin)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_rope_bwd(q, None, cos, sin)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_rope_append(q, k, v, cos, sin, kp, vp_, table, lens)


def test_binding_checks():
    q, k, v, cos, sin, kp, vp_, table, lens = _tensors()
    call = attn.attn_rope_append
    with pytest.raises(TypeError, match="q: dtype"):
        call(q.half(), k, v, cos, sin, kp, vp_, table, lens)
    with pytest.raises(TypeError, match="k: dtype"):
        attn.attn_rope(q, k.float(), cos, sin)
    with pytest.raises(TypeError, match="expected float32, float16"):
        attn.attn_rope(q.double(), k.double(), cos, sin)
    with pytest.raises(TypeError, match="cos"):
        call(q, k, v, cos.double(), sin, kp, vp_, table, lens)
    with pytest.raises(ValueError, match="cos and sin"):
        call(q, k, v, cos, None, kp, vp_, table, lens)
    with pytest.raises(ValueError, match="sin"):
        call(q, k, v, cos, sin[:, :16], kp, vp_, table, lens)
    with pytest.raises(ValueError, match="v: shape"):
        call(q, k, v[:, :2], cos, sin, kp, vp_, table, lens)
    with pytest.raises(ValueError, match="k: shape"):
        call(q, k[:1], v, cos, sin, kp, vp_, table, lens)
    with pytest.raises(ValueError, match="q: shape"):
        call(q[0], k, v, cos, sin, kp, vp_, table, lens)
    with pytest.raises(ValueError, match="pairs"):
        call(q, k, v, cos, sin, kp, vp_, table, lens, pairs="neox")
    with pytest.raises(ValueError, match="positions"):
        call(q, k, v, cos, sin, kp, vp_, table, lens, positions=lens)
    with pytest.raises(TypeError, match="k_pages"):
        call(q, k, v, cos, sin, kp.half(), vp_, table, lens)
    with pytest.raises(ValueError, match="seqlens_k"):
        call(q, k, v, cos, sin, kp, vp_, table, lens[:1])
    with pytest.raises(ValueError, match="k: shape"):
        attn.attn_rope_append_varlen(q, k, v, lens, 3, cos, sin, kp, vp_, table, lens)
    with pytest.raises(ValueError, match="k_out without k"):
        attn.attn_rope(q, None, cos, sin, None, k)
    with pytest.raises(TypeError, match="int8"):
        attn.attn_rope_append_q8(q, k, v, cos, sin, kp, vp_, cos, sin, table, lens)


def test_rows_of_views():
    x = torch.zeros((2, 3, 10, 8))
    dense = torch.Size((2, 3, 4, 8))
    assert _rows("x", x[:, :, :4].contiguous(), dense, torch.float32, -1)[1] == 32
    assert _rows("x", x[:, :, 2:6], dense, torch.float32, -1) == (x.data_ptr() + 64, 80)
    assert _rows("x", x[:1, :1, 2:6], torch.Size((1, 1, 4, 8)), torch.float32, -1)[1] == 32
    assert _rows("x", x[:, :1, 2:6], torch.Size((2, 1, 4, 8)), torch.float32, -1)[1] == 240
    assert _rows("x", x[0, :, 2:6], torch.Size((3, 4, 8)), torch.float32, -1)[1] == 80
    for bad in (x[:, :2, 2:6], x[:, :, ::2][:, :, :4], x[..., :4], x.transpose(0, 1)[..., :4, :]):
        with pytest.raises(ValueError, match="contiguous|spaced"):
            _rows("x", bad, bad.shape, torch.float32, -1)


# ------------------------------------------------------------------ the restatement

@pytest.mark.parametrize("pairs", ["half", "adjacent"])
def test_restatement_keeps_lengths_and_inner_products(pairs):
    g = np.random.default_rng(5)
    x, y = g.standard_normal((2, 7, 2, 12))
    f = 10000.0 ** (-np.arange(4) / 4)
    cos, sin = np.cos(np.arange(40)[:, None] * f), np.sin(np.arange(40)[:, None] * f)
    pos = np.array([0, 1, 5, 9, 17, 3, 30])
    a, b = (rope_ref.rotate(t, cos, sin, pos, pairs) for t in (x, y))
    assert np.array_equal(a[0], x[0]) and np.array_equal(a[..., 8:], x[..., 8:])
    # the same turn of both keeps their products; a shift of both positions too
    assert np.allclose((a * b).sum(-1), (x * y).sum(-1), rtol=0, atol=1e-12)
    p, q = rope_ref.rotate(x, cos, sin, pos + 4, pairs), rope_ref.rotate(y, cos, sin, pos + 9, pairs)
    r, s = rope_ref.rotate(x, cos, sin, pos, pairs), rope_ref.rotate(y, cos, sin, pos + 5, pairs)
    assert np.allclose((p * q).sum(-1), (r * s).sum(-1), rtol=0, atol=1e-12)
    assert np.allclose(rope_ref.rotate(a, cos, sin, pos, pairs, inverse=True), x, rtol=0, atol=1e-12)
    # the transpose: <R x, y> = <x, R' y>
    assert np.isclose((a * y).sum(), (x * rope_ref.rotate(y, cos, sin, pos, pairs, inverse=True)).sum())
    assert np.isnan(rope_ref.rotate(x, cos, sin, np.full(7, 40), pairs)[..., :8]).all()
