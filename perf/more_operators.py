"""The position rotation, appending rotated rows to a paged cache, and attention over a
shared prefix, as cases that can be measured.

``rope`` rotates the queries and keys of a training step, or the gradients of such
rotated ones.  ``append`` takes the projected q, k and v of a serving step: q comes
back rotated, k goes rotated and v as it is into the pages (16 or 32 bits, or 8-bit
codes with a scale for each block of tokens and head).  ``shared`` is the attention
of a batch whose sequences have long common beginnings, in the same pages.  ``run``
computes a case with elementary torch operations, or through the package's entry
points when ``own`` is set; ``exact`` computes the same in 64 bits.

Layout: pages [P, page, Hkv, D], key j of sequence b in row j % page of page
block_table[b, j // page]; 8-bit pages with scales [P, page / block, Hkv].  Tables of
angles: cos and sin [positions, rot / 2] for the first rot columns of a head.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_QMAX = {"int8": 127.0, "e4m3": 448.0}
_MIN_EXP = -100  # the smallest scale is 2^-100


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short fp32 sequence, as a test of a training step has it: latency
        dict(name="rope b1 n64 fp32", op="rope", B=1, N=64, Hq=4, Hkv=2, D=64, rot=64, dtype="fp32",
             pairs="half", back=False, docs=1),
        # the queries and keys of the benchmark's training-sized prefill
        dict(name="rope b4 n4096", op="rope", B=4, N=4096, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
             pairs="half", back=False, docs=1),
        # their gradients: several documents a row, adjacent pairs, half of each head rotated
        dict(name="rope back b2 n5001", op="rope", B=2, N=5001, Hq=16, Hkv=4, D=96, rot=48, dtype="fp16",
             pairs="adjacent", back=True, docs=7),
        # one token of every sequence of a decode batch
        dict(name="append b64 n1", op="append", B=64, N=1, Hq=32, Hkv=8, D=128, rot=128, K=8192, page=64,
             block=64, code="none", dtype="bf16", pairs="half", packed=False),
        # prompts: ragged, up to 4096 rows a sequence, packed
        dict(name="append b16 n4096", op="append", B=16, N=4096, Hq=32, Hkv=8, D=128, rot=128, K=4096,
             page=64, block=64, code="none", dtype="bf16", pairs="half", packed=True),
        # one token of every sequence into an int8 cache
        dict(name="append b64 n1 int8", op="append", B=64, N=1, Hq=32, Hkv=8, D=128, rot=128, K=8192,
             page=64, block=64, code="int8", dtype="bf16", pairs="half", packed=False),
        # the prompts into an e4m3 cache
        dict(name="append b16 n4096 e4m3", op="append", B=16, N=4096, Hq=32, Hkv=8, D=128, rot=128,
             K=4096, page=64, block=64, code="e4m3", dtype="bf16", pairs="half", packed=False),
        # one beam search step: four beams of each of four short requests
        dict(name="shared 4x4 k320", op="shared", groups=4, members=4, K=320, tail=40, Q=1, Hq=32, Hkv=8,
             D=128, page=64, dtype="bf16"),
        # 64 samples of one long prompt, some hundreds of tokens in
        dict(name="shared 1x64 k32768", op="shared", groups=1, members=64, K=32768, tail=500, Q=1, Hq=32,
             Hkv=8, D=128, page=64, dtype="bf16"),
        # 32 requests of up to eight beams over long contexts
        dict(name="shared 32x8 k8192", op="shared", groups=32, members=8, K=8192, tail=64, Q=1, Hq=32,
             Hkv=8, D=128, page=128, dtype="bf16"),
        # a document of 100 thousand tokens, 21 questions, four drafted tokens each, 64-wide heads
        dict(name="shared 1x21 q4 k100000", op="shared", groups=1, members=21, K=100000, tail=301, Q=4,
             Hq=16, Hkv=4, D=64, page=32, dtype="fp16"),
        # a system prompt, and 130 more tokens of each of 24 requests at once (chunked prefill)
        dict(name="shared 2x12 q130 k4096", op="shared", groups=2, members=12, K=4096, tail=700, Q=130,
             Hq=24, Hkv=4, D=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "shared", "shared", "shared"])
    c = dict(op=op, Hkv=rng.randint(1, 8), D=rng.choice([64, 64, 80, 96, 112, 128, 128, 128]))
    if op == "shared":
        c["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
        c["page"] = rng.choice([16, 32, 64, 64, 128, 256])
        c["Q"] = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 130)])
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 4, 5, 6, 8])
        c["groups"], c["members"] = _log(rng, 1, 32), _log(rng, 2, 64)
        seqs = c["groups"] * c["members"]
        c["tail"] = c["Q"] + _log(rng, 1, 700)
        # no more than the largest listed: 24 * 130 * 24 heads over 4800 keys; keys of 1 GB
        most = min(100000, (24 * 130 * 24 * 128 * 4800) // (seqs * c["Q"] * c["Hq"] * c["D"]) - c["tail"],
                   32 * 8192 * 1024 // (c["groups"] * c["Hkv"] * c["D"]))
        c["tail"] = min(c["tail"], c["Q"] + 32 * 8192 * 1024 // (8 * seqs * c["Hkv"] * c["D"]))
        c["K"] = max(c["page"], _log(rng, 64, max(64, most)) // c["page"] * c["page"])
        return c
    c["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    c["pairs"] = rng.choice(["half", "half", "adjacent"])
    c["rot"] = rng.choice([c["D"], c["D"], c["D"] // 2])
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 4, 6, 8])
    token = (c["Hq"] + 2 * c["Hkv"]) * c["D"] * _SIZE[c["dtype"]]
    if op == "rope":
        c["B"] = _log(rng, 1, 16)
        c["N"] = _log(rng, 1, max(2, min(8192, 4 * 4096 * 48 * 128 * 2 // (c["B"] * token))))
        c["back"], c["docs"] = rng.random() < 0.5, rng.choice([1, 1, rng.randint(1, 9)])
        return c
    c["page"] = rng.choice([16, 32, 64, 64, 128, 256])
    c["code"] = rng.choice(["none", "none", "int8", "e4m3"])
    c["block"] = rng.choice([b for b in (8, 16, 32, 64, 128) if b <= c["page"]])
    c["packed"] = rng.random() < 0.4
    c["B"] = _log(rng, 1, 64)
    c["N"] = rng.choice([1, _log(rng, 2, max(3, min(4096, 16 * 4096 * 48 * 128 * 2 // (c["B"] * token))))])
    c["K"] = c["N"] + _log(rng, 1, 2048)
    return c


def _lens(n, most, least=0):
    """Ragged lengths that the case alone decides: the first is `most`, the others spread over [least, most]."""
    return [most if b == 0 else least + ((most - least + 1) * ((b * 40503 + 9973) % 65536) >> 16) for b in range(n)]


def _ceil(a, b):
    return -(-a // b)


def _shares(c):
    """(members, shared keys) of each group, and the own keys of each sequence."""
    sizes = _lens(c["groups"], c["members"], 1)
    pre = [n // c["page"] * c["page"] for n in _lens(c["groups"], c["K"], c["K"] // 2)]
    return sizes, pre, _lens(sum(sizes), c["tail"], c["Q"])


def work(c):
    es, width = _SIZE[c["dtype"]], c["Hkv"] * c["D"]
    if c["op"] == "rope":
        rows = c["B"] * c["N"]
        return {"bytes": 2 * rows * (c["Hq"] + c["Hkv"]) * c["D"] * es + 4 * c["rot"] * min(c["N"], rows),
                "flops": 3 * rows * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "append":
        n = sum(min(c["N"], x) for x in _lens(c["B"], c["N"]))
        out = 1 if c["code"] != "none" else es
        return {"bytes": n * (2 * c["Hq"] * c["D"] * es + 2 * width * (es + out)) + 4 * c["rot"] * min(n, c["K"]) +
                (8 * n * c["Hkv"] / c["block"] if out == 1 else 0),
                "flops": 3 * n * (c["Hq"] + c["Hkv"]) * c["rot"]}
    sizes, pre, tails = _shares(c)
    keys, seqs, Q = sum(pre) + sum(tails), sum(sizes), c["Q"]
    pairs = sum(s * p for s, p in zip(sizes, pre)) * Q + sum(Q * t - Q * (Q - 1) // 2 for t in tails)
    return {"bytes": keys * 2 * width * es + seqs * Q * c["Hq"] * (2 * c["D"] * es + 4),
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ inputs

def _activations(shape, gen, dtype):
    """What a projection gives: normal, with a spread over the channels and some larger rows."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[-1:], generator=gen, device="cuda"))
    x *= torch.exp2(torch.randint(-1, 2, shape[:-1] + (1,), generator=gen, device="cuda").float())
    return x.to(dtype)


def _angles(c, positions):
    """cos and sin of every position up to the last, as a model lays them out once (base 10000, in 64 bits)."""
    f = 10000.0 ** (-torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda") / (c["rot"] // 2))
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def _scale_for(amax, code):
    """The smallest power of two s >= 2^-100 with amax <= qmax * s; NaN where amax is not finite."""
    mant, exp = torch.frexp(amax / _QMAX[code])  # mant in [0.5, 1): 2^(exp - 1) only if mant is 0.5
    exp = torch.where(mant == 0.5, exp - 1, exp).clamp(min=_MIN_EXP)
    s = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, exp, torch.full_like(exp, _MIN_EXP)))
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, math.nan))


def _quantize(x, s, code):
    y = x / s
    y = torch.where(torch.isfinite(y), y, torch.zeros_like(y))
    return torch.round(y).to(torch.int8) if code == "int8" else y.to(torch.float8_e4m3fn)


def _pool(c, pages, gen):
    """Pages that hold activations, and the scales of 8-bit ones (else None)."""
    shape = (pages, c["page"], c["Hkv"], c["D"])
    if c.get("code", "none") == "none":
        return _activations(shape, gen, _DTYPES[c["dtype"]]), None
    x = _activations(shape, gen, torch.bfloat16).float().view(pages, -1, c["block"], c["Hkv"], c["D"])
    s = _scale_for(x.abs().amax(dim=(2, 4)), c["code"])
    return _quantize(x, s[:, :, None, :, None], c["code"]).view(shape), s


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(c)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    dtype, Hq, Hkv, D = _DTYPES[c["dtype"]], c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        st["q"], st["k"] = (_activations((c["B"], c["N"], h, D), gen, dtype) for h in (Hq, Hkv))
        st["cos"], st["sin"] = _angles(c, c["N"])
        st["pos"] = None
        if c["docs"] > 1:  # documents behind one another in a row, each from position 0
            at = torch.arange(c["N"], device="cuda").expand(c["B"], -1)
            cuts = torch.randint(0, c["N"], (c["B"], c["docs"] - 1), generator=gen, device="cuda").sort(1).values
            which = torch.searchsorted(cuts, at.contiguous(), right=True)
            starts = torch.cat([torch.zeros_like(cuts[:, :1]), cuts], 1)
            st["pos"] = (at - starts.gather(1, which)).to(torch.int32)
        return st
    if c["op"] == "append":
        lens = _lens(c["B"], c["K"])
        new = [min(n, x) for n, x in zip(lens, _lens(c["B"], c["N"]))]
        need = [max(1, _ceil(n, c["page"])) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = np.full((c["B"], max(need)), -1, np.int64)
        for b, e in enumerate(np.cumsum(need)):
            table[b, : need[b]] = np.arange(e - need[b], e)
        at = torch.from_numpy(table).cuda()
        st["table"] = torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(at, -1, dtype=torch.int32))
        st["kp"], st["ks"] = _pool(c, pages, gen)
        st["vp"], st["vs"] = _pool(c, pages, gen)
        st["lens"], st["new"] = ints([n - x for n, x in zip(lens, new)]), ints(new)
        st["cu"] = ints([0, *np.cumsum(new).tolist()])
        rows = (sum(new),) if c["packed"] else (c["B"], c["N"])
        st["q"], st["k"], st["v"] = (_activations(rows + (h, D), gen, dtype) for h in (Hq, Hkv, Hkv))
        st["cos"], st["sin"] = _angles(c, c["K"])
        return st
    # the shared pages of a group, then those of its members alone
    page = c["page"]
    sizes, pre, tails = _shares(c)
    need = [_ceil(t, page) for t in tails]
    pages = sum(pre) // page + sum(need) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    group = np.repeat(np.arange(len(sizes)), sizes)
    table = np.full((len(tails), max(pre[g] // page + n for g, n in zip(group, need))), -1, np.int64)
    starts = np.concatenate([[0], np.cumsum(pre)]) // page
    at = int(starts[-1])
    for b, n in enumerate(need):
        s = pre[group[b]] // page
        table[b, :s] = np.arange(starts[group[b]], starts[group[b]] + s)
        table[b, s: s + n] = np.arange(at, at + n)
        at += n
    table = torch.from_numpy(table).cuda()
    st["table"] = torch.where(table >= 0, order[table.clamp(min=0)], torch.full_like(table, -1, dtype=torch.int32))
    st["kp"], _ = _pool(c, pages, gen)
    st["vp"], _ = _pool(c, pages, gen)
    st["q"] = torch.randn((len(tails), c["Q"], Hq, D), generator=gen, device="cuda").to(dtype)
    st["lens"] = ints([pre[g] + t for g, t in zip(group, tails)])
    st["cu"], st["pre"] = ints([0, *np.cumsum(sizes).tolist()]), ints(pre)
    st["most"] = (max(sizes), max(pre), max(tails))
    return st


# ------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, rot, pairs):
    """x [..., H, D] in 32 bits; cos, sin [..., rot / 2] of its rows."""
    c, s = cos[..., None, :], sin[..., None, :]
    y = x.clone()
    if pairs == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _rope(st):
    pos = torch.arange(st["N"], device="cuda") if st["pos"] is None else st["pos"].long()
    cos, sin = st["cos"][pos], st["sin"][pos] * (-1.0 if st["back"] else 1.0)
    return tuple(_rotate(st[n].float(), cos, sin, st["rot"], st["pairs"]).to(st[n].dtype) for n in ("q", "k"))


def _append_8bit(x, pages, scales, st):
    """Writes the fp32 rows [B, N, Hkv, D] behind each sequence's into blocks of codes; a block that gets rows is read, requantised and written."""
    P, page, Hkv, D = pages.shape
    nb, blk, code, lens, new = scales.shape[1], st["block"], st["code"], st["lens"].long(), st["new"].long()
    B, N = x.shape[:2]
    j = (lens // blk)[:, None] + torch.arange(_ceil(N - 1, blk) + 1, device=x.device)  # [B, T] blocks
    entry = j * blk // page
    touched = (j * blk < (lens + new)[:, None]) & (new > 0)[:, None] & (entry < st["table"].shape[1])
    pg = st["table"].gather(1, entry.clamp(max=st["table"].shape[1] - 1)).long().clamp(0, P - 1)
    i = j[:, :, None] * blk + torch.arange(blk, device=x.device) - lens[:, None, None]
    is_new = ((i >= 0) & (i < new[:, None, None]))[..., None, None]
    rows = x[torch.arange(B, device=x.device)[:, None, None], i.clamp(0, N - 1)]       # [B, T, blk, Hkv, D]
    rows = torch.where(is_new, rows, torch.zeros_like(rows))
    mag = torch.where(torch.isnan(rows), torch.full_like(rows, math.inf), rows.abs())
    need, have, sub = _scale_for(mag.amax(dim=(2, 4)), code), scales[pg, j % nb], j % nb
    s = torch.where((j * blk >= lens[:, None])[..., None], need, torch.maximum(have, need))
    raw = pages.view(torch.uint8).view(P, nb, blk, Hkv, D)
    was = raw[pg, sub]
    old = was.view(pages.dtype).float() * (have / s)[:, :, None, :, None]
    old = torch.where(torch.isfinite(old), old, torch.zeros_like(old))
    old = torch.round(old).to(torch.int8) if code == "int8" else old.to(torch.float8_e4m3fn)
    put = _quantize(rows, s[:, :, None, :, None], code)
    out = torch.where(is_new, put.view(torch.uint8), torch.where((i < 0)[..., None, None], old.view(torch.uint8), was))
    raw[pg[touched], sub[touched]] = out[touched]
    scales[pg[touched], sub[touched]] = s[touched]


def _append(st):
    lens, new = st["lens"].long(), st["new"].long()
    B, N, page = lens.shape[0], st["N"], st["page"]
    i = torch.arange(N, device="cuda").expand(B, N)
    real = i < new[:, None]
    q, k, v = st["q"], st["k"], st["v"]
    if st["packed"]:  # rows of the padded form
        row = (st["cu"][:-1].long()[:, None] + i).clamp(max=max(0, q.shape[0] - 1))
        q, k, v = q[row], k[row], v[row]
    pos = lens[:, None] + i
    cos, sin = (t[pos.clamp(max=t.shape[0] - 1)] for t in (st["cos"], st["sin"]))
    qr = _rotate(q.float(), cos, sin, st["rot"], st["pairs"])
    kr = _rotate(k.float(), cos, sin, st["rot"], st["pairs"])
    if st["code"] != "none":
        _append_8bit(kr, st["kp"], st["ks"], st)
        _append_8bit(v.float(), st["vp"], st["vs"], st)
    else:
        pg = st["table"].gather(1, (pos // page).clamp(max=st["table"].shape[1] - 1)).long()[real]
        st["kp"][pg, pos[real] % page] = kr[real].to(st["kp"].dtype)
        st["vp"][pg, pos[real] % page] = v[real]
    if st["packed"]:
        return qr[real].to(q.dtype)
    return torch.where(real[..., None, None], qr, torch.zeros_like(qr)).to(q.dtype)


def _shared(st):
    q, lens, pre, cu, page = st["q"], st["lens"].long(), st["pre"].long(), st["cu"].long(), st["page"]
    B, Q, Hq, D = q.shape
    Hkv, (most, K, T) = st["Hkv"], st["most"]
    G, dev = Hq // Hkv, q.device
    seq = torch.arange(B, device=dev)
    group = torch.searchsorted(cu, seq, right=True) - 1
    place = seq - cu[group]
    own_from = pre[group]
    rows = q.float().view(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D) * (1.0 / math.sqrt(D))
    last = ((lens - Q)[:, None] + torch.arange(Q, device=dev)).repeat_interleave(G, 1)  # [B, Q * G]

    def keys(table, pools):  # [X, entries] -> [X, Hkv, entries * page, D] in 32 bits
        x = pools[table.long().clamp(0, pools.shape[0] - 1)].float()
        return x.view(table.shape[0], -1, Hkv, D).transpose(1, 2)

    # the shared keys: the rows of a group's members together
    shared = st["table"][cu[:-1], : _ceil(K, page)]
    packed = torch.zeros((pre.shape[0], most, Hkv, Q * G, D), device=dev)
    packed[group, place] = rows
    packed = packed.transpose(1, 2).reshape(-1, Hkv, most * Q * G, D)
    s1 = torch.matmul(packed, keys(shared, st["kp"]).transpose(2, 3)).view(-1, Hkv, most, Q * G, shared.shape[1] * page)
    s1 = s1.transpose(1, 2)[group, place]                                              # [B, Hkv, Q * G, K]
    at = torch.arange(s1.shape[-1], device=dev)
    s1 = s1.masked_fill(((at >= own_from[:, None, None]) | (at > last[..., None]))[:, None], -math.inf)
    # the keys of each sequence alone
    entry = (own_from // page)[:, None] + torch.arange(_ceil(T, page), device=dev)
    entry = st["table"].gather(1, entry.clamp(max=st["table"].shape[1] - 1))
    s2 = torch.matmul(rows, keys(entry, st["kp"]).transpose(2, 3))
    at = own_from[:, None] + torch.arange(s2.shape[-1], device=dev)
    s2 = s2.masked_fill(((at >= lens[:, None])[:, None] | (at[:, None] > last[..., None]))[:, None], -math.inf)
    m = torch.maximum(s1.amax(-1), s2.amax(-1))
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p1, p2 = torch.exp(s1 - m[..., None]), torch.exp(s2 - m[..., None])
    total = p1.sum(-1) + p2.sum(-1)
    packed = torch.zeros((pre.shape[0], most, Hkv, Q * G, p1.shape[-1]), device=dev)
    packed[group, place] = p1
    o = torch.matmul(packed.transpose(1, 2).reshape(-1, Hkv, most * Q * G, p1.shape[-1]), keys(shared, st["vp"]))
    o = o.view(-1, Hkv, most, Q * G, D).transpose(1, 2)[group, place]
    o = (o + torch.matmul(p2, keys(entry, st["vp"]))) / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    back = lambda t: t.view(B, Hkv, Q, G, -1).transpose(1, 2).reshape(B, Q, Hq, -1)  # noqa: E731
    return back(o).to(q.dtype), back(m + torch.log(total)).squeeze(-1)


def _buffers(st):
    """The pages, and the scales of 8-bit ones."""
    return [st[n] for n in ("kp", "vp", "ks", "vs") if st[n] is not None]


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "rope":
        return _rope(st)
    if st["op"] == "append":
        return (_append(st), *_buffers(st))
    return _shared(st)


def _run_own(st):
    import causal_gqa_attention_online_gb300 as attn
    if st["op"] == "rope":
        f = attn.attn_rope_bwd if st["back"] else attn.attn_rope
        return f(st["q"], st["k"], st["cos"], st["sin"], positions=st["pos"], pairs=st["pairs"])
    if st["op"] == "shared":
        return attn.attn_fwd_paged_shared(st["q"], st["kp"], st["vp"], st["table"], st["lens"], st["cu"], st["pre"])
    qkv, angles, cache = (st["q"], st["k"], st["v"]), (st["cos"], st["sin"]), (st["kp"], st["vp"])
    where = (st["table"], st["lens"])
    if st["code"] != "none":
        cache += (st["ks"], st["vs"])
        if st["packed"]:
            q = attn.attn_rope_append_q8_varlen(*qkv, st["cu"], st["N"], *angles, *cache, *where, pairs=st["pairs"])
        else:
            q = attn.attn_rope_append_q8(*qkv, *angles, *cache, *where, seqlens_new=st["new"], pairs=st["pairs"])
    elif st["packed"]:
        q = attn.attn_rope_append_varlen(*qkv, st["cu"], st["N"], *angles, *cache, *where, pairs=st["pairs"])
    else:
        q = attn.attn_rope_append(*qkv, *angles, *cache, *where, seqlens_new=st["new"], pairs=st["pairs"])
    return (q, *_buffers(st))


# ------------------------------------------------------------------ 64 bits

def _turned(x, cos, sin, rot, pairs):
    """Pairs as complex numbers, turned; x [rows, H, D] in 64 bits, cos and sin [rows, rot / 2]."""
    t = torch.complex(cos, sin)[:, None]
    if pairs == "half":
        z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * t
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)
    z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * t
    return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)


def _e4m3_values():
    """The finite values of e4m3, ascending."""
    v = [m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
    return np.array([-x for x in v[:0:-1]] + v)


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "rope":
        pos = torch.arange(c["N"], device="cuda").expand(c["B"], -1) if st["pos"] is None else st["pos"].long()
        pos = pos.reshape(-1)
        cos, sin = st["cos"].double()[pos], st["sin"].double()[pos]
        sin = -sin if c["back"] else sin
        return tuple(_turned(st[n].double().flatten(0, 1), cos, sin, c["rot"], c["pairs"]).view(st[n].shape) for n in ("q", "k"))
    if c["op"] == "append":
        return _exact_append(c, st)
    Q, Hq, Hkv, D, page = c["Q"], c["Hq"], c["Hkv"], c["D"], c["page"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        j = torch.arange(n, device="cuda")
        pg = st["table"][b].long()[j // page]
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k, v = st["kp"][pg, j % page, h].double(), st["vp"][pg, j % page, h].double()
            s = torch.einsum("ihd,kd->ihk", st["q"][b, :, heads].double(), k) / math.sqrt(D)
            s = s.masked_fill((j > (torch.arange(Q, device="cuda") + n - Q)[:, None])[:, None], -math.inf)
            lse[b, :, heads] = torch.logsumexp(s, -1)
            o[b, :, heads] = torch.einsum("ihk,kd->ihd", torch.exp(s - lse[b, :, heads, None]), v)
    return o, lse


def _exact_append(c, st):
    lens, new, page, blk = st["lens"].tolist(), st["new"].tolist(), c["page"], c["block"]
    q = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    eight = c["code"] != "none"
    if eight:
        if c["code"] == "int8":  # its codes are whole numbers
            pools = scales = [None, None]
        else:
            pools = [p.float().double() for p in (st["kp"], st["vp"])]
            scales = [s.double() for s in (st["ks"], st["vs"])]
            steps = torch.from_numpy(_e4m3_values()).cuda()
    else:
        pools = [p.double() for p in (st["kp"], st["vp"])]
    for b in range(c["B"]):
        if not new[b]:
            continue
        rows = (lambda t: t[st["cu"][b]: st["cu"][b + 1]]) if c["packed"] else (lambda t: t[b, : new[b]])
        pos = torch.arange(lens[b], lens[b] + new[b], device="cuda")
        cos, sin = st["cos"].double()[pos], st["sin"].double()[pos]
        rows(q)[:] = _turned(rows(st["q"]).double(), cos, sin, c["rot"], c["pairs"])
        if eight and c["code"] == "int8":
            continue
        pg = st["table"][b].long()
        for w, x in enumerate((_turned(rows(st["k"]).double(), cos, sin, c["rot"], c["pairs"]), rows(st["v"]).double())):
            if not eight:
                pools[w][pg[pos // page], pos % page] = x
                continue
            # scales by block from 64-bit logarithms, codes by search among the values
            first, end = lens[b] // blk, lens[b] + new[b]
            full = torch.zeros(((_ceil(end, blk) - first) * blk, *x.shape[1:]), dtype=torch.float64, device="cuda")
            full[pos - first * blk] = x
            a = full.view(-1, blk, *x.shape[1:]).abs().amax((1, 3))
            e = torch.ceil(torch.log2((a / 448.0).clamp(min=2.0 ** -1000))).clamp(min=-100)
            e = torch.where(a > 448.0 * torch.exp2(e), e + 1, torch.where((a <= 448.0 * torch.exp2(e - 1)) & (e > -100), e - 1, e))
            s = torch.exp2(e)
            at = torch.arange(first, first + s.shape[0], device="cuda")
            bp, sub = pg[at * blk // page], at * blk % page // blk
            nearest = lambda y: steps[torch.searchsorted((steps[1:] + steps[:-1]) / 2, y.contiguous())]  # noqa: E731
            if lens[b] % blk:  # rows that were there, under the larger scale
                had = scales[w][bp[0], sub[0]].clone()
                s[0] = torch.maximum(s[0], had)
                t = torch.arange(first * blk, lens[b], device="cuda")
                old = pools[w][bp[0], t % page]
                pools[w][bp[0], t % page] = torch.where((s[0] > had)[:, None], nearest(old * (had / s[0])[:, None]), old)
            scales[w][bp, sub] = s
            pools[w][pg[pos // page], pos % page] = nearest(x / s[pos // blk - first][..., None])
    return (q, *pools, *scales) if eight else (q, *pools)
