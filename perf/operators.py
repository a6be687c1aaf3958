"""The operators of an 8-bit paged K/V cache, as cases that can be measured.

Each case is one call of a serving program: attention over the cache
(``attend``), writing new keys and values into it (``append``), and the
management of its pages (``copy``, ``fork``, ``compact``).  ``run`` computes a
case with elementary torch operations, or through the package's entry points
when ``own`` is set; ``exact`` computes the same in 64 bits.

Layout: pages [P, page, Hkv, D] of int8 or e4m3 codes, one fp32 scale for each
block of ``block`` tokens of a page and head [P, page / block, Hkv]; key j of a
sequence is row j % page of page block_table[b, j // page], and stands for
code * scale.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_QMAX = {"int8": 127.0, "e4m3": 448.0}
_MIN_EXP = -100  # the smallest scale is 2^-100


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a single conversation: the latency of one token's attention
        dict(name="attend b1 k700", op="attend", B=1, Q=1, Hq=32, Hkv=8, D=128, K=700, page=64,
             block=64, code="e4m3", dtype="bf16", window=0),
        # the batched decode of the benchmark (64 ragged sequences up to 8192 keys), cache in int8
        dict(name="attend b64 k8192", op="attend", B=64, Q=1, Hq=32, Hkv=8, D=128, K=8192, page=64,
             block=64, code="int8", dtype="bf16", window=0),
        # two documents of 100 thousand tokens, four drafted tokens each, 64-wide heads
        dict(name="attend b2 q4 k100003", op="attend", B=2, Q=4, Hq=16, Hkv=4, D=64, K=100003,
             page=128, block=32, code="e4m3", dtype="fp16", window=0),
        # chunked prefill: 512 new rows of each of four sequences over what is cached
        dict(name="attend b4 q512 k8192", op="attend", B=4, Q=512, Hq=32, Hkv=8, D=128, K=8192,
             page=64, block=64, code="e4m3", dtype="bf16", window=0),
        # one token of every sequence of a decode batch
        dict(name="append b64 n1", op="append", B=64, N=1, Hkv=8, D=128, K=8192, page=64, block=64,
             code="int8", dtype="bf16"),
        # prompts: ragged, up to 4096 rows a sequence
        dict(name="append b16 n4096", op="append", B=16, N=4096, Hkv=8, D=128, K=4096, page=64,
             block=64, code="e4m3", dtype="bf16"),
        # a few small pages of one layer (a shared prefix of a short prompt)
        dict(name="copy 7 pages", op="copy", n=7, layers=1, Hkv=2, D=64, page=16, block=16,
             code="int8"),
        # a long prompt's pages of eight layers into another place
        dict(name="copy 500 pages", op="copy", n=500, layers=8, Hkv=8, D=128, page=64, block=64,
             code="int8"),
        # one beam search step: four beams of each of four requests, short
        dict(name="fork 4x4 k300", op="fork", groups=4, beams=4, K=300, layers=1, Hkv=8, D=128,
             page=64, block=64, code="int8"),
        # eight beams of 32 requests over long contexts, four layers of pages
        dict(name="fork 32x8 k8192", op="fork", groups=32, beams=8, K=8192, layers=4, Hkv=8, D=128,
             page=64, block=64, code="int8"),
        # a small pool with holes
        dict(name="compact 100 pages", op="compact", B=4, K=1000, holes=0.5, layers=1, Hkv=2, D=64,
             page=64, block=64, code="int8"),
        # a pool half empty after many requests have left
        dict(name="compact 4096 pages", op="compact", B=64, K=4096, holes=0.5, layers=4, Hkv=8,
             D=128, page=64, block=64, code="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "copy", "fork", "compact"])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    c = dict(op=op, Hkv=rng.randint(1, 8), D=rng.choice([64, 64, 96, 128, 128, 128, 80, 256]),
             page=page, block=rng.choice([b for b in (8, 16, 32, 64, 128) if b <= page]),
             code=rng.choice(["int8", "e4m3"]))
    width = c["Hkv"] * c["D"]
    if op == "attend":
        c["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
        c["Q"] = rng.choice([1, 1, 1, rng.randint(2, 4), _log(rng, 5, 512)])
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 4, 6, 8])
        c["B"] = _log(rng, 1, 64) if c["Q"] <= 4 else rng.randint(1, 4)
        most = min(100003, 64 * 8192 * 1024 // (c["B"] * width))
        if c["Q"] > 4:
            most = min(most, 8192, 4 * 512 * 32 * 128 * 8192 // (c["B"] * c["Q"] * c["Hq"] * c["D"]))
        c["K"] = max(c["Q"], _log(rng, 32, max(64, most)))
        c["window"] = rng.choice([0, 0, 0, rng.randint(1, 2 * c["K"])])
    elif op == "append":
        c["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c["B"] = _log(rng, 1, 64)
        c["N"] = rng.choice([1, _log(rng, 2, max(3, min(4096, 16 * 4096 * 1024 // (c["B"] * width))))])
        c["K"] = c["N"] + _log(rng, 1, 2048)
    else:
        c["layers"] = rng.randint(1, 4)
        size = width * page * c["layers"]
        if op == "copy":
            c["n"] = _log(rng, 1, max(2, min(500, 500 * 8 * 65536 // size)))
        elif op == "fork":
            c["groups"], c["beams"] = _log(rng, 1, 32), rng.randint(2, 8)
            c["K"] = _log(rng, 1, max(2, min(8192, 4 * 32 * 8192 * 1024 // (c["groups"] * width * c["layers"]))))
        else:
            c["B"] = _log(rng, 1, 64)
            c["K"] = _log(rng, 16, max(32, min(4096, 64 * 4096 * 4096 // (c["B"] * width * c["layers"]))))
            c["holes"] = round(rng.uniform(0.1, 0.9), 2)
    return c


def _lens(n, most):
    """Ragged lengths that the case alone decides: the first is `most`, the others spread over [0, most]."""
    return [most if b == 0 else (most + 1) * ((b * 40503 + 9973) % 65536) >> 16 for b in range(n)]


def _ceil(a, b):
    return -(-a // b)


def work(c):
    width = c["Hkv"] * c["D"]
    es = {"bf16": 2, "fp16": 2, "fp32": 4}.get(c.get("dtype"), 0)
    if c["op"] == "attend":
        keys = pairs = 0
        for n in _lens(c["B"], c["K"]):
            lo = max(0, n - c["Q"] - c["window"] + 1) if c["window"] else 0
            keys += n - lo
            for off in (range(c["Q"]) if c["Q"] <= 4 or c["window"] else ()):
                hi = max(0, n - c["Q"] + off + 1)
                pairs += hi - (max(0, hi - c["window"]) if c["window"] else 0)
            if not (c["Q"] <= 4 or c["window"]):
                r = min(c["Q"], n)
                pairs += r * n - r * (r - 1) // 2
        rows = c["B"] * c["Q"] * c["Hq"]
        return {"bytes": keys * (2 * width + 8 * c["Hkv"] / c["block"]) + rows * (2 * c["D"] * es + 4),
                "flops": 4 * pairs * c["Hq"] * c["D"]}
    if c["op"] == "append":
        n = sum(min(c["N"], x) for x in _lens(c["B"], c["N"]))
        return {"bytes": 2 * n * width * (es + 1) + 8 * n * c["Hkv"] / c["block"], "flops": 2 * n * width}
    page_bytes = 2 * c["page"] * width + 8 * c["Hkv"] * (c["page"] // c["block"])
    if c["op"] == "copy":
        return {"bytes": c["n"] * (8 + 2 * c["layers"] * page_bytes), "flops": 0}
    if c["op"] == "fork":
        m = _ceil(c["K"] + 1, c["page"])
        copies = sum((c["beams"] // 2) * (n % c["page"] > 0) for n in _lens(c["groups"], c["K"]))
        entries = c["groups"] * c["beams"] * m
        return {"bytes": 8 * entries + 8 * _pool_pages(c) + 2 * copies * c["layers"] * page_bytes, "flops": 0}
    pages = sum(_ceil(n, c["page"]) for n in _lens(c["B"], c["K"]))
    total = _pool_pages(c)
    moved = max(0, round(pages * (1 - pages / total)))
    return {"bytes": 8 * c["B"] * _ceil(c["K"], c["page"]) + 12 * total + 2 * moved * c["layers"] * page_bytes, "flops": 0}


def _pool_pages(c):
    if c["op"] == "fork":
        used = sum(_ceil(n, c["page"]) + c["beams"] for n in _lens(c["groups"], c["K"]))
        return used + 2 * c["groups"] * c["beams"] + 8
    if c["op"] == "copy":
        return 2 * c["n"] + 5
    if c["op"] == "compact":
        pages = sum(_ceil(n, c["page"]) for n in _lens(c["B"], c["K"]))
        return max(pages + 1, int(pages / (1 - c["holes"])))
    return sum(max(1, _ceil(n, c["page"])) for n in _lens(c["B"], c["K"])) + 3


# ------------------------------------------------------------------ inputs

def _activations(shape, gen, dtype):
    """Keys / values as a layer makes them: normal, with a spread over the channels and some larger rows."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.7 * torch.randn(shape[-1:], generator=gen, device="cuda"))
    x *= torch.exp2(torch.randint(-1, 2, shape[:-1] + (1,), generator=gen, device="cuda").float())
    return x.to(dtype)


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
    """A pool of pages that hold quantised activations, and its scales."""
    x = _activations((pages, c["page"], c["Hkv"], c["D"]), gen, torch.bfloat16).float()
    x = x.view(pages, c["page"] // c["block"], c["block"], c["Hkv"], c["D"])
    s = _scale_for(x.abs().amax(dim=(2, 4)), c["code"])
    y = _quantize(x, s[:, :, None, :, None], c["code"])
    return y.view(pages, c["page"], c["Hkv"], c["D"]), s


def _pages_of(lens, page, m, pages, gen):
    """A block table whose sequences own shuffled pages; -1 where they own none."""
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    need = [max(1, _ceil(n, page)) for n in lens]
    at = np.full((len(lens), m), -1, np.int64)
    ends = np.cumsum(need)
    for b, (n, e) in enumerate(zip(need, ends)):
        at[b, :n] = np.arange(e - n, e)
    at = torch.from_numpy(at).cuda()
    return torch.where(at >= 0, order[at.clamp(min=0)], torch.full_like(at, -1, dtype=torch.int32))


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(c)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = _pool_pages(c)
    if c["op"] in ("attend", "append"):
        m = max(1, _ceil(c["K"], c["page"]))
        st["kp"], st["ks"] = _pool(c, pages, gen)
        st["vp"], st["vs"] = _pool(c, pages, gen)
        lens = _lens(c["B"], c["K"])
        st["table"] = _pages_of(lens, c["page"], m, pages, gen)
        if c["op"] == "attend":
            q = torch.randn((c["B"], c["Q"], c["Hq"], c["D"]), generator=gen, device="cuda")
            st["q"], st["lens"] = q.to(_DTYPES[c["dtype"]]), ints(lens)
        else:  # the last rows of each sequence are new
            new = [min(n, x) for n, x in zip(lens, _lens(c["B"], c["N"]))]
            st["lens"] = ints([n - x for n, x in zip(lens, new)])
            st["new"] = ints(new)
            shape = (c["B"], c["N"], c["Hkv"], c["D"])
            st["k"] = _activations(shape, gen, _DTYPES[c["dtype"]])
            st["v"] = _activations(shape, gen, _DTYPES[c["dtype"]])
        return st
    st["pools"] = []
    for _ in range(c["layers"]):
        st["pools"] += [*_pool(c, pages, gen), *_pool(c, pages, gen)]
    if c["op"] == "copy":
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        st["src"], st["dst"] = order[: c["n"]].contiguous(), order[c["n"]: 2 * c["n"]].contiguous()
    elif c["op"] == "compact":
        lens = _lens(c["B"], c["K"])
        st["table"] = _pages_of(lens, c["page"], max(1, _ceil(c["K"], c["page"])), pages, gen)
        held = torch.tensor(lens, device="cuda")[:, None] > torch.arange(st["table"].shape[1], device="cuda") * c["page"]
        st["table"] = torch.where(held, st["table"], torch.full_like(st["table"], -1))
        st["refs"] = torch.bincount(st["table"][held].long(), minlength=pages).to(torch.int32)
    else:
        # beams of a request share their full pages; each has a last page of its own
        m, beams = _ceil(c["K"] + 1, c["page"]), c["beams"]
        lens = _lens(c["groups"], c["K"])
        shared = _pages_of([n // c["page"] * c["page"] for n in lens], c["page"], m, pages - c["groups"] * beams, gen)
        full = torch.tensor([n // c["page"] for n in lens], device="cuda").repeat_interleave(beams)
        part = torch.tensor([n % c["page"] > 0 for n in lens], device="cuda").repeat_interleave(beams)
        table = shared.repeat_interleave(beams, 0)
        at = torch.arange(m, device="cuda")[None]
        tails = torch.arange(pages - c["groups"] * beams, pages, device="cuda", dtype=torch.int32)[:, None]
        table = torch.where(at < full[:, None], table, torch.where((at == full[:, None]) & part[:, None], tails, torch.full_like(table, -1)))
        st["table"] = table.contiguous()
        st["lens"] = ints(lens).repeat_interleave(beams)
        st["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
        # each kept beam goes on twice (the last one once where their number is odd)
        pick = torch.rand((c["groups"], beams), generator=gen, device="cuda").argsort(1)
        child = pick[:, torch.arange(beams, device="cuda") // 2] + beams * torch.arange(c["groups"], device="cuda")[:, None]
        st["parents"] = child.reshape(-1).to(torch.int32)
        st["new"] = torch.ones_like(st["parents"])
    return st


# ------------------------------------------------------------------ plain forms

def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _gathered(pages, scales, table, dtype):
    """The keys or values of every sequence [B, M * page, Hkv, D] as numbers."""
    at = table.long().clamp(0, pages.shape[0] - 1)
    x = _bytes(pages)[at].view(pages.dtype).to(dtype)
    B, M, page, Hkv, D = x.shape
    nb = scales.shape[1]
    x = x.view(B, M, nb, page // nb, Hkv, D) * scales[at].to(dtype)[:, :, :, None, :, None]
    return x.view(B, M * page, Hkv, D)


def _attend(st):
    q, lens = st["q"], st["lens"].long()
    B, Q, Hq, D = q.shape
    k = _gathered(st["kp"], st["ks"], st["table"], torch.float32)
    v = _gathered(st["vp"], st["vs"], st["table"], torch.float32)
    K, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    key = torch.arange(K, device=q.device)
    diag = torch.arange(Q, device=q.device)[None] + (lens - Q)[:, None]          # [B, Q]
    legal = key <= diag[:, :, None]
    if st["window"]:
        legal &= key > diag[:, :, None] - st["window"]
    v = v * (key < lens[:, None])[:, :, None, None]
    rows = q.float().view(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)
    s = torch.matmul(rows, k.permute(0, 2, 3, 1)).view(B, Hkv, G, Q, K) * (1.0 / math.sqrt(D))
    s = s.masked_fill(~legal[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(B, Q, Hq)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p.view(B, Hkv, G * Q, K), v.permute(0, 2, 1, 3)).view(B, Hkv, G, Q, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D).to(q.dtype), lse


def _append_one(x, pages, scales, st):
    """Writes the rows of `x` behind each sequence's; the blocks that get rows are read, requantised and written."""
    P, page, Hkv, D = pages.shape
    nb, blk, code, lens, new = scales.shape[1], st["block"], st["code"], st["lens"].long(), st["new"].long()
    B, N = x.shape[:2]
    first = lens // blk
    # blocks that a sequence's new rows can touch
    j = first[:, None] + torch.arange(_ceil(N - 1, blk) + 1, device=x.device)    # [B, T]
    touched = (j * blk < (lens + new)[:, None]) & (new > 0)[:, None]
    pg = st["table"].gather(1, (j * blk // page).clamp(max=st["table"].shape[1] - 1)).long()
    touched &= (pg >= 0) & (pg < P) & (j * blk // page < st["table"].shape[1])
    pos = j[:, :, None] * blk + torch.arange(blk, device=x.device)               # [B, T, blk]
    i = pos - lens[:, None, None]
    is_new = (i >= 0) & (i < new[:, None, None])
    is_old = i < 0
    b = torch.arange(B, device=x.device)[:, None, None]
    rows = x[b, i.clamp(0, N - 1)].float() * is_new[..., None, None]
    rows = torch.where(is_new[..., None, None], rows, torch.zeros_like(rows))    # [B, T, blk, Hkv, D]
    mag = torch.where(torch.isnan(rows), torch.full_like(rows, math.inf), rows.abs())
    need = _scale_for(mag.amax(dim=(2, 4)), code)
    keep = pg.clamp(0, P - 1)
    sub = j % nb
    have = scales[keep, sub]
    s = torch.where((j * blk >= lens[:, None])[..., None], need, torch.maximum(have, need))
    held = _bytes(pages).view(P, nb, blk, Hkv, D)
    old = held[keep, sub].view(pages.dtype).float() * (have / s)[:, :, None, :, None]
    old = torch.where(torch.isfinite(old), old, torch.zeros_like(old))
    old = torch.round(old).to(torch.int8) if code == "int8" else old.to(torch.float8_e4m3fn)
    put = _quantize(rows, s[:, :, None, :, None], code)
    was = held[keep, sub]
    out = torch.where(is_new[..., None, None], _bytes(put), torch.where(is_old[..., None, None], _bytes(old), was))
    held[keep[touched], sub[touched]] = out[touched]
    scales[keep[touched], sub[touched]] = s[touched]


def _fork(st):
    table, lens, refs, page = st["table"], st["lens"].long(), st["refs"], st["page"]
    S, M = table.shape
    P = refs.shape[0]
    par, N = st["parents"].long(), st["parents"].shape[0]
    some = (par >= 0) & (par < S)
    n = torch.where(some, lens[par.clamp(0, S - 1)].clamp(0, M * page), torch.zeros_like(par))
    want = (n + torch.where(some, st["new"].long().clamp(min=0), torch.zeros_like(par)) + page - 1) // page
    wide = (want > M).sum()
    at = torch.arange(M, device=table.device)[None]
    cand = torch.where(some[:, None], table[par.clamp(0, S - 1)].long(), torch.full_like(at, -1))
    ok = (cand >= 0) & (cand < P)
    full = at < (n // page)[:, None]
    todo = ~full & (at < want[:, None])
    one = lambda t: t.reshape(-1)  # noqa: E731
    count = lambda t, w: torch.zeros(P + 1, dtype=torch.long, device=t.device).index_add_(  # noqa: E731
        0, one(torch.where(w, t, torch.full_like(t, P))), torch.ones_like(one(t)))[:P]
    was = count(table.long(), (table >= 0) & (table < P))
    pinned = (count(cand, ok & full) > 0) | (refs > was)
    line = torch.arange(N * M, device=table.device)
    claim = torch.full((P + 1,), N * M, device=table.device).scatter_reduce_(
        0, one(torch.where(ok & todo, cand, torch.full_like(cand, P))), line, "amin")
    c = cand.clamp(0, P - 1)
    keep = todo & ok & (refs[c] > 0) & ~pinned[c] & (claim[c] == line.view(N, M))
    get = todo & ~keep
    free = torch.where(refs == 0, torch.arange(P, device=table.device), torch.full_like(refs, P, dtype=torch.long)).sort().values
    total = get.sum()
    missing = (total - (refs == 0).sum()).clamp(min=0)
    fine = (missing == 0) & (wide == 0)
    taken = free[(one(get).cumsum(0).view(N, M) - 1).clamp(0, P - 1)]
    none = torch.full_like(cand, -1)
    out = torch.where(fine, torch.where(get, taken, torch.where((full & ok) | keep, cand, none)), none)
    left = torch.where(fine, refs - was + count(out, out >= 0), refs).to(torch.int32)
    moves = get & ok & fine & (at == (n // page)[:, None]) & (n % page > 0)[:, None]
    src, dst = cand[moves], out[moves]
    [_bytes(p).index_copy_(0, dst, _bytes(p)[src]) for p in st["pools"]]
    status = torch.stack([missing, wide, torch.where(fine, total, 0), moves.sum()]).to(torch.int32)
    return out.to(torch.int32), torch.where(fine, n, 0).to(torch.int32), left, status


def _compact(st):
    table, refs = st["table"], st["refs"]
    P = refs.shape[0]
    live = refs > 0
    n = live.sum()
    at = torch.arange(P, device=refs.device)
    src = at[live & (at >= n)]
    dst = at[~live & (at < n)]
    remap = torch.where(live, at, torch.full_like(at, -1))
    remap[src] = dst
    [_bytes(p).index_copy_(0, dst, _bytes(p)[src]) for p in st["pools"]]
    ok = (table >= 0) & (table < P)
    out = torch.where(ok, remap[table.long().clamp(0, P - 1)], torch.full_like(table, -1, dtype=torch.long))
    left = torch.zeros_like(refs).index_copy_(0, remap[live], refs[live])
    return out.to(torch.int32), left, remap.to(torch.int32), n.to(torch.int32)


def run(st):
    if own:
        return _run_own(st)
    if st["op"] == "attend":
        return _attend(st)
    if st["op"] == "append":
        _append_one(st["k"], st["kp"], st["ks"], st)
        _append_one(st["v"], st["vp"], st["vs"], st)
        return st["kp"], st["vp"], st["ks"], st["vs"]
    if st["op"] == "copy":
        src, dst = st["src"].long(), st["dst"].long()
        [_bytes(p).index_copy_(0, dst, _bytes(p)[src]) for p in st["pools"]]
        return st["pools"]
    return (*(_fork(st) if st["op"] == "fork" else _compact(st)), st["pools"])


def _run_own(st):
    import causal_gqa_attention_online_gb300 as attn
    if st["op"] == "attend":
        return attn.attn_fwd_paged_q8(st["q"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"],
                                      st["lens"], window=st["window"])
    if st["op"] == "append":
        attn.attn_cache_append(st["k"], st["v"], st["kp"], st["vp"], st["ks"], st["vs"], st["table"],
                               st["lens"], seqlens_new=st["new"])
        return st["kp"], st["vp"], st["ks"], st["vs"]
    if st["op"] == "copy":
        attn.attn_pages_copy(st["pools"], st["pools"], st["src"], st["dst"])
        return st["pools"]
    if st["op"] == "fork":
        return (*attn.attn_pages_fork(st["pools"], st["table"], st["lens"], st["refs"], st["parents"],
                                      st["page"], new_tokens=st["new"]), st["pools"])
    return (*attn.attn_pages_compact(st["pools"], st["table"], st["refs"]), st["pools"])


# ------------------------------------------------------------------ 64 bits

def _e4m3_values():
    """What the codes 0..255 of e4m3 stand for (NaN at 127 and 255)."""
    v = [(m / 8.0 * 2.0 ** -6) if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    v[127] = math.nan
    return np.array(v + [-x for x in v])


def exact(c, seed):
    if c["op"] not in ("attend", "append"):
        return None  # whole numbers and copies
    st = prepare(c, seed)
    values = torch.from_numpy(_e4m3_values()).cuda()
    as64 = lambda t: values[t.view(torch.uint8).long()] if t.dtype == torch.float8_e4m3fn else t.double()  # noqa: E731
    page, block, D = c["page"], c["block"], c["D"]
    if c["op"] == "attend":
        B, Q, Hq, Hkv = c["B"], c["Q"], c["Hq"], c["Hkv"]
        o = torch.zeros((B, Q, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.full((B, Q, Hq), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(st["lens"].tolist()):
            j = torch.arange(n, device="cuda")
            pg = st["table"][b].long()[j // page]
            for h in range(Hkv):
                k = as64(st["kp"][:, :, h][pg, j % page] if c["code"] == "int8" else st["kp"].view(torch.uint8)[:, :, h][pg, j % page].view(torch.float8_e4m3fn))
                v = as64(st["vp"][:, :, h][pg, j % page] if c["code"] == "int8" else st["vp"].view(torch.uint8)[:, :, h][pg, j % page].view(torch.float8_e4m3fn))
                k = k * st["ks"][pg, j % page // block, h].double()[:, None]
                v = v * st["vs"][pg, j % page // block, h].double()[:, None]
                heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                for i0 in range(max(0, Q - n), Q, 64):
                    i = torch.arange(i0, min(Q, i0 + 64), device="cuda")
                    last = i + n - Q
                    s = torch.einsum("ihd,kd->ihk", st["q"][b, i, heads].double(), k) / math.sqrt(D)
                    bad = j[None] > last[:, None]
                    if c["window"]:
                        bad |= j[None] <= last[:, None] - c["window"]
                    s = s.masked_fill(bad[:, None], -math.inf)
                    z = torch.logsumexp(s, -1)
                    lse[b, i, heads] = z
                    o[b, i, heads] = torch.einsum("ihk,kd->ihd", torch.exp(s - z[..., None]), v)
        return o, lse
    # append: scales as 64-bit logarithms, codes by search among the values
    out = []
    qmax = _QMAX[c["code"]]
    table, lens, new = st["table"].cpu().numpy(), st["lens"].tolist(), st["new"].tolist()
    steps = np.arange(-127, 128.0) if c["code"] == "int8" else np.unique(_e4m3_values()[np.isfinite(_e4m3_values())])
    steps = torch.from_numpy(steps).cuda()
    even = torch.arange(len(steps), device="cuda") % 2 == (len(steps) // 2) % 2  # zero's code is even
    middles = (steps[1:] + steps[:-1]) / 2

    def nearest(y):
        lo = torch.searchsorted(middles, y.contiguous())                         # ties come out low
        tie = (lo < len(middles)) & (middles[lo.clamp(max=len(middles) - 1)] == y)
        return steps[torch.where(tie & ~even[lo], lo + 1, lo)]

    for x, pages, scales in ((st["k"], st["kp"], st["ks"]), (st["v"], st["vp"], st["vs"])):
        held, sc = as64(pages), scales.double()
        for b in range(c["B"]):
            if not new[b]:
                continue
            end = lens[b] + new[b]
            for j in sorted({lens[b] // block} | {min(end - 1, lens[b] // block * block + block) // block}):
                # the block that may hold old rows by itself, then every fresh one at once
                lo = max(lens[b], j * block)
                fresh = j * block >= lens[b]
                hi = end if fresh else min(end, (j + 1) * block)
                cnt = _ceil(hi - j * block, block)
                t = torch.arange(lo, hi, device="cuda")
                rows = torch.zeros((cnt * block, c["Hkv"], D), dtype=torch.float64, device="cuda")
                rows[t - j * block] = x[b, t - lens[b]].double()
                a = rows.view(cnt, block, c["Hkv"], D).abs().amax((1, 3))
                e = torch.ceil(torch.log2((a / qmax).clamp(min=2.0 ** -1000))).clamp(min=-100)
                e = torch.where(a > qmax * torch.exp2(e), e + 1, torch.where((a <= qmax * torch.exp2(e - 1)) & (e > -100), e - 1, e))
                s = torch.exp2(e)
                jj = torch.arange(j, j + cnt, device="cuda")
                pg = torch.from_numpy(table[b].astype(np.int64)).cuda()[jj * block // page]
                sub = jj * block % page // block
                if not fresh:
                    s = torch.maximum(s, sc[pg, sub])
                    t0 = torch.arange(j * block, lens[b], device="cuda")
                    held[pg[0], t0 % page] = nearest(held[pg[0], t0 % page] * (sc[pg, sub] / s)[0][None, :, None])
                sc[pg, sub] = s
                held[pg[(t - j * block) // block], t % page] = nearest(x[b, t - lens[b]].double() / s[(t - j * block) // block][:, :, None])
        out += [held, sc]
    return out[0], out[2], out[1], out[3]
