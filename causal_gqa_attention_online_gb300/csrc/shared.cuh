// shared.cuh -- attention of a batch whose sequences begin alike: how its work is cut
// into equal shares, for the kernel that computes partial results, the one that joins
// them, and tests on the host.
//
// Entities are the groups (their shared keys, for the rows of all members together),
// then the sequences (the keys that are theirs alone).  An entity has a job for each KV
// head and each block of at most two tiles of query tokens; a job walks
// `nt` tiles of 128 keys.  Jobs lie one behind the other on an axis of cost, and CTA c
// of n takes the part [c * W / n, (c + 1) * W / n) of it: whole jobs, and pieces of the
// first and the last.  A piece leaves, for each of its rows, an unnormalised output
// with its maximum and sum; the join adds up the pieces of both of a row's jobs.
#pragma once

#include "common.cuh"

namespace attn {

// Costs, in units of about 100 cycles of an SM: of a tile of keys for one tile of rows (64
// or 128 columns of K and V: the latter wait for memory) and for two, and what a job costs
// besides, the most of it for the partials of two tiles of rows on their way out (a fit of
// the CTAs' clocks in one call, 2 x 12 sequences of 130 tokens: 3200 cycles a tile, 16000 a
// piece.  It takes 277 us with 20 and 36 for a job's start and its tiles, 225 with 110 and
// 36, 210 with 190 and 33; no other call was fitted.)
constexpr int kCostTile64 = 22, kCostTile128 = 28, kCostTwo = 33;
constexpr int kCostStart = 20, kCostStartTwo = 190;

struct SharedArgs {
    AttnParams p;
    const int32_t *cu_groups;    // [N + 1] sequences
    const int32_t *shared_lens;  // [N]
    int N;
    int tile_tokens;   // query tokens of a tile of rows: 128 / G
    int tile_align;    // keys: tiles of a sequence's own keys start on multiples of it
    int ctas;
    int entities;      // N + B, or N where another kernel takes the sequences' own keys
    int own_splits;    // that kernel's parts of a sequence's own keys, or 0
    int cost_one;      // of a tile of keys for one tile of rows
    float c_scale;     // |scale| * log2(e)  (> 0)
    uint32_t idesc_s, idesc_o;
    // workspace
    float *part_o[2];  // shared keys, own keys: [rows / 32][Dv / 4][32][4]; of own_splits
                       // [part][B * Q * Hq][Dv]
    float2 *part_ml[2];  // maximum (log2 units), sum
    int4 *info;        // [B] of each sequence: its group's first, how many, shared keys
    int2 *span[2];     // [kind][B * Q * Hkv] first and last CTA of the job that begins there
};

struct SharedEntity {
    int kind;      // 0 a group's shared keys, 1 a sequence's own
    int b0, s;     // first sequence, how many
    int lo, end;   // keys [lo, end)
    int Qb;        // a sequence's query tokens
    int kv_start;  // first key of tile 0
    int nt;        // tiles of a job (the most, of a sequence's blocks)
    int blocks;    // of query tokens
    bool two[2];   // two tiles of rows: a block but the last, the last
    int w[2];      // cost of a tile in either
    int cb;        // cost of a block but the last
    int jobs;      // KV heads, `blocks` jobs each
    long long cj;  // cost of a head's
};

// The lengths that the entities depend on: the caller's arrays, or copies of them.
struct SharedLens {
    const int32_t *cu, *shared, *k, *q;  // q: null for Q of each
};
__host__ __device__ __forceinline__ SharedLens shared_lens_of(const SharedArgs &a) {
    return {a.cu_groups, a.shared_lens, a.p.seqlens_k, a.p.seqlens_q};
}

// Group n's sequences [g0, g0 + s).
__host__ __device__ __forceinline__ void shared_group(const SharedArgs &a, const SharedLens &z, int n, int &g0,
                                                      int &s) {
    g0 = clamp_len(z.cu[n], a.p.B);
    s = clamp_len(z.cu[n + 1], a.p.B) - g0;
    if (s < 0) s = 0;
}

// The keys that the members of a group attend to together: those of the first member,
// whose table they are read through.
__host__ __device__ __forceinline__ int shared_keys(const SharedArgs &a, const SharedLens &z, int n, int g0, int s) {
    if (s < 1) return 0;
    const int len = clamp_len(z.k[g0], a.p.K);
    return clamp_len(z.shared[n], len);
}

// The group of sequence b, or -1.
__host__ __device__ __forceinline__ int shared_group_of(const SharedArgs &a, const SharedLens &z, int b) {
    int lo = 0, hi = a.N;  // the last group that begins at or before b
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (z.cu[mid] <= b) lo = mid + 1;
        else hi = mid;
    }
    if (lo == 0) return -1;
    return b < z.cu[lo] ? lo - 1 : -1;
}

__host__ __device__ __forceinline__ int shared_start(bool two) { return two ? kCostStartTwo : kCostStart; }

// (tokens: of all blocks together)
__host__ __device__ __forceinline__ void shared_cost(const SharedArgs &a, SharedEntity &e, int tokens) {
    const int last = tokens - (e.blocks - 1) * 2 * a.tile_tokens;
    e.two[0] = true;
    e.two[1] = last > a.tile_tokens;
    for (int i = 0; i < 2; ++i) e.w[i] = e.two[i] ? kCostTwo : a.cost_one;
    if (e.nt == 0) {  // nothing to do: a little cost, so that no CTA passes over many
        e.jobs = e.blocks = 1;
        e.cj = e.cb = 1;
        return;
    }
    e.jobs = a.p.Hkv;
    e.cb = shared_start(true) + e.w[0] * e.nt;
    e.cj = (e.blocks - 1) * (long long)e.cb + shared_start(e.two[1]) + e.w[1] * e.nt;
}

// Entity e of N + B; n: the group of a sequence.
__host__ __device__ __forceinline__ SharedEntity shared_entity(const SharedArgs &a, const SharedLens &z, int e, int n) {
    const AttnParams &p = a.p;
    SharedEntity x;
    if (e < a.N) {
        x.kind = 0;
        x.Qb = 0;
        shared_group(a, z, e, x.b0, x.s);
        x.lo = 0;
        x.end = shared_keys(a, z, e, x.b0, x.s);
        x.kv_start = 0;
        x.nt = (x.end + 127) >> 7;
        const int tokens = x.s * p.Q;
        x.blocks = (tokens + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
        shared_cost(a, x, tokens);
        return x;
    }
    x.kind = 1;
    x.b0 = e - a.N;
    x.s = 1;
    x.lo = 0;
    if (n >= 0) {
        int g0, s;
        shared_group(a, z, n, g0, s);
        x.lo = shared_keys(a, z, n, g0, s);
    }
    x.end = clamp_len(z.k[x.b0], p.K);
    x.Qb = z.q ? clamp_len(z.q[x.b0], p.Q) : p.Q;
    x.kv_start = x.lo & ~(a.tile_align - 1);
    x.nt = x.end > x.lo && x.Qb > 0 ? (x.end - x.kv_start + 127) >> 7 : 0;
    // (blocks of padded tokens alone have no keys)
    const int two = 2 * a.tile_tokens;
    x.blocks = x.Qb > two ? (x.Qb + two - 1) / two : 1;
    shared_cost(a, x, p.Q < x.blocks * two ? p.Q : x.blocks * two);
    return x;
}

struct SharedJob {
    int kvh, tok0, ntok;  // first query token (of all B * Q), how many
    int nt, end;          // tiles of this block, end of the keys that its rows use
    long long at;         // its first (token, KV head) among those of the entities of this kind
};

// Block `block` of KV head kvh.
__host__ __device__ __forceinline__ SharedJob shared_job(const SharedArgs &a, const SharedEntity &x, int kvh,
                                                         int block) {
    const AttnParams &p = a.p;
    SharedJob k;
    k.kvh = kvh;
    const int first = block * 2 * a.tile_tokens, tokens = x.s * p.Q;
    k.tok0 = x.b0 * p.Q + first;
    k.ntok = tokens - first < 2 * a.tile_tokens ? tokens - first : 2 * a.tile_tokens;
    k.nt = x.nt;
    k.end = x.end;
    if (x.kind == 1) {  // the last real token of the block bounds its keys
        const int last = (first + k.ntok < x.Qb ? first + k.ntok : x.Qb) - 1;
        k.end = last < first ? 0 : x.end - x.Qb + last + 1;
        k.nt = k.end > x.lo ? (k.end - x.kv_start + 127) >> 7 : 0;
    }
    k.at = (long long)x.b0 * p.Q * p.Hkv + (long long)k.kvh * tokens + first;
    return k;
}

// Tiles of a job (the first at cost js) before cost x.
__host__ __device__ __forceinline__ int shared_cut(long long x, long long js, int w, int nt) {
    const long long d = x - js;
    if (d <= 0) return 0;
    if (d >= (long long)w * nt) return nt;
    return (int)((uint32_t)d / (uint32_t)w);
}

// CTAs that get a share: each share is at least a tile, so that every CTA between a
// job's first piece and its last has one.
__host__ __device__ __forceinline__ int shared_ctas(long long W, int ctas) {
    const long long n = W / kCostTwo;
    return n < 1 ? 1 : n < ctas ? (int)n : ctas;
}
// Where CTA c's share begins, of n (W from the last one's end on).
__host__ __device__ __forceinline__ long long shared_bound(long long W, int c, int n) {
    if (c >= n) return W;
    if (W < (1LL << 22) && n < 1024) return (uint32_t)W * (uint32_t)c / (uint32_t)n;
    return W * c / n;
}

// A piece's rows in the partials: pieces that follow one another on the axis advance
// the job, the CTA or both, so none of them overlap (at most 256 rows a piece, and
// twice a job's rows where tiles alternate between two chains).
__host__ __device__ __forceinline__ long long shared_base(long long at, int G, int c) {
    return 2 * at * G + 256LL * c;
}
__host__ __device__ __forceinline__ long long shared_rows(const AttnParams &p, int ctas) {
    return 2LL * p.B * p.Q * p.Hq + 256LL * ctas;
}

// Where a share begins: the entity at its first cost, where that one begins, its group
// (-1 for none) and the group's members.
struct SharedBegin {
    long long es;
    int e, n, g0, g1;
    SharedEntity x;
};
__host__ __device__ __forceinline__ SharedBegin shared_begin(const SharedArgs &a, const SharedLens &z, int e, int n,
                                                             long long es) {
    SharedBegin s;
    s.es = es;
    s.e = e;
    s.n = n;
    s.g0 = s.g1 = 0;
    if (e >= a.N) {
        s.g0 = e - a.N;
        s.g1 = s.g0 + 1;
        if (n >= 0) {
            int m;
            shared_group(a, z, n, s.g0, m);
            s.g1 = s.g0 + m;
        }
    }
    s.x = shared_entity(a, z, e, n);
    return s;
}

// The pieces of a CTA's share, one after the other (every lane of a warp alike).
struct SharedWalker {
    const SharedArgs &a;
    long long x0, x1;  // share
    int kvh, block;    // job of the entity
    long long js;      // where it begins
    bool done;
    SharedBegin s;     // the entity

    // (from == to, or an entity past the last: an empty share)
    __host__ __device__ __forceinline__ SharedWalker(const SharedArgs &args, long long from, long long to,
                                                     const SharedBegin &begin)
        : a(args), x0(from), x1(to), kvh(0), block(0), js(begin.es),
          done(from >= to || begin.e >= args.entities), s(begin) {
        if (done) return;
        const long long d = x0 - s.es;
        const bool small = ((d | s.x.cj) >> 31) == 0;
        kvh = small ? (int)((uint32_t)d / (uint32_t)s.x.cj) : (int)(d / s.x.cj);
        const long long in = d - kvh * s.x.cj;
        const int at = (in >> 31) == 0 ? (int)((uint32_t)in / (uint32_t)s.x.cb) : (int)(in / s.x.cb);
        block = at < s.x.blocks ? at : s.x.blocks - 1;
        js += kvh * s.x.cj + (long long)block * s.x.cb;
    }
    __host__ __device__ __forceinline__ void load() {
        if (s.e >= a.entities || s.es >= x1) {
            done = true;
            return;
        }
        const SharedLens z = shared_lens_of(a);
        const int b = s.e - a.N;
        if (b >= 0 && (b < s.g0 || b >= s.g1)) s = shared_begin(a, z, s.e, shared_group_of(a, z, b), s.es);
        else s.x = shared_entity(a, z, s.e, s.n);
    }
    // the next piece with tiles [t0, t1) of job k; false: no more
    __host__ __device__ __forceinline__ bool next(SharedJob &k, int &t0, int &t1) {
        while (!done) {
            if (kvh >= s.x.jobs) {
                s.es += s.x.jobs * s.x.cj;
                js = s.es;
                kvh = block = 0;
                ++s.e;
                load();
                continue;
            }
            if (js >= x1) break;
            t0 = t1 = 0;
            const bool last = block == s.x.blocks - 1;
            if (s.x.nt > 0) {
                k = shared_job(a, s.x, kvh, block);
                const int w = last ? s.x.w[1] : s.x.w[0];
                const long long first = js + shared_start(last ? s.x.two[1] : s.x.two[0]);
                t0 = shared_cut(x0, first, w, k.nt);
                t1 = shared_cut(x1, first, w, k.nt);
            }
            if (last) {
                js = s.es + ++kvh * s.x.cj;
                block = 0;
            } else {
                js += s.x.cb;
                ++block;
            }
            if (t1 > t0) return true;
        }
        done = true;
        return false;
    }
};

// Part s of the keys [lo, end) that a sequence has alone, in whole tiles of 64 and at
// least kOwnKeys of them; empty where beg >= fin.
constexpr int kOwnKeys = 256;
__host__ __device__ __forceinline__ int own_part(int lo, int end, int splits) {
    const uint32_t keys = (uint32_t)(end - (lo & ~63));
    const uint32_t per = (keys / (uint32_t)splits + (keys % (uint32_t)splits != 0) + 63u) & ~63u;
    return per < (uint32_t)kOwnKeys ? kOwnKeys : (int)per;
}
// How many of them have keys (end > lo).
__host__ __device__ __forceinline__ int own_parts(int lo, int end, int splits) {
    const uint32_t keys = (uint32_t)(end - (lo & ~63)), per = (uint32_t)own_part(lo, end, splits);
    return (int)((keys - 1) / per) + 1;
}
__host__ __device__ __forceinline__ void own_split(int lo, int end, int splits, int s, int &beg, int &fin) {
    beg = fin = 0;
    if (end <= lo) return;
    const long long per = own_part(lo, end, splits), b0 = (lo & ~63) + s * per;
    if (b0 >= end) return;
    beg = s == 0 ? lo : (int)b0;
    fin = b0 + per < end ? (int)(b0 + per) : end;
}

// A row's job of either kind, from what the sequence's info says.
struct SharedRow {
    long long at;    // the job's first (token, KV head)
    int ntok, lr;    // its tokens; the row's place among its rows
    bool some;       // whether the job has a tile
};
__host__ __device__ __forceinline__ SharedRow shared_row(const SharedArgs &a, int kind, int g0, int s, int keys,
                                                         int b, int i, int h, int len, int Qb) {
    const AttnParams &p = a.p;
    const int kvh = h / p.G, two = 2 * a.tile_tokens;
    const int b0 = kind == 0 ? g0 : b, tokens = kind == 0 ? s * p.Q : p.Q, off = (b - b0) * p.Q + i;
    const int first = off / two * two;
    SharedRow r;
    r.ntok = tokens - first < two ? tokens - first : two;
    r.lr = (off - first) * p.G + (h - kvh * p.G);
    r.at = (long long)b0 * p.Q * p.Hkv + (long long)kvh * tokens + first;
    r.some = keys > 0;
    if (kind == 1) {  // (as shared_job)
        const int last = (first + r.ntok < Qb ? first + r.ntok : Qb) - 1;
        r.some = last >= first && len - Qb + last + 1 > keys;
    }
    return r;
}

}  // namespace attn
