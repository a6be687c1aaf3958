// shared.cuh -- attention of a batch whose sequences begin alike: how its work is cut
// into equal shares, for the kernel that computes partial results, the one that joins
// them, and tests on the host.
//
// Entities are the groups (their shared keys, for the rows of all members together),
// then the sequences (the keys that are theirs alone).  An entity has `jobs` jobs of
// equal cost: KV heads times blocks of at most two tiles of query tokens; a job walks
// `nt` tiles of 128 keys.  Jobs lie one behind the other on an axis of cost, and CTA c
// of n takes the part [c * W / n, (c + 1) * W / n) of it: whole jobs, and pieces of the
// first and the last.  A piece leaves, for each of its rows, an unnormalised output
// with its maximum and sum; the join adds up the pieces of both of a row's jobs.
#pragma once

#include "common.cuh"

namespace attn {

// Cost of a piece's start, and of a tile of keys for one and for two tiles of rows, in
// units of about 0.4 us on one SM (measured: see kernel_shared_tc.cu).
constexpr int kCostStart = 2, kCostTile = 3, kCostTwo = 4;

struct SharedArgs {
    AttnParams p;
    const int32_t *cu_groups;    // [N + 1] sequences
    const int32_t *shared_lens;  // [N]
    int N;
    int tile_tokens;   // query tokens of a tile of rows: 128 / G
    int own_blocks;    // blocks of query tokens of a sequence
    int tile_align;    // keys: tiles of a sequence's own keys start on multiples of it
    int ctas;
    float c_scale;     // |scale| * log2(e)  (> 0)
    uint32_t idesc_s, idesc_o;
    // workspace
    float *part_o[2];  // [kind][rows][Dv]: shared keys, own keys
    float2 *part_ml[2];  // maximum (log2 units), sum
    long long *start;  // [N + B + 1] first cost of each entity; the last: W
    int32_t *group;    // [B] group of each sequence, -1 for none
};

struct SharedEntity {
    int kind;      // 0 a group's shared keys, 1 a sequence's own
    int b0, s;     // first sequence, how many
    int lo, end;   // keys [lo, end)
    int kv_start;  // first key of tile 0
    int nt;        // tiles of a job (the most, of a sequence's blocks)
    int blocks;    // of query tokens
    int w;         // cost of a tile
    int jobs;      // KV heads x blocks
    int cj;        // cost of a job
};

__host__ __device__ __forceinline__ int shared_at(const int32_t *p, long long i) {
#ifdef __CUDA_ARCH__
    return __ldg(p + i);
#else
    return p[i];
#endif
}

// Group n's sequences [g0, g0 + s).
__host__ __device__ __forceinline__ void shared_group(const SharedArgs &a, int n, int &g0, int &s) {
    g0 = clamp_len(shared_at(a.cu_groups, n), a.p.B);
    s = clamp_len(shared_at(a.cu_groups, n + 1), a.p.B) - g0;
    if (s < 0) s = 0;
}

// The keys that the members of a group attend to together: those of the first member,
// whose table they are read through; none for less than two members.
__host__ __device__ __forceinline__ int shared_keys(const SharedArgs &a, int n, int g0, int s) {
    if (s < 2) return 0;
    const int len = clamp_len(shared_at(a.p.seqlens_k, g0), a.p.K);
    return clamp_len(shared_at(a.shared_lens, n), len);
}

// The group of sequence b, or -1.
__host__ __device__ __forceinline__ int shared_group_of(const SharedArgs &a, int b) {
    int lo = 0, hi = a.N;  // the last group that begins at or before b
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (shared_at(a.cu_groups, mid) <= b) lo = mid + 1;
        else hi = mid;
    }
    if (lo == 0) return -1;
    return b < shared_at(a.cu_groups, lo) ? lo - 1 : -1;
}

__host__ __device__ __forceinline__ void shared_cost(const SharedArgs &a, SharedEntity &e, bool two) {
    e.w = two ? kCostTwo : kCostTile;
    if (e.nt == 0) {  // nothing to do: a little cost, so that no CTA passes over many
        e.jobs = 1;
        e.cj = 1;
        return;
    }
    e.jobs = a.p.Hkv * e.blocks;
    e.cj = kCostStart + e.w * e.nt;
}

// Entity e of N + B; n: the group of a sequence.
__host__ __device__ __forceinline__ SharedEntity shared_entity(const SharedArgs &a, int e, int n) {
    const AttnParams &p = a.p;
    SharedEntity x;
    if (e < a.N) {
        x.kind = 0;
        shared_group(a, e, x.b0, x.s);
        x.lo = 0;
        x.end = shared_keys(a, e, x.b0, x.s);
        x.kv_start = 0;
        x.nt = (x.end + 127) >> 7;
        const int tokens = x.s * p.Q;
        x.blocks = (tokens + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
        shared_cost(a, x, tokens > a.tile_tokens);
        return x;
    }
    x.kind = 1;
    x.b0 = e - a.N;
    x.s = 1;
    x.lo = 0;
    if (n >= 0) {
        int g0, s;
        shared_group(a, n, g0, s);
        x.lo = shared_keys(a, n, g0, s);
    }
    x.end = clamp_len(shared_at(p.seqlens_k, x.b0), p.K);
    const int Qb = p.seqlens_q ? clamp_len(shared_at(p.seqlens_q, x.b0), p.Q) : p.Q;
    x.kv_start = x.lo & ~(a.tile_align - 1);
    x.nt = x.end > x.lo && Qb > 0 ? (x.end - x.kv_start + 127) >> 7 : 0;
    x.blocks = a.own_blocks;
    shared_cost(a, x, p.Q > a.tile_tokens);
    return x;
}

struct SharedJob {
    int kvh, tok0, ntok;  // first query token (of all B * Q), how many
    int nt, end;          // tiles of this block, end of the keys that its rows use
    long long row0;       // first row among the rows of the entities of this kind
};

__host__ __device__ __forceinline__ SharedJob shared_job(const SharedArgs &a, const SharedEntity &x, int j) {
    const AttnParams &p = a.p;
    SharedJob k;
    k.kvh = j / x.blocks;
    const int first = (j - k.kvh * x.blocks) * 2 * a.tile_tokens, tokens = x.s * p.Q;
    k.tok0 = x.b0 * p.Q + first;
    k.ntok = tokens - first < 2 * a.tile_tokens ? tokens - first : 2 * a.tile_tokens;
    k.nt = x.nt;
    k.end = x.end;
    if (x.kind == 1) {  // the last real token of the block bounds its keys
        const int Qb = p.seqlens_q ? clamp_len(shared_at(p.seqlens_q, x.b0), p.Q) : p.Q;
        const int last = (first + k.ntok < Qb ? first + k.ntok : Qb) - 1;
        k.end = last < first ? 0 : x.end - Qb + last + 1;
        k.nt = k.end > x.lo ? (k.end - x.kv_start + 127) >> 7 : 0;
    }
    k.row0 = (long long)x.b0 * p.Q * p.Hq + ((long long)k.kvh * tokens + first) * p.G;
    return k;
}

// Tiles of a job (its start at cost js) before cost x.
__host__ __device__ __forceinline__ int shared_cut(long long x, long long js, int w, int nt) {
    const long long d = x - js - kCostStart;
    if (d <= 0) return 0;
    const long long t = d / w;
    return t < nt ? (int)t : nt;
}

__host__ __device__ __forceinline__ long long shared_bound(long long W, int c, int n) {
    return W * c / n;
}

// A piece's rows in the partials: pieces that follow one another on the axis advance
// the job, the CTA or both, so none of them overlap (at most 256 rows a piece, and
// twice a job's rows where tiles alternate between two chains).
__host__ __device__ __forceinline__ long long shared_base(long long row0, int c) {
    return 2 * row0 + 256LL * c;
}
__host__ __device__ __forceinline__ long long shared_rows(const AttnParams &p, int ctas) {
    return 2LL * p.B * p.Q * p.Hq + 256LL * ctas;
}

// The pieces of a CTA's share, one after the other (every lane of a warp alike).
struct SharedWalker {
    const SharedArgs &a;
    long long x0, x1, es;  // share, first cost of the entity
    int e, j;              // entity, job
    int n;                 // group of a sequence, -1 for none
    SharedEntity x;
    bool done;

    // (es0: the first cost of entity e0, where the share begins; x0 < x1)
    __host__ __device__ __forceinline__ SharedWalker(const SharedArgs &args, long long from, long long to,
                                                     long long es0, int e0)
        : a(args), x0(from), x1(to), es(es0), e(e0), j(0), n(-1), x(), done(from >= to) {
        if (done) return;
        load();
        if (!done) j = (int)((x0 - es) / x.cj);
    }
    __host__ __device__ __forceinline__ void load() {
        if (e >= a.N + a.p.B || es >= x1) {
            done = true;
            return;
        }
        n = e >= a.N ? shared_group_of(a, e - a.N) : -1;
        x = shared_entity(a, e, n);
    }
    // the next piece with tiles [t0, t1) of job k; false: no more
    __host__ __device__ __forceinline__ bool next(SharedJob &k, int &t0, int &t1) {
        while (!done) {
            const long long js = es + (long long)j * x.cj;
            if (j >= x.jobs) {
                es += (long long)x.jobs * x.cj;
                j = 0;
                ++e;
                load();
                continue;
            }
            if (js >= x1) break;
            if (x.nt > 0) {
                k = shared_job(a, x, j);
                t0 = shared_cut(x0, js, x.w, k.nt);
                t1 = shared_cut(x1, js, x.w, k.nt);
            } else {
                t0 = t1 = 0;
            }
            ++j;
            if (t1 > t0) return true;
        }
        done = true;
        return false;
    }
};

// The partials of a row: of its entity's job, from CTAs [c0, c1], two chains each.
struct SharedRow {
    SharedEntity x;
    SharedJob k;
    long long js;  // cost where the job begins
    int lr;        // row of the job
    int c0, c1;
    bool two;
};
__host__ __device__ __forceinline__ SharedRow shared_row(const SharedArgs &a, int e, int n, long long es,
                                                         long long W, int token, int h) {
    SharedRow r;
    r.x = shared_entity(a, e, n);
    if (r.x.nt == 0) return r;
    const int kvh = h / a.p.G, off = token - r.x.b0 * a.p.Q, blk = off / (2 * a.tile_tokens);
    const int j = kvh * r.x.blocks + blk;
    r.k = shared_job(a, r.x, j);
    r.two = r.k.ntok > a.tile_tokens;
    r.lr = (off - blk * 2 * a.tile_tokens) * a.p.G + (h - kvh * a.p.G);
    r.js = es + (long long)j * r.x.cj;
    // the first CTA whose share ends behind js, the last one whose share begins before
    // the job's end (bounds round down)
    r.c0 = (int)(((r.js + 1) * a.ctas + W - 1) / W) - 1;
    r.c1 = (int)(((r.js + r.x.cj) * a.ctas + W - 1) / W) - 1;
    return r;
}
// Where CTA c's chain left the row's partial, or -1.
__host__ __device__ __forceinline__ long long shared_partial(const SharedArgs &a, const SharedRow &r,
                                                             long long W, int c, int chain) {
    const int t0 = shared_cut(shared_bound(W, c, a.ctas), r.js, r.x.w, r.k.nt);
    const int t1 = shared_cut(shared_bound(W, c + 1, a.ctas), r.js, r.x.w, r.k.nt);
    if (r.two ? (t1 <= t0 || chain > 0) : t1 - t0 <= chain) return -1;
    return shared_base(r.k.row0, c) + (r.two ? 0 : chain * r.k.ntok * a.p.G) + r.lr;
}

}  // namespace attn
