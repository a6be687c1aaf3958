// kernel_q8_decode.cu -- split-KV tensor-core decode over the 8-bit paged cache
// (bf16 / fp16 queries, widths multiples of 16 up to 256, pages of at least 8 rows,
// the rows of a KV group in row groups of 16 or fewer).
//
// The products are those of the 16-bit decode, keys (or value columns) on M and
// the rows of the KV group on N,
//
//     S^T[key, row] = code_K[key, :] . Q[row, :],   x = S^T * ks[key]
//     p = 2^(x f[row] - m + 14),   O^T[dv, row] += code_V^T[dv, key] . (p * vs[key] / u)^T
//
// with m16n8k16 f16 products, fp32 accumulation.  Codes become f16 pairs in
// registers, exactly (q8.cuh), and the scales multiply scores and probabilities
// in fp32, so no key or value is rounded:
//
// * Q rows are brought to [2^14, 2^15) by a power of two (in f[row], with the
//   softmax scale; its sign goes to Q), so that bf16's 8 bits stay exact down to
//   2^-29 of the row's largest element.
// * Probabilities are in (0, 2^14], times vs / u in f16, where u is the largest value
//   scale a warp has seen (2^-112 at the least: its reciprocal times 2^14 is an fp32
//   number): 11 bits down to 2^-28 of p = 2^14 and vs = u, steps of 2^-38 below.  O is
//   rescaled when m or u grow.  The 2^14 cancels against the row sum, u comes back in the
//   final normalisation.
// * That serves every row while the scales seen lie within a factor of 64 (kSpread): a
//   row's largest weight p * vs is then 2^8 or more, whichever keys it attends to.  A warp
//   that meets a wider spread does the rest of the sequence with a unit for each row,
//   which brings the step's largest weight of the row to [2^13, 2^14) (own_steps): a large
//   scale on a key that a row does not attend to, or that hardly counts, costs it nothing.
//   So does one that meets scores past 2^22 (kMaxScore), whose product with f is rounded
//   by too much for x f - m f: there the difference comes first, and a power of two of f
//   goes to the key scales, so that x is an fp32 number wherever the score is.
// * Which bytes pair up is chosen so that no byte is moved across lanes: the two
//   pairs of a 32-bit word are the two halves of a k16 step (K: Q's columns are
//   permuted to match) or the rows dv = 2g and 2g + 1 (V: a transposed ldmatrix of
//   byte pairs gives two keys' pairs in one word).
//
// Bound: HBM, one byte an element -- at 8 flops a byte, twice the 16-bit
// decode's arithmetic per byte, the conversions (4 to 5 instructions for four
// codes) have to stay out of the way.  A CTA is four consumer warps of 32 keys
// each and a producer warp: it looks pages up 32 boxes at a time and a group ahead, issues one TMA
// box per page piece (up to 64 rows) and the block scales as 4-byte cp.async,
// all completing on the stage's mbarrier; consumers free a stage with one
// arrival a warp, so no warp waits for another within a tile.  Tiles that every
// row attends to whole take a step without tests; in the others masked scores
// are -inf and V's words are cleared where a key takes no part for any row (a code there
// may be anything); e4m3's NaN codes on the others' keys count as 0, and find_nans finds
// the elements of the rows that attend to them.
//
// Work: the 128-key tiles of all sequences, in order, are cut into equal shares
// whatever the lengths, and a CTA takes one share for one KV head (and row group) -- as many
// shares as give every resident CTA one, so that the heads of a page are read at
// the same time (with the heads one after the other, the 256-byte reads of
// 128-byte head rows brought in 719 MB for 547).  The producer runs from one
// sequence into the next without draining the ring.  A sequence that lies in one
// share is written out by its CTA; shares that begin or end inside one leave a
// partial each (at most two a CTA, so the workspace does not grow with the
// keys), and the merge kernel, a block for each place where a share begins
// inside a sequence, head and row, joins those.  Small problems (at most four
// tiles a CTA with every CTA resident) give each (sequence, head) a cluster of up
// to eight CTAs, which split its tiles and join their states through distributed
// shared memory: one launch and no workspace.
//
// Measured: 64 ragged sequences up to 8192 keys (Hq 32, Hkv 8, D 128) in 102 us
// with int8 codes (5.36 TB/s, 0.79 of a plain copy) and 95 with e4m3; in a graph 98, of
// which 89 remain without the arithmetic, ten of them launch and first tile.  Two
// sequences of 100003 keys, four rows each of 16 heads over 4, D 64, e4m3: 37 us (2.45
// TB/s); in a graph 35, of which 26 remain without the arithmetic: launch, first tile,
// the end of the shares and the merge.  One sequence of 700 keys: 8.4 us in a graph.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <climits>

#include <cooperative_groups.h>
#include <cstring>

#include "common.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "q8.cuh"
#include "sm100_ptx.cuh"
#include "tc_softmax.cuh"

namespace attn {
namespace {

constexpr int kTile = 128;  // keys a tile: 4 warps x 32
constexpr int kThreads = 160;
constexpr float kPOff = 14.f;  // p is scaled by 2^14
constexpr float kLeastUnit = 1.92592994e-34f;  // 2^-112
// Value scales under one unit lie within this factor.  64 sequences of up to 8192 keys, D
// 128: 98 us in a graph, and 135 with scales spread over 2^24, where every row has its unit.
constexpr float kSpread = 64.f;
constexpr float kMaxScore = 4194304.f;  // 2^22: x f - m f is off by 2^-2 at most, for all keys alike
constexpr int kMaxRows = 1024;  // rows of a KV group at most

struct Q8Args {
    AttnParams p;
    Q8Cache c;
    int box_rows;  // rows of a TMA box: min(page_size, 64)
    int box_shift;
    bool bf16;
    int cluster;   // CTAs of a (sequence, head), or 0: shares
    int shares;    // shares at most (no more than there are tiles are used)
    int groups;    // row groups of a KV head, of R rows each (the last may have fewer)
    // workspace: for each share {sequence, its first share, its last} where the
    // merge of a sequence is found (its second share; {-1} elsewhere), partials
    // [CTA][2][R] of normalised rows and log2 sums (CTA: share, head, row group)
    int4 *seam;
    float *part_o, *part_lse;
};

// Resident CTAs an SM: two, one where a row is wider than 128; three for 64-wide
// heads with up to eight rows (125 registers), whose tiles are half as large: 32
// sequences of up to 8192 keys and eight heads 43.3 us for 45.3, 64 of 4096 41.3 for
// 43.8 (16 rows would spill and are slower: 24.7 for 22.7).
constexpr int resident(int DP, int NT) { return DP > 128 ? 1 : DP == 64 && NT == 1 ? 3 : 2; }

template <int DP, int NT> struct Ring {
    static constexpr int HALF = DP > 128 ? 128 : DP;  // bytes of a box row
    static constexpr int TILE = kTile * DP;
    static constexpr int STAGE = 2 * TILE + 2 * kTile * 4;
    static constexpr int NS = DP > 64 ? 3 : NT == 1 ? 4 : 5;
    // the warps' O are merged MC columns at a time through two warps' buffers
    static constexpr int R = NT * 8;
    static constexpr int MC = DP == 64 ? 64 : DP / NT;
    static constexpr int PITCH = MC + 4;
    static constexpr int MERGE = NS * STAGE;
    static constexpr int STATS = MERGE + 2 * R * PITCH * 4;  // m, l, u [4][R]
    static constexpr int BARS = STATS + 3 * 4 * R * 4;
    static constexpr int SHARE = BARS + 16 * NS;  // {left, sequence, tile}, abort flag
    static constexpr int SMEM = SHARE + 32;
    // (an SM has 228 KB, a CTA takes 1 KB more than its own)
    static_assert(SMEM <= (228 / resident(DP, NT) - 1) * 1024, "resident() CTAs an SM");
};

// Byte offset of 16-byte chunk c of row r: rows of 64 bytes in the 64-byte
// swizzle, of 128 in the 128-byte one, 256 as two 128-byte halves.
template <int DP> __device__ __forceinline__ int chunk_at(int r, int c) {
    if (DP == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// The keys some row of sequence b attends to, [lo, hi), from a multiple of the
// box on, so that a box is one page's; and how many tiles they take.
struct UnitKeys {
    SeqInfo si;
    int klo, kbeg, kend, ntiles;
};
__device__ __forceinline__ UnitKeys unit_of(const Q8Args &a, int b) {
    UnitKeys u;
    u.si = seq_info(a.p, b);
    unit_keys(u.si.Qb, u.si.Kb, a.p.window, a.p.mask, u.klo, u.kend);
    u.kbeg = u.klo & ~(a.box_rows - 1);
    u.ntiles = (int)(((long long)u.kend - u.kbeg + kTile - 1) / kTile);
    return u;
}

// T tiles in n shares, 1 <= n <= T: the first T % n of them have a tile more.  (In
// 32 bits, with one division: 64-bit ones in the prologue cost a CTA 0.3 us each.)
struct Shares {
    uint32_t q, r;
    __host__ __device__ __forceinline__ Shares(uint32_t T, uint32_t n) : q(T / n), r(T - T / n * n) {}
    // the first tile of share i, and the share of tile t
    __host__ __device__ __forceinline__ uint32_t begin(uint32_t i) const { return i * q + (i < r ? i : r); }
    __host__ __device__ __forceinline__ uint32_t of(uint32_t t) const {
        const uint32_t head = r * (q + 1);
        return t < head ? t / (q + 1) : r + (t - head) / q;
    }
};

// Four columns of a joined row: acc / sum, and its LSE from the log2 sums' maximum
// (a row without keys: +0 and -inf; one with a NaN key: NaN).
__device__ __forceinline__ void put_row(const Q8Args &a, int b, int kvh, int row, int c, const float4 &acc,
                                        float sum, float mx) {
    const AttnParams &p = a.p;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long orow = ((long long)b * p.Q + row / p.G) * p.Hq + kvh * p.G + row % p.G;
    uint2 w;
    if (a.bf16) {
        w.x = MmaOp<__nv_bfloat16>::pack(acc.x * inv, acc.y * inv);
        w.y = MmaOp<__nv_bfloat16>::pack(acc.z * inv, acc.w * inv);
    } else {
        w.x = MmaOp<__half>::pack(acc.x * inv, acc.y * inv);
        w.y = MmaOp<__half>::pack(acc.z * inv, acc.w * inv);
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + orow * p.Dv + 4 * c) = w;
    if (c == 0 && p.lse)
        p.lse[orow] = sum != sum ? sum : sum > 0.f ? (mx + __log2f(sum)) * kLn2 : -INFINITY;
}

// The rows of a sequence without keys, by a warp: +0 and -inf.
__device__ __forceinline__ void empty_rows(const Q8Args &a, int b, int kvh, int lane) {
    const AttnParams &p = a.p;
    const int c8 = p.Dv / 8;
    for (int i = lane; i < p.Q * p.G * c8; i += 32) {
        const int row = i / c8, c = i - row * c8;
        const long long orow = ((long long)b * p.Q + row / p.G) * p.Hq + kvh * p.G + row % p.G;
        reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.o) + orow * p.Dv)[c] = make_uint4(0, 0, 0, 0);
        if (c == 0 && p.lse) p.lse[orow] = -INFINITY;
    }
}

// The joint rows of a cluster's CTAs, whose own are at xrow [R][DP] and xlse [R] of
// each: four columns a thread, the (row, column) pairs spread over the CTAs.  (A
// function of its own, so that its registers do not add to the main loop's.)
template <int DP>
__device__ __noinline__ void join_cluster(const Q8Args &a, int b, int kvh, int row0, int rows, int rank, int ntiles,
                                          float *xrow, float *xlse) {
    const AttnParams &p = a.p;
    auto cluster = cooperative_groups::this_cluster();
    const int C = a.cluster, C4 = p.Dv / 4;
    for (int i = rank * kThreads + threadIdx.x; i < rows * C4; i += C * kThreads) {
        const int row = i / C4, c = i - row * C4;
        float lw[8], mx = -INFINITY;
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            lw[r] = -INFINITY;
            v[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            // (a CTA without tiles has no rows)
            if (r < C && (r + 1) * ntiles / C > r * ntiles / C) {
                lw[r] = cluster.map_shared_rank(xlse, r)[row];
                v[r] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(xrow, r) + row * DP + 4 * c);
            }
            mx = fmaxf(mx, lw[r]);
        }
        const float mref = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float w = exp2f(lw[r] - mref);
            sum += w;
            acc.x = fmaf(w, v[r].x, acc.x);
            acc.y = fmaf(w, v[r].y, acc.y);
            acc.z = fmaf(w, v[r].z, acc.z);
            acc.w = fmaf(w, v[r].w, acc.w);
        }
        put_row(a, b, kvh, row0 + row, c, acc, sum, mx);
    }
}

// 2^x as a float, -126 <= x <= 127.
__device__ __forceinline__ float pow2(int x) { return __uint_as_float((uint32_t)(127 + x) << 23); }

// The unit of a row for a step whose largest weight (p at most 1) is w, and the factor
// that brings O, whose elements are o at most, to it: w * 2^14 in [2^13, 2^14), but for
// weights so far below what O may hold that it would pass 2^100.
__device__ __forceinline__ float own_unit(float w, float o, float &unit) {
    const int ew = min(max((int)(__float_as_uint(w) >> 23) - 127, -113), 125);
    const int eo = min(max((int)(__float_as_uint(o) >> 23) - 127, -27), 127);
    const float next = pow2(-1 - ew), f = next / unit, most = pow2(99 - eo);
    if (f <= most) {
        unit = next;
        return f;
    }
    unit *= most;
    return most;
}

// What own_steps keeps for each row: the power of two of f that key scales are
// multiplied by, O's unit, and a bound of O's elements.
template <int NT> struct Own {
    float kf[NT][2], unit[NT][2], bound[NT][2];
};

// What a warp holds of a sequence.  A thread's columns of S^T and O^T are rows 2 tig and
// 2 tig + 1 of each eight.
template <int DP, int NT> struct Rows {
    uint32_t q[DP / 16][NT][2];  // Q^T fragments
    float f[NT][2];              // x to log2 units
    int lo[NT][2], hi[NT][2];    // legal keys
    float m[NT][2], l[NT][2];    // the largest x; the sum of p
    float o[DP / 16][NT][4];
    float u, u_min;              // value scales seen: O's unit, and the least
};

// Which halves of a word of V^T codes (columns 2 g, 2 g + 1 of keys k and k + 1) belong to
// keys that some row attends to.
__device__ __forceinline__ uint32_t key_mask(int k, int klo, int kend) {
    return (k >= klo && k < kend ? 0xffffu : 0u) | (k + 1 >= klo && k + 1 < kend ? 0xffff0000u : 0u);
}

// The sign bits of the bytes that are e4m3's NaN codes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// O's elements whose row attends to a key whose value is NaN there, a bit each (o[mt][nt][j]
// of word mt / 4, bit (mt % 4 * NT + nt) * 4 + j): the product of [code is NaN] and [row
// attends] is not 0.  (For steps that some rows' keys end in and that hold such a code; the
// product with P, where 0 * NaN would reach every row, takes those codes as 0.)
struct NanBits {
    uint32_t w[4];
};
template <int NT> struct Legal {
    int lo[NT][2], hi[NT][2];
};
template <int DP, int NT>
__device__ __noinline__ NanBits find_nans(Legal<NT> w, uint32_t vs, int kw0, int key0, int klo, int kend) {
    using Op = CodeOps<kCodeE4m3>;
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    NanBits bits = {{0, 0, 0, 0}};
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = key0 + g + 8 * i;
            float on[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) on[e] = key >= w.lo[nt][e] && key < w.hi[nt][e] ? 1.f : 0.f;
            pb[i >> 1][nt][i & 1] = movmatrix_trans(MmaOp<__half>::pack(on[0], on[1]));
        }
#pragma unroll
    for (int cc = 0; cc < DP / 16; cc += 2) {
        float n[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) n[h][nt][j] = 0.f;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            uint32_t r[4];
            ldmatrix_x4_trans(r, vs + chunk_at<DP>(kw0 + kt * 16 + (lane & 15), cc + (lane >> 4)));
#pragma unroll
            for (int i = 0; i < 4; ++i)  // 0x38 is 1
                r[i] = (nan_codes(r[i] & key_mask(key0 + kt * 16 + (i & 1) * 8 + 2 * tig, klo, kend)) >> 7) * 0x38u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t f[4];
                Op::even_odd(r[2 * h], f[0], f[1]);
                Op::even_odd(r[2 * h + 1], f[2], f[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) MmaOp<__half>::run(n[h][nt], f, pb[kt][nt][0], pb[kt][nt][1]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n[h][nt][j] > 0.f) bits.w[(cc + h) / 4] |= 1u << (((cc + h) % 4 * NT + nt) * 4 + j);
    }
    return bits;
}

// One step: the warp's 32 keys from key0 on, codes at ks and vs, scales at sc (values'
// kTile behind).  EDGE: some row may not attend to all of them, and some may be outside
// [klo, kend), where no row does.  OWN: rows have units of their own; a step without gives
// up, with nothing changed, where scales spread too far for one or scores are too large.
template <int CODE, int DP, int NT, bool EDGE, bool OWN>
__device__ __forceinline__ bool q8_step(Rows<DP, NT> &w, uint32_t ks, uint32_t vs, const float *sc, int kw0, int key0,
                                        int klo, int kend, Own<NT> &own) {
    using Op = CodeOps<CODE>;
    const int lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    // S^T = K Q^T
    float sacc[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) sacc[mt][nt][j] = 0.f;
#pragma unroll
    for (int kk = 0; kk < DP / 16; kk += 2) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t r[4];
            ldmatrix_x4(r, ks + chunk_at<DP>(kw0 + mt * 16 + (lane & 15), kk + (lane >> 4)));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t f[4];
                Op::k_pairs(r[2 * h], f[0], f[2]);
                Op::k_pairs(r[2 * h + 1], f[1], f[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    MmaOp<__half>::run(sacc[mt][nt], f, w.q[kk + h][nt][0], w.q[kk + h][nt][1]);
            }
        }
    }

    float unew = 1.f, least = 0.f, inv_u = 1.f;
    if (!OWN) {
        // the finite value scales so far, of keys some row attends to
        const int uk = key0 + lane;
        uint32_t ub = __float_as_uint(sc[kTile + lane]) & 0x7fffffffu;
        const bool no = ub >= 0x7f800000u || (EDGE && !(uk >= klo && uk < kend));
        unew = fmaxf(w.u, __uint_as_float(__reduce_max_sync(0xffffffffu, no ? 0u : ub)));
        least = fminf(w.u_min, __uint_as_float(__reduce_min_sync(0xffffffffu, no ? 0x7f800000u : ub)));
        inv_u = 1.f / unew;
    }

    float kscale[4], vw[4];  // keys g, g + 8, g + 16, g + 24
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        kscale[i] = sc[g + 8 * i];
        vw[i] = sc[kTile + g + 8 * i] * inv_u;
    }
    float x[NT][2][4], mx[NT][2], ref[NT][2];
    const bool spread = !OWN && unew > kSpread * least;
    bool grew = OWN || unew > w.u || spread, leave = spread;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[nt][e][i] = sacc[i >> 1][nt][2 * (i & 1) + e] * (OWN ? kscale[i] * own.kf[nt][e] : kscale[i]);
                if (EDGE) {
                    const int key = key0 + g + 8 * i;
                    if (!(key >= w.lo[nt][e] && key < w.hi[nt][e])) x[nt][e][i] = -INFINITY;
                }
            }
            float v = tcfwd::fmax3(x[nt][e][0], x[nt][e][1], fmaxf(x[nt][e][2], x[nt][e][3]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = tcfwd::fmax3(v, __shfl_xor_sync(0xffffffffu, v, 16), w.m[nt][e]);
            mx[nt][e] = v;
            ref[nt][e] = v == -INFINITY ? 0.f : OWN ? v : kPOff - v * w.f[nt][e];
            grew |= v > w.m[nt][e];
            // (-inf: a row that attends to keys here, and every score of it so far is)
            if (!OWN && v == -INFINITY && (!EDGE || max(w.lo[nt][e], key0) < min(w.hi[nt][e], key0 + 32)))
                grew = leave = true;
        }
    float to[NT][2];  // (OWN) what O is multiplied by for its new unit
    if (OWN) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float most = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (x[nt][e][i] != -INFINITY)
                        most = fmaxf(most, fabsf(tcfwd::ex2((x[nt][e][i] - mx[nt][e]) * w.f[nt][e]) * vw[i]));
#pragma unroll
                for (int d = 4; d <= 16; d *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                if (mx[nt][e] > w.m[nt][e])
                    own.bound[nt][e] *= tcfwd::ex2((w.m[nt][e] - mx[nt][e]) * w.f[nt][e]);
                to[nt][e] = own_unit(most, own.bound[nt][e], own.unit[nt][e]);
                // (a step adds 32 weights of 2^15 times codes of 448 at most)
                own.bound[nt][e] = own.bound[nt][e] * to[nt][e] + 0x1p29f;
            }
    }
    if (__any_sync(0xffffffffu, grew)) {
        if (!OWN) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) leave |= fabsf(ref[nt][e]) > kMaxScore;
            if (__any_sync(0xffffffffu, leave)) return false;
        }
        const float ru = unew > w.u ? w.u * inv_u : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // (no key yet: both -inf, and nothing to rescale)
                const float alpha =
                    mx[nt][e] > w.m[nt][e] ? tcfwd::ex2((w.m[nt][e] - mx[nt][e]) * w.f[nt][e]) : 1.f;
                w.m[nt][e] = mx[nt][e];
                w.l[nt][e] *= alpha;
                const float f = alpha * (OWN ? to[nt][e] : ru);
#pragma unroll
                for (int mt = 0; mt < DP / 16; ++mt) {
                    w.o[mt][nt][e] *= f;
                    w.o[mt][nt][2 + e] *= f;
                }
            }
        if (!OWN) w.u = unew;
    }
    if (!OWN) w.u_min = least;
    uint32_t pb[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float pv[4][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float pe[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pe[i] = tcfwd::ex2(OWN ? fmaf(x[nt][e][i] - ref[nt][e], w.f[nt][e], kPOff)
                                       : fmaf(x[nt][e][i], w.f[nt][e], ref[nt][e]));
            w.l[nt][e] += (pe[0] + pe[1]) + (pe[2] + pe[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)  // (a scale that is no number counts only where its key does)
                pv[i][e] = EDGE && x[nt][e][i] == -INFINITY ? 0.f : (OWN ? pe[i] * own.unit[nt][e] : pe[i]) * vw[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pb[i >> 1][nt][i & 1] = movmatrix_trans(MmaOp<__half>::pack(pv[i][0], pv[i][1]));
    }

    // O^T += V^T P^T: rows g and g + 8 of a 16-column step are its columns
    // 2 g and 2 g + 1
    uint32_t vmask[2][2], nans = 0;
    if (EDGE) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int h = 0; h < 2; ++h) vmask[kt][h] = key_mask(key0 + kt * 16 + h * 8 + 2 * tig, klo, kend);
    }
#pragma unroll
    for (int cc = 0; cc < DP / 16; cc += 2) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
            uint32_t r[4];
            ldmatrix_x4_trans(r, vs + chunk_at<DP>(kw0 + kt * 16 + (lane & 15), cc + (lane >> 4)));
            if (EDGE) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    r[i] &= vmask[kt][i & 1];
                    if (CODE == kCodeE4m3) {
                        const uint32_t n = nan_codes(r[i]);
                        nans |= n;
                        r[i] &= ~((n >> 7) * 0xffu);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t f[4];
                Op::even_odd(r[2 * h], f[0], f[1]);
                Op::even_odd(r[2 * h + 1], f[2], f[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    MmaOp<__half>::run(w.o[cc + h][nt], f, pb[kt][nt][0], pb[kt][nt][1]);
            }
        }
    }
    if (EDGE && CODE == kCodeE4m3 && __any_sync(0xffffffffu, nans != 0)) {
        Legal<NT> legal;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                legal.lo[nt][e] = w.lo[nt][e];
                legal.hi[nt][e] = w.hi[nt][e];
            }
        const NanBits bits = find_nans<DP, NT>(legal, vs, kw0, key0, klo, kend);
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((bits.w[mt / 4] >> ((mt % 4 * NT + nt) * 4 + j)) & 1u)
                        w.o[mt][nt][j] = __int_as_float(0x7fffffff);
    }
    return true;
}

// The rest of a sequence's tiles, [t, end), in stages from it on, with a unit for each row
// (unit[]: what O is in at the end).  (A function of its own: its code would cost the
// others' steps registers.)
template <int CODE, int DP, int NT>
__device__ __noinline__ bool own_steps(const Q8Args &a, Rows<DP, NT> &rows, float (&unit)[NT][2], uint8_t *smem,
                                       int kbeg, int klo, int kend, int t, int end, uint32_t it) {
    using L = Ring<DP, NT>;
    constexpr int NS = L::NS;
    const uint32_t sbase = smem_u32(smem), full = sbase + L::BARS, empty = full + 8 * NS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::SHARE + 24);
    const int kw0 = (threadIdx.x >> 5) * 32;
    Rows<DP, NT> w = rows;
    Own<NT> own;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            own.unit[nt][e] = 1.f / w.u;
            own.bound[nt][e] = 0x1p55f;  // (of 2^31 keys)
            const int ef = min(max((int)(__float_as_uint(w.f[nt][e]) >> 23) - 127, -60), 0);
            own.kf[nt][e] = pow2(ef);
            w.f[nt][e] *= pow2(-ef);
            w.m[nt][e] *= pow2(ef);
        }
    bool ok = true;
    for (; t < end; ++t, ++it) {
        const uint32_t s = it % NS;
        const bool got = sm100::mbar_wait(full + 8 * s, (it / NS) & 1u, abort_flag, a.p.wait_ns);
        if (!__all_sync(0xffffffffu, got)) {
            if ((threadIdx.x & 31) == 0) {
                *abort_flag = 1;
                report_status(a.p.status, kStatusTimeoutDecode);
            }
            ok = false;
            break;
        }
        const int key0 = kbeg + t * kTile + kw0;
        const uint32_t st = sbase + s * L::STAGE;
        const float *sc = reinterpret_cast<const float *>(smem + s * L::STAGE + 2 * L::TILE) + kw0;
        if (key0 < kend)
            q8_step<CODE, DP, NT, true, true>(w, st, st + L::TILE, sc, kw0, key0, klo, kend, own);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(empty + 8 * s);
    }
    rows = w;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) unit[nt][e] = own.unit[nt][e];
    return ok;
}

// GROUPED: a KV head's rows are more than one group (a form of its own: the group's
// first row, carried along, costs the others 1 us of 36).
template <int CODE, int DP, int NT, bool GROUPED>
__global__ void __launch_bounds__(kThreads, resident(DP, NT))
    q8_decode_kernel(const __grid_constant__ Q8Args a, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
    using Op = CodeOps<CODE>;
    using L = Ring<DP, NT>;
    constexpr int NS = L::NS;
    constexpr int R = L::R;
    extern __shared__ __align__(1024) uint8_t smem[];
    const AttnParams &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, tig = lane & 3;
    // shares: CTA (share: y; head, row group: x); clusters: (sequence, head, row
    // group, rank).  (A division by what the host chose costs the prologue 0.3 us.)
    const int C = a.cluster, vheads = p.Hkv * a.groups;
    int share_i = blockIdx.y, head_i = blockIdx.x;
    if (C) {
        head_i /= C;
        share_i = head_i / vheads;
        head_i -= share_i * vheads;
    }
    int kvh = head_i, row0 = 0;
    if (GROUPED) {
        kvh /= a.groups;
        row0 = (head_i - kvh * a.groups) * R;
    }
    const int rank = C ? blockIdx.x % C : 0;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full = sbase + L::BARS, empty = full + 8 * NS;
    long long *share = reinterpret_cast<long long *>(smem + L::SHARE);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(share + 3);

    // let the merge grid (a programmatic dependent launch) be scheduled
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (warp == 4) {
        if (lane == 0) {
            for (int s = 0; s < NS; ++s) {
                sm100::mbar_init(full + 8 * s, 33);  // the bytes, and each producer lane's scales
                sm100::mbar_init(empty + 8 * s, 4);
            }
            *abort_flag = 0;
            sm100::fence_mbar_init();
            sm100::tma_prefetch_desc(&tmK);
            sm100::tma_prefetch_desc(&tmV);
        }
    }
    if (C == 0 && warp == 4) {
        // this CTA's share of the tiles of all sequences, and where it begins; the
        // first 128 sequences' tiles stay in registers between the two passes
        constexpr int CH = 4;
        int n0[CH];
        uint32_t T = 0;
#pragma unroll
        for (int k = 0; k < CH; ++k) n0[k] = 32 * k + lane < p.B ? unit_of(a, 32 * k + lane).ntiles : 0;
#pragma unroll
        for (int k = 0; k < CH; ++k) T += n0[k];
        for (int b0 = 32 * CH; b0 < p.B; b0 += 32)
            if (b0 + lane < p.B) T += unit_of(a, b0 + lane).ntiles;
        T = __reduce_add_sync(0xffffffffu, T);
        const uint32_t shares = min((uint32_t)a.shares, T);
        const Shares sh(T, shares > 0 ? shares : 1);
        uint32_t t0 = 0, left = 0;
        if (share_i < (int)shares) {
            t0 = sh.begin(share_i);
            left = sh.begin(share_i + 1) - t0;
        }
        uint32_t before = 0;
        bool found = left == 0;
        auto look = [&](int b0, int n) {
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const uint32_t first = before + incl - n;
            const bool here = t0 >= first && t0 < first + n;
            if (here) {
                share[1] = b0 + lane;
                share[2] = t0 - first;
                if (head_i == 0) {
                    // where the sequence's first seam is this share's beginning
                    int4 v = make_int4(-1, 0, 0, 0);
                    const int c0 = (int)sh.of(first);
                    if (t0 > first && c0 == share_i - 1)
                        v = make_int4(b0 + lane, c0, (int)sh.of(first + n - 1), sh.begin(c0) < first ? 1 : 0);
                    a.seam[share_i] = v;
                }
            }
            found = __any_sync(0xffffffffu, here);
            before += __shfl_sync(0xffffffffu, incl, 31);
        };
#pragma unroll
        for (int k = 0; k < CH; ++k)
            if (!found && 32 * k < p.B) look(32 * k, n0[k]);
        for (int b0 = 32 * CH; !found && b0 < p.B; b0 += 32)
            look(b0, b0 + lane < p.B ? unit_of(a, b0 + lane).ntiles : 0);
        if (lane == 0) {
            share[0] = left;
            if (left == 0 && head_i == 0) a.seam[share_i] = make_int4(-1, 0, 0, 0);
        }
    } else if (C == 0) {
        // meanwhile: the rows of sequences without keys, +0 and -inf (each lane
        // looks at one of the CTA's sequences and heads, the warp writes)
        const uint32_t units = (uint32_t)p.B * p.Hkv, step = gridDim.x * gridDim.y;
        const uint32_t cta = blockIdx.y * gridDim.x + blockIdx.x;
        for (uint64_t x0 = cta + (uint64_t)warp * 32 * step; x0 < units; x0 += 128ull * step) {
            const uint64_t x = x0 + (uint64_t)lane * step;
            const uint32_t b = x < units ? (uint32_t)x / (uint32_t)p.Hkv : 0u;
            unsigned todo = __ballot_sync(0xffffffffu, x < units && unit_of(a, b).ntiles == 0);
            for (; todo; todo &= todo - 1) {
                const uint32_t y = (uint32_t)x0 + (__ffs(todo) - 1) * step;
                empty_rows(a, y / (uint32_t)p.Hkv, y % (uint32_t)p.Hkv, lane);
            }
        }
    }
    UnitKeys un;
    if (C) un = unit_of(a, share_i);
    __syncthreads();
    long long left;
    int b, tile;
    if (C) {
        b = share_i;
        if (un.ntiles == 0) {  // (so it is for the whole cluster)
            if (rank == 0 && row0 == 0 && warp == 0) empty_rows(a, b, kvh, lane);
            return;
        }
        tile = rank * un.ntiles / C;  // (some ranks have none where there are few)
        left = (rank + 1) * un.ntiles / C - tile;
    } else {
        left = share[0];
        if (left == 0) return;
        b = (int)share[1];
        tile = (int)share[2];
        un = unit_of(a, b);
    }
    // the next sequence that has tiles
    auto advance = [&]() {
        tile = 0;
        do {
            ++b;
            un = unit_of(a, b);
        } while (un.ntiles == 0);
    };

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        const int nblk = a.c.nblk, nbox = kTile >> a.box_shift;
        const int pmask = p.page_size - 1;
        uint32_t it = 0;  // tiles issued by this CTA
        bool ok = true;
        while (left > 0 && ok) {
            const int n = (int)min((long long)(un.ntiles - tile), left);
            const int32_t *table = p.block_table + (long long)b * p.max_pages;
            // pages a warp's width of boxes at a time, one group ahead: lane i of
            // group x has box 32 x + i, counted from the segment's first tile
            const int tiles_a_group = 32 / nbox;
            auto pages_of = [&](int x) -> int {
                const long long key =
                    (long long)un.kbeg + (long long)tile * kTile + ((long long)(32 * x + lane) << a.box_shift);
                int pg = 0;
                if (key < un.kend) pg = __ldg(table + (key >> p.page_shift));
                return min(max(pg, 0), p.num_pages - 1);
            };
            int pg_group = pages_of(0), pg_next = pages_of(1);
            for (int t = tile; t < tile + n; ++t, ++it) {
                const uint32_t s = it % NS;
                const uint32_t fb = full + 8 * s, st = sbase + s * L::STAGE;
                const int in_group = (t - tile) % tiles_a_group;
                if (in_group == 0 && t > tile) {
                    pg_group = pg_next;
                    pg_next = pages_of((t - tile) / tiles_a_group + 1);
                }
                // lane i: the page of box i
                const int pg = __shfl_sync(0xffffffffu, pg_group, (in_group * nbox + lane) & 31);
                if (it >= (uint32_t)NS) {
                    const bool got = sm100::mbar_wait(empty + 8 * s, (it / NS - 1) & 1u, abort_flag, p.wait_ns);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                }
                const int key0 = un.kbeg + t * kTile;
                const int boxes = min(nbox, (un.kend - key0 + a.box_rows - 1) >> a.box_shift);
                if (lane == 0)
                    sm100::mbar_arrive_expect_tx(fb, (uint32_t)boxes * a.box_rows * DP * 2);
                __syncwarp();
                if (lane < boxes) {
                    const int row = (pg << p.page_shift) + ((key0 + (lane << a.box_shift)) & pmask);
                    const uint32_t at = st + (lane << a.box_shift) * L::HALF;
#pragma unroll
                    for (int h = 0; h < DP / L::HALF; ++h) {
                        sm100::tma_load_4d(at + h * kTile * 128, &tmK, fb, h * 128, kvh, row, 0);
                        sm100::tma_load_4d(at + L::TILE + h * kTile * 128, &tmV, fb, h * 128, kvh, row, 0);
                    }
                }
#pragma unroll
                for (int j = 0; j < kTile / 32; ++j) {
                    const int i = lane + 32 * j;
                    const unsigned key = (unsigned)key0 + i;
                    const int pk = __shfl_sync(0xffffffffu, pg, i >> a.box_shift);
                    const bool in = key < (unsigned)un.kend;
                    const long long at =
                        in ? ((long long)pk * nblk + ((key & pmask) >> a.c.blk_shift)) * p.Hkv + kvh : 0;
                    cp_async4(st + 2 * L::TILE + 4 * i, a.c.ks + at, in ? 4 : 0);
                    cp_async4(st + 2 * L::TILE + 4 * (kTile + i), a.c.vs + at, in ? 4 : 0);
                }
                cp_async_arrive(fb);
            }
            left -= n;
            if (left > 0 && ok) advance();
        }
        if (!ok && lane == 0) {  // a wait ran out
            *abort_flag = 1;
            report_status(p.status, kStatusTimeoutDecode);
        }
        // every copy issued lands before the block exits, also after an abort
        cp_async_wait<0>();
        for (uint32_t k = it > (uint32_t)NS ? it - NS : 0; k < it; ++k)
            sm100::mbar_wait_drain(full + 8 * (k % NS), (k / NS) & 1u);
        if (C <= 1) return;
    }

    // --------------------------------------------------------------- consumers
    // (clusters: the CTA's rows and log2 sums in the drained ring)
    float *xrow = reinterpret_cast<float *>(smem), *xlse = xrow + R * DP;
    const int G = p.G;
    const int nrows = min(R, p.Q * G - row0);  // rows of the CTA's group
    const int kw0 = warp * 32;
    float *stat_m = reinterpret_cast<float *>(smem + L::STATS), *stat_l = stat_m + 4 * R;
    float *stat_u = stat_l + 4 * R;
    float *mbuf = reinterpret_cast<float *>(smem + L::MERGE);
    uint32_t it = 0;
    bool ok = true;
    for (bool first_seg = true; left > 0 && warp < 4; first_seg = false) {
        const int n = (int)min((long long)(un.ntiles - tile), left);
        const int nvalid = un.si.Qb * G - row0;
        // Q^T fragments (B operand of S^T): column n = row g; in each 16 columns
        // lane tig holds columns 4 tig to 4 tig + 3, paired as the codes' bytes are.
        Rows<DP, NT> w;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + g;
            float amax = 0.f;
            uint2 raw[DP / 16];
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) raw[kk] = make_uint2(0, 0);
            if (row < nvalid) {
                const int qi = (row0 + row) / G, h = kvh * G + (row0 + row) % G;
                const uint16_t *src = static_cast<const uint16_t *>(p.q) +
                                      ((un.si.q_off + qi) * p.Hq + h) * (long long)p.D + 4 * tig;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk)
                    if (kk * 16 < p.D) raw[kk] = __ldg(reinterpret_cast<const uint2 *>(src + kk * 16));
            }
            auto val = [&](int kk, int j) -> float {
                const uint32_t two = j < 2 ? raw[kk].x : raw[kk].y;
                const uint16_t hb = (uint16_t)(two >> (16 * (j & 1)));
                return a.bf16 ? __uint_as_float((uint32_t)hb << 16) : __half2float(__ushort_as_half(hb));
            };
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fabsf(val(kk, j)));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^ea <= amax < 2^(ea + 1); the row is multiplied by 2^(14 - ea)
            const int ea = max((int)(__float_as_uint(amax) >> 23) - 127, -112);
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 14 - ea) << 23), p.scale_log2);
            // (not 0, so that it orders -inf; x f is 0 all the same for a scale of 0)
            const float f = fmaxf(fabsf(p.scale_log2) * __uint_as_float((uint32_t)max(127 + ea - 14, 1) << 23), 1e-37f);
            constexpr int J1 = Op::kPerm ? 2 : 1, J2 = Op::kPerm ? 1 : 2;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                w.q[kk][nt][0] = MmaOp<__half>::pack(val(kk, 0) * up, val(kk, J1) * up);
                w.q[kk][nt][1] = MmaOp<__half>::pack(val(kk, J2) * up, val(kk, 3) * up);
            }
            w.f[nt][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
            w.f[nt][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
        }
        // Legal keys of the two rows (per n-tile) this thread's columns hold, and
        // of all rows.
        w.u = kLeastUnit;
        w.u_min = INFINITY;
        int lo_all = 0, hi_all = INT_MAX;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * tig + e;
                int lo = 0, hi = 0;
                if (row < nvalid) legal_range((row0 + row) / G, un.si.Qb, un.si.Kb, p.window, p.mask, lo, hi);
                w.lo[nt][e] = lo;
                w.hi[nt][e] = hi;
                if (row < nrows) {
                    lo_all = max(lo_all, lo);
                    hi_all = min(hi_all, hi);
                }
                w.m[nt][e] = -INFINITY;
                w.l[nt][e] = 0.f;
            }
        lo_all = __reduce_max_sync(0xffffffffu, lo_all);
        hi_all = __reduce_min_sync(0xffffffffu, hi_all);
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) w.o[mt][nt][j] = 0.f;

        float ur[NT][2];   // what a 1 in O is
        bool own = false;  // rows have units of their own
        Own<NT> none;
        for (int t = tile; t < tile + n && ok; ++t, ++it) {
            const uint32_t s = it % NS;
            const bool got = sm100::mbar_wait(full + 8 * s, (it / NS) & 1u, abort_flag, p.wait_ns);
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0) {
                    *abort_flag = 1;
                    report_status(p.status, kStatusTimeoutDecode);
                }
                ok = false;
                break;
            }
            const int key0 = un.kbeg + t * kTile + kw0;
            const uint32_t st = sbase + s * L::STAGE;
            const float *sc = reinterpret_cast<const float *>(smem + s * L::STAGE + 2 * L::TILE) + kw0;
            bool fits = true;
            if (key0 >= lo_all && hi_all - key0 >= 32)
                fits = q8_step<CODE, DP, NT, false, false>(w, st, st + L::TILE, sc, kw0, key0, 0, 0, none);
            else if (key0 < un.kend)
                fits = q8_step<CODE, DP, NT, true, false>(w, st, st + L::TILE, sc, kw0, key0, un.klo, un.kend, none);
            if (!fits) {
                Rows<DP, NT> rest = w;
                float unit[NT][2];
                ok = own_steps<CODE, DP, NT>(a, rest, unit, smem, un.kbeg, un.klo, un.kend, t, tile + n, it);
                w = rest;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) ur[nt][e] = 1.f / unit[nt][e];
                own = true;
                it += tile + n - t;
                break;
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(empty + 8 * s);
        }

        // Merge the four warps: their maxima, sums and units through shared memory,
        // then O, brought to the common ones: warps 2 and 3 hand theirs to 0 and 1,
        // warp 1 to warp 0.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!own) ur[nt][e] = w.u;
                float ls = w.l[nt][e];
                ls += __shfl_xor_sync(0xffffffffu, ls, 4);
                ls += __shfl_xor_sync(0xffffffffu, ls, 8);
                ls += __shfl_xor_sync(0xffffffffu, ls, 16);
                w.m[nt][e] *= w.f[nt][e];  // in log2 units from here on
                if (g == 0) {
                    stat_m[warp * R + nt * 8 + 2 * tig + e] = w.m[nt][e];
                    stat_l[warp * R + nt * 8 + 2 * tig + e] = ls;
                    stat_u[warp * R + nt * 8 + 2 * tig + e] = ur[nt][e];
                }
            }
        // the four warps go on or give up together
        ok = sm100::bar_red_and(1, 128, ok);
        if (!ok) break;
        float M[NT][2], Lsum[NT][2], U[NT][2];  // U: the largest ur, brought to M
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float *sm = stat_m + nt * 8 + 2 * tig + e, *sl = stat_l + nt * 8 + 2 * tig + e;
                const float *su = stat_u + nt * 8 + 2 * tig + e;
                const float mx = fmaxf(fmaxf(sm[0], sm[R]), fmaxf(sm[2 * R], sm[3 * R]));
                const float mref = mx == -INFINITY ? 0.f : mx;
                float ls = 0.f, um = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float e2 = exp2f(sm[k * R] - mref);
                    ls += sl[k * R] * e2;
                    um = fmaxf(um, su[k * R] * e2);
                }
                M[nt][e] = mx;
                Lsum[nt][e] = ls;
                U[nt][e] = um;
                // (a row without keys: 0, and so is O)
                const float f = um > 0.f ? exp2f(w.m[nt][e] - mref) * ur[nt][e] / um : 0.f;
#pragma unroll
                for (int mt = 0; mt < DP / 16; ++mt) {
                    w.o[mt][nt][e] *= f;
                    w.o[mt][nt][2 + e] *= f;
                }
            }
#pragma unroll
        for (int c0 = 0; c0 < DP / 16; c0 += L::MC / 16) {
            auto at = [&](int k, int mt, int nt, int e) -> float2 * {
                return reinterpret_cast<float2 *>(mbuf + (k * R + nt * 8 + 2 * tig + e) * L::PITCH + mt * 16 + 2 * g);
            };
            auto put = [&](int k) {
#pragma unroll
                for (int mt = 0; mt < L::MC / 16; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *at(k, mt, nt, e) = make_float2(w.o[c0 + mt][nt][e], w.o[c0 + mt][nt][2 + e]);
            };
            auto add = [&](int k) {
#pragma unroll
                for (int mt = 0; mt < L::MC / 16; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 v = *at(k, mt, nt, e);
                            w.o[c0 + mt][nt][e] += v.x;
                            w.o[c0 + mt][nt][2 + e] += v.y;
                        }
            };
            if (c0 > 0) sm100::named_bar_sync(1, 128);
            if (warp >= 2) put(warp - 2);
            sm100::named_bar_sync(1, 128);
            if (warp < 2) add(warp);
            if (warp == 1) put(1);
            sm100::named_bar_sync(1, 128);
            if (warp == 0) add(1);
        }

        // A whole unit goes out; a piece of one becomes a partial, the CTA's first
        // or its last.
        if (warp == 0) {
            const bool whole = n == un.ntiles && C <= 1;
            const long long slot = 2LL * (blockIdx.y * gridDim.x + blockIdx.x) + (first_seg ? 0 : 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = nt * 8 + 2 * tig + e;
                    if (row >= nrows) continue;
                    // a row without keys: +0 and -inf; one with a NaN key: NaN
                    const float ls = Lsum[nt][e];
                    const float inv = ls == 0.f ? 0.f : 1.f / ls;
                    const float unit = U[nt][e];
                    const float lse2 = ls != ls ? ls : ls > 0.f ? M[nt][e] - kPOff + __log2f(ls) : -INFINITY;
                    if (whole) {
                        const int qi = (row0 + row) / G, h = kvh * G + (row0 + row) % G;
                        const long long orow = (un.si.q_off + qi) * p.Hq + h;
                        uint16_t *dst = static_cast<uint16_t *>(p.o) + orow * p.Dv + 2 * g;
#pragma unroll
                        for (int mt = 0; mt < DP / 16; ++mt)
                            if (mt * 16 < p.Dv) {
                                const float x = w.o[mt][nt][e] * inv * unit, y = w.o[mt][nt][2 + e] * inv * unit;
                                *reinterpret_cast<uint32_t *>(dst + mt * 16) =
                                    a.bf16 ? MmaOp<__nv_bfloat16>::pack(x, y) : MmaOp<__half>::pack(x, y);
                            }
                        if (g == 0 && p.lse) p.lse[orow] = lse2 * kLn2;
                    } else {
                        const long long prow = C ? row : slot * R + row;
                        float *dst = C ? xrow + row * DP + 2 * g : a.part_o + prow * p.Dv + 2 * g;
#pragma unroll
                        for (int mt = 0; mt < DP / 16; ++mt)
                            if (mt * 16 < p.Dv)
                                *reinterpret_cast<float2 *>(dst + mt * 16) = make_float2(
                                    w.o[mt][nt][e] * inv * unit, w.o[mt][nt][2 + e] * inv * unit);
                        // (+inf, so that the merge's maximum does not pass a NaN by)
                        if (g == 0) (C ? xlse : a.part_lse)[prow] = lse2 != lse2 ? INFINITY : lse2;
                    }
                }
        }
        left -= n;
        if (left > 0) advance();
    }
    if (C <= 1) return;

    cooperative_groups::this_cluster().sync();
    join_cluster<DP>(a, b, kvh, row0, nrows, rank, un.ntiles, xrow, xlse);
    cooperative_groups::this_cluster().sync();  // every CTA's rows are read before it exits
}

// Joins the partials of a sequence that spans several shares, one row a block:
// groups of Dv / 4 threads take every ngrp-th partial, four loads in flight each
// under a running maximum, then the groups are added up.  4 to 5 us: the seam, the
// partials, the output, each a memory latency.
constexpr int kMergeThreads = 128;

__global__ void __launch_bounds__(kMergeThreads) q8_merge_kernel(const __grid_constant__ Q8Args a, int R) {
    __shared__ float4 red[kMergeThreads];
    const AttnParams &p = a.p;
    const int nrows = p.Q * p.G, per_share = p.Hkv * nrows;
    const int x = blockIdx.x / per_share, y = blockIdx.x - x * per_share;
    const int seams = gridDim.x / per_share;
    const int kvh = y / nrows, row = y - kvh * nrows;
    const int tid = threadIdx.x;
    // launched as a programmatic dependent of the decode kernel
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // the x-th seam: of share x + 1 where there can be one at each, else (fewer
    // sequences than shares) by a search
    int at_share = x + 1;
    if (seams < a.shares - 1) {
        at_share = 0;
        for (int s0 = 1, seen = 0; s0 < a.shares && at_share == 0; s0 += 32) {
            const int i = s0 + (tid & 31);
            const unsigned m = __ballot_sync(0xffffffffu, i < a.shares && __ldcg(&a.seam[i].x) >= 0);
            if (x < seen + __popc(m)) at_share = s0 + __fns(m, 0, x - seen + 1);
            seen += __popc(m);
        }
        if (at_share == 0) return;
    }
    const int4 seam = __ldcg(a.seam + at_share);
    if (seam.x < 0) return;
    const int np = seam.z - seam.y + 1;
    // the row's group and place in it (R is 8, of one group, or 16)
    const int head_i = kvh * a.groups + (a.groups > 1 ? row >> 4 : 0), r = a.groups > 1 ? row & 15 : row;
    const int C4 = p.Dv / 4, ngrp = kMergeThreads / C4, grp = tid / C4, c = tid - grp * C4;
    // the first share's last partial (unless it begins with the sequence), the
    // others' first
    auto part = [&](int i) -> long long {
        const long long cta = (long long)(seam.y + i) * (p.Hkv * a.groups) + head_i;
        return (2 * cta + (i == 0 ? seam.w : 0)) * R + r;
    };
    // a running maximum a thread, four partials loaded at a time
    float mx = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (grp < ngrp) {
        for (int i0 = grp; i0 < np; i0 += 4 * ngrp) {
            float lw[4];
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * ngrp;
                lw[k] = -INFINITY;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < np) {
                    const long long at = part(i);
                    lw[k] = __ldcg(a.part_lse + at);
                    v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * p.Dv) + c);
                }
            }
            const float mnew = fmaxf(fmaxf(fmaxf(lw[0], lw[1]), fmaxf(lw[2], lw[3])), mx);
            const float mref = mnew == -INFINITY ? 0.f : mnew;
            const float f = exp2f(mx - mref);
            mx = mnew;
            sum *= f;
            acc.x *= f;
            acc.y *= f;
            acc.z *= f;
            acc.w *= f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float w = exp2f(lw[k] - mref);
                sum += w;
                acc.x = fmaf(w, v[k].x, acc.x);
                acc.y = fmaf(w, v[k].y, acc.y);
                acc.z = fmaf(w, v[k].z, acc.z);
                acc.w = fmaf(w, v[k].w, acc.w);
            }
        }
    }
    __shared__ float2 stat[kMergeThreads];  // maximum, sum
    red[tid] = acc;
    stat[tid] = make_float2(mx, sum);
    __syncthreads();
    if (tid < C4) {
        for (int k = 1; k < ngrp; ++k) mx = fmaxf(mx, stat[k * C4 + tid].x);
        const float mref = mx == -INFINITY ? 0.f : mx;
        sum = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < ngrp; ++k) {
            const float4 v = red[k * C4 + tid];
            const float2 st = stat[k * C4 + tid];
            const float f = exp2f(st.x - mref);
            sum = fmaf(st.y, f, sum);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        put_row(a, seam.x, kvh, row, tid, acc, sum, mx);
    }
}

// The driver's cuTensorMapEncodeTiled, or null.
PFN_cuTensorMapEncodeTiled_v12000 tma_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// 3-D pool [rows][Hkv][D] of bytes as a 4-D map: boxes of box_rows rows of one
// head, `inner` bytes wide (columns past D read as zeros).
int pool_map(CUtensorMap *map, const void *ptr, int D, int Hkv, uint64_t rows, int inner, int box_rows) {
    auto fn = tma_encode_fn();
    if (fn == nullptr) {
        set_error("cuTensorMapEncodeTiled is not available from the driver");
        return 3;
    }
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, rows, 1};
    const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)D * Hkv, (cuuint64_t)D * Hkv * rows};
    const cuuint32_t box[4] = {(cuuint32_t)inner, 1, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(ptr), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          inner == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("cuTensorMapEncodeTiled failed (%d)", (int)r);
        return 3;
    }
    return 0;
}

template <int CODE, int DP, int NT, bool GROUPED>
int launch_t(const Q8Args &a, cudaStream_t stream) {
    using L = Ring<DP, NT>;
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)a.p.num_pages * a.p.page_size;
    int rc = pool_map(&tk, a.c.k, a.p.D, a.p.Hkv, rows, L::HALF, a.box_rows);
    if (rc == 0) rc = pool_map(&tv, a.c.v, a.p.Dv, a.p.Hkv, rows, L::HALF, a.box_rows);
    if (rc) return rc;
    auto kern = q8_decode_kernel<CODE, DP, NT, GROUPED>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) {
        set_error("8-bit decode kernel: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 3;
    }
    cudaLaunchConfig_t cfg = {};
    const unsigned heads = (unsigned)(a.p.Hkv * a.groups);
    cfg.gridDim = a.cluster ? dim3(a.p.B * a.cluster * heads) : dim3(heads, a.shares);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    if (a.cluster > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = a.cluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    e = cudaLaunchKernelEx(&cfg, kern, a, tk, tv);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("8-bit decode kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    if (a.cluster || a.shares == 1) return 0;
    // a sequence has one seam at most, and so has a share
    const int seams = a.p.B < a.shares - 1 ? a.p.B : a.shares - 1;
    cfg.gridDim = dim3((unsigned)(seams * a.p.Hkv * a.p.Q * a.p.G));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, q8_merge_kernel, a, (int)L::R);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("8-bit decode merge launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <int CODE, int DP> int launch_nt(const Q8Args &a, cudaStream_t stream) {
    if (a.groups > 1) return launch_t<CODE, DP, 2, true>(a, stream);
    return a.p.Q * a.p.G <= 8 ? launch_t<CODE, DP, 1, false>(a, stream)
                              : launch_t<CODE, DP, 2, false>(a, stream);
}

template <int CODE> int launch_code(const Q8Args &a, cudaStream_t stream) {
    const int w = a.p.D > a.p.Dv ? a.p.D : a.p.Dv;
    if (w <= 64) return launch_nt<CODE, 64>(a, stream);
    if (w <= 128) return launch_nt<CODE, 128>(a, stream);
    return launch_nt<CODE, 256>(a, stream);
}

int groups_of(const AttnParams &p) { return (p.Q * p.G + 15) / 16; }

int resident_ctas(const AttnParams &p, int nsm) {
    const int w = p.D > p.Dv ? p.D : p.Dv;
    return (nsm < 1 ? 1 : nsm) * resident(w <= 64 ? 64 : w <= 128 ? 128 : 256, p.Q * p.G <= 8 ? 1 : 2);
}

// CTAs of a (sequence, head) in cluster mode, 0 for shares: as many as are all
// resident, and no more than its tiles, when that leaves a CTA at most four.
int cluster_of(const AttnParams &p, int nsm) {
    const long long units = (long long)p.B * p.Hkv * groups_of(p), tiles = ((long long)p.K + kTile - 1) / kTile;
    int c = 8;
    while (c > 1 && (units * c > resident_ctas(p, nsm) || c >= 2 * tiles)) c /= 2;
    return tiles <= 4 * c && units < (1LL << 31) ? c : 0;
}

// Shares: a wave of resident CTAs, or up to four where one would leave many of them
// over: as many as take the least time, a wave's launch and first tile counted as
// eight tiles (256 rows of 8 heads, D 64, over 2000 keys: 25 us, 49 with the four waves that
// fill the GPU best).  No more than the tables' capacity has tiles.
int shares_of(const AttnParams &p, int nsm) {
    const long long ctas = resident_ctas(p, nsm), heads = (long long)p.Hkv * groups_of(p);
    const long long tiles = (long long)p.B * (((long long)p.K + kTile - 1) / kTile);
    long long best = 1, least = LLONG_MAX;
    for (int w = 1; w <= 4; ++w) {
        const long long m = w * ctas / heads, n = m < 1 ? 1 : m > tiles && tiles > 0 ? tiles : m;
        const long long cost = (n * heads + ctas - 1) / ctas * (8 + (tiles + n - 1) / n);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return (int)best;
}

}  // namespace

bool q8_decode_supported(const AttnParams &p, int dtype) {
    if (dtype != 1 && dtype != 2) return false;
    // TMA copies rows of D bytes from 16-byte boundaries, and whole 8-row swizzle atoms
    if (p.D % 16 || p.Dv % 16 || p.D > 256 || p.Dv > 256 || p.page_size < 8) return false;
    if ((long long)p.Q * p.G > kMaxRows || p.Q < 1) return false;
    // CTAs, merge blocks and tiles are counted in 32 bits
    return p.Hkv <= 65535 && (long long)p.B * p.Hkv <= (1LL << 30) &&
           (long long)p.B * (((long long)p.K + kTile - 1) / kTile) < (1LL << 31);
}

// More than 16 rows of a KV group are row groups of 16, each of which reads the codes
// (mostly from the L2: the groups of a head run at the same time), against an
// expansion of twice the codes' bytes and a prefill that does not split the keys.
// The groups win with few rows, and with more while they fill the GPU about once.
// Of the GPU's time, int8, up to K keys a sequence, groups and expansion (us):
//   D 128, 24 rows: 2 sequences of 25744, 4 heads 41 and 580; 64 of 4096, 8 heads 196
//     and 344; 64 rows: 57 and 557, 352 and 337
//   D 128, 8 heads: 256 rows over 25744 (0.8 groups an SM) 202 and 376; 4 x 128 over
//     8192 (1.7) 99 and 185, 4 x 256 (3.4) 183 and 142
//   D 256, 8 heads: 48 rows over 300 keys 21 and 16; 96 over 2000 (0.3) 33 and 38; 128
//     over 25744 (0.4) 264 and 364, 256 (0.8) 482 and 365
bool q8_decode_wins(const AttnParams &p, int nsm) {
    const int rows = p.Q * p.G;
    const long long all = (long long)p.B * p.Hkv * groups_of(p);
    if (p.D <= 128 && p.Dv <= 128) return rows <= 64 || all <= 2LL * nsm;
    return rows <= 32 || (2 * all <= nsm && p.K >= 1024);
}

unsigned long long q8_decode_workspace(const AttnParams &p, int nsm) {
    if (cluster_of(p, nsm)) return 0;
    const unsigned long long shares = shares_of(p, nsm);
    const unsigned long long rows = 2 * shares * p.Hkv * groups_of(p) * (p.Q * p.G <= 8 ? 8 : 16);
    return shares * sizeof(int4) + rows * 4 * (p.Dv + 1ull);
}

int launch_q8_decode(const AttnParams &p, const Q8Cache &c, int dtype, int nsm, void *ws,
                     cudaStream_t stream) {
    Q8Args a;
    a.p = p;
    a.c = c;
    a.bf16 = dtype == 2;
    a.box_rows = p.page_size < 64 ? p.page_size : 64;
    a.box_shift = 0;
    while ((1 << a.box_shift) < a.box_rows) ++a.box_shift;
    a.cluster = cluster_of(p, nsm);
    a.shares = shares_of(p, nsm);
    a.groups = groups_of(p);
    a.seam = static_cast<int4 *>(ws);
    a.part_o = reinterpret_cast<float *>(a.seam + a.shares);
    a.part_lse = a.part_o + 2ull * a.shares * p.Hkv * a.groups * (p.Q * p.G <= 8 ? 8 : 16) * p.Dv;
    return c.code == kCodeE4m3 ? launch_code<kCodeE4m3>(a, stream)
                               : launch_code<kCodeInt8>(a, stream);
}

}  // namespace attn
