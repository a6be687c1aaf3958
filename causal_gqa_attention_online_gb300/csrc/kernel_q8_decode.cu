// kernel_q8_decode.cu -- split-KV tensor-core decode over the 8-bit paged cache
// (bf16 / fp16 queries, at most 16 rows of a KV group, widths multiples of 16
// up to 256, pages of at least 8 rows).
//
// The products are those of the 16-bit decode, keys (or value columns) on M and
// the rows of the KV group on N,
//
//     S^T[key, row] = code_K[key, :] . Q[row, :],   s = S^T * ks[key] * f[row]
//     O^T[dv, row] += code_V^T[dv, key] . (p * vs[key] / u)^T[key, row]
//
// with m16n8k16 f16 products, fp32 accumulation.  Codes become f16 pairs in
// registers, exactly (q8.cuh), and the scales multiply scores and probabilities
// in fp32, so no key or value is rounded:
//
// * Q rows are brought to [2^14, 2^15) by a power of two (in f[row] again), so
//   that bf16's 8 bits stay exact down to 2^-29 of the row's largest element.
// * Probabilities are p = 2^(s - m + 14), in (0, 2^14]: f16's 11 bits down to
//   2^-28 of the largest, steps of 2^-38 below.  u is the largest value scale a
//   warp has seen, so p * vs / u stays in range; O is rescaled when m or u grow.
//   The 2^14 cancels against the row sum, u and the codes' unit come back in the
//   final normalisation.
// * Which bytes pair up is chosen so that no byte is moved across lanes: the
//   even and the odd bytes of a 32-bit word are the two halves of a k16 step
//   (K: Q's columns are permuted to match) or the rows dv = 2g and 2g + 1 (V: a
//   transposed ldmatrix of byte pairs gives two keys' pairs in one word).
//
// Bound: HBM, one byte an element -- at 8 flops a byte, twice the 16-bit
// decode's arithmetic per byte, the conversions (7 or 5 instructions for four
// codes) have to stay out of the way.  A CTA is four consumer warps of 32 keys
// each and a producer warp: it looks pages up one tile ahead, issues one TMA
// box per page piece (up to 64 rows) and the block scales as 4-byte cp.async,
// all completing on the stage's mbarrier; consumers free a stage with one
// arrival a warp, so no warp waits for another within a tile.  V rows past the
// last key need no zeroing: any byte is a finite f16 here, and its p is 0.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cstring>

#include "common.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "q8.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kTile = 128;  // keys a tile: 4 warps x 32
constexpr int kThreads = 160;
constexpr float kPOff = 14.f;  // p is scaled by 2^14

struct Q8Args {
    AttnParams p;
    Q8Cache c;
    int box_rows;  // rows of a TMA box: min(page_size, 64)
    int box_shift;
    bool bf16;
};

template <int DP> struct Ring {
    static constexpr int HALF = DP > 128 ? 128 : DP;  // bytes of a box row
    static constexpr int TILE = kTile * DP;
    static constexpr int STAGE = 2 * TILE + 2 * kTile * 4;
    static constexpr int NS = DP == 64 ? 5 : 3;
    static constexpr int BARS = NS * STAGE;
    static constexpr int SMEM = BARS + 16 * NS + 16;
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

template <int CODE, int DP, int NT>
__global__ void __launch_bounds__(kThreads, DP > 128 ? 1 : 2)
    q8_decode_kernel(const __grid_constant__ Q8Args a, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
    using Op = CodeOps<CODE>;
    using L = Ring<DP>;
    constexpr int NS = L::NS;
    constexpr int R = NT * 8;
    constexpr int OPITCH = DP + 4;
    static_assert(4 * R * OPITCH * 4 + 3 * 4 * R * 4 <= NS * L::STAGE, "merge buffer");
    extern __shared__ __align__(1024) uint8_t smem[];
    const AttnParams &p = a.p;

    const int split = blockIdx.x;
    const int b = blockIdx.y / p.Hkv, kvh = blockIdx.y % p.Hkv;
    const SeqInfo si = seq_info(p, b);
    const int G = p.G;
    const int nrows = p.Q * G;  // rows this unit writes (<= R)
    const int nvalid = si.Qb * G;

    // Block-uniform: key range of this split and whether it owns any row.
    int lo_min = INT_MAX, hi_max = 0;
    bool mine = false;
    for (int qi = 0; qi < p.Q; ++qi) {
        int lo = 0, hi = 0;
        if (qi < si.Qb) legal_range(qi, si.Qb, si.Kb, p.window, p.mask, lo, hi);
        const SplitSpan sp = split_span(lo, hi, p.split_len);
        if (sp.direct ? sp.first == split : (split >= sp.first && split <= sp.last)) mine = true;
        if (hi > lo) {
            lo_min = min(lo_min, lo);
            hi_max = max(hi_max, hi);
        }
    }
    // let the combine grid (a programmatic dependent launch) be scheduled
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (!mine) return;
    // tiles start on a multiple of the box, so that a box is one page's
    // (a unit without keys has no tile: lo_min is still INT_MAX there)
    const int klo = hi_max > 0 ? max(lo_min, split * p.split_len) : 0;
    const int kbeg = klo & ~(a.box_rows - 1);
    const int kend = (int)min((long long)hi_max, (split + 1LL) * p.split_len);
    const int ntiles = kend > kbeg ? (kend - kbeg + kTile - 1) / kTile : 0;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, tig = lane & 3;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full = sbase + L::BARS, empty = full + 8 * NS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::BARS + 16 * NS);
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            sm100::mbar_init(full + 8 * s, 33);  // the bytes, and each producer lane's scales
            sm100::mbar_init(empty + 8 * s, 4);
        }
        *abort_flag = 0;
        sm100::fence_mbar_init();
    }
    __syncthreads();

    float m[NT][2], l[NT][2], u = 0.f;
    float oacc[DP / 16][NT][4];

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        const int nblk = a.c.nblk, nbox = kTile >> a.box_shift;
        const int pmask = p.page_size - 1;
        const int32_t *table = p.block_table + (long long)b * p.max_pages;
        auto page_of = [&](int t) -> int {  // lane i: the page of box i of tile t
            const unsigned key = (unsigned)(kbeg + t * kTile) + ((unsigned)lane << a.box_shift);
            int pg = 0;
            if (t < ntiles && lane < nbox && key < (unsigned)kend) pg = __ldg(table + (key >> p.page_shift));
            return min(max(pg, 0), p.num_pages - 1);
        };
        int pg_next = page_of(0);
        int t = 0;
        for (; t < ntiles; ++t) {
            const int s = t % NS;
            const uint32_t fb = full + 8 * s, st = sbase + s * L::STAGE;
            const int pg = pg_next;
            pg_next = page_of(t + 1);
            if (t >= NS) {
                const bool got = sm100::mbar_wait(empty + 8 * s, (uint32_t)(t / NS - 1) & 1u, abort_flag,
                                                  p.wait_ns);
                if (!__all_sync(0xffffffffu, got)) break;
            }
            const int key0 = kbeg + t * kTile;
            const int boxes = min(nbox, (kend - key0 + a.box_rows - 1) >> a.box_shift);
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
                const int i = lane + 32 * j, key = key0 + i;
                const int pk = __shfl_sync(0xffffffffu, pg, i >> a.box_shift);
                const bool ok = (unsigned)key < (unsigned)kend;
                const long long at = ok ? ((long long)pk * nblk + ((key & pmask) >> a.c.blk_shift)) * p.Hkv + kvh : 0;
                cp_async4(st + 2 * L::TILE + 4 * i, a.c.ks + at, ok ? 4 : 0);
                cp_async4(st + 2 * L::TILE + 4 * (kTile + i), a.c.vs + at, ok ? 4 : 0);
            }
            cp_async_arrive(fb);
        }
        if (t < ntiles && lane == 0) {  // a wait ran out
            *abort_flag = 1;
            report_status(p.status, kStatusTimeoutDecode);
        }
        // every copy issued lands before the block goes on, also after an abort
        cp_async_wait<0>();
        for (int k = max(0, t - NS); k < t; ++k)
            sm100::mbar_wait_drain(full + 8 * (k % NS), (uint32_t)(k / NS) & 1u);
    } else {
        // ----------------------------------------------------------- consumers
        // Q^T fragments (B operand of S^T): column n = row g; in each 16 columns
        // lane tig holds columns 4 tig + {0, 2} and 4 tig + {1, 3}, as the codes'
        // even and odd bytes pair.
        uint32_t qf[DP / 16][NT][2];
        float rowf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = nt * 8 + g;
            float amax = 0.f;
            uint2 raw[DP / 16];
            if (row < nvalid) {
                const int qi = row / G, h = kvh * G + row % G;
                const long long at = ((si.q_off + qi) * p.Hq + h) * (long long)p.D;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    raw[kk] = make_uint2(0, 0);
                    if (kk * 16 < p.D)
                        raw[kk] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.q) +
                                                                        at + kk * 16 + 4 * tig));
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) raw[kk] = make_uint2(0, 0);
            }
            auto val = [&](int kk, int j) -> float {
                const uint32_t w = j < 2 ? raw[kk].x : raw[kk].y;
                const uint16_t hb = (uint16_t)(w >> (16 * (j & 1)));
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
            const float up = __uint_as_float((uint32_t)(127 + 14 - ea) << 23);
            const float f = p.scale_log2 * Op::kUnit * __uint_as_float((uint32_t)(max(127 + ea - 14, 1)) << 23);
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                qf[kk][nt][0] = MmaOp<__half>::pack(val(kk, 0) * up, val(kk, 2) * up);
                qf[kk][nt][1] = MmaOp<__half>::pack(val(kk, 1) * up, val(kk, 3) * up);
            }
            rowf[nt][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
            rowf[nt][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
        }
        // Legal keys of the two rows (per n-tile) this thread's columns hold.
        int rlo[NT][2], rhi[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * tig + e;
                int lo = 0, hi = 0;
                if (row < nvalid) legal_range(row / G, si.Qb, si.Kb, p.window, p.mask, lo, hi);
                rlo[nt][e] = max(lo, split * p.split_len);
                rhi[nt][e] = min(hi, kend);
                m[nt][e] = -INFINITY;
                l[nt][e] = 0.f;
            }
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) oacc[mt][nt][j] = 0.f;

        const int kw0 = warp * 32;
        for (int t = 0; t < ntiles; ++t) {
            const int s = t % NS;
            const bool got = sm100::mbar_wait(full + 8 * s, (uint32_t)(t / NS) & 1u, abort_flag, p.wait_ns);
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0) {
                    *abort_flag = 1;
                    report_status(p.status, kStatusTimeoutDecode);
                }
                break;
            }
            const int key0 = kbeg + t * kTile + kw0;
            if (key0 < kend) {
                const uint32_t ks = sbase + s * L::STAGE, vs = ks + L::TILE;
                const float *sc = reinterpret_cast<const float *>(smem + s * L::STAGE + 2 * L::TILE) + kw0;

                // S^T = K Q^T for this warp's 32 keys
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
                            const uint32_t f[4] = {Op::even(r[2 * h]), Op::even(r[2 * h + 1]),
                                                   Op::odd(r[2 * h]), Op::odd(r[2 * h + 1])};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                MmaOp<__half>::run(sacc[mt][nt], f, qf[kk + h][nt][0], qf[kk + h][nt][1]);
                        }
                    }
                }

                // the largest finite value scale so far, of keys some row attends to
                const int uk = key0 + lane;
                uint32_t ub = uk >= klo && uk < kend ? __float_as_uint(sc[kTile + lane]) & 0x7fffffffu : 0u;
                if (ub >= 0x7f800000u) ub = 0u;
                const float un = fmaxf(u, __uint_as_float(__reduce_max_sync(0xffffffffu, ub)));
                const float inv_u = un > 0.f ? 1.f / un : 0.f;
                const float ru = un > u ? u * inv_u : 1.f;
                u = un;

                float kscale[4], vw[4];  // keys g, g + 8, g + 16, g + 24
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kscale[i] = sc[g + 8 * i];
                    vw[i] = sc[kTile + g + 8 * i] * inv_u;
                }
                uint32_t pb[2][NT][2];
                bool rescale = ru != 1.f;
                float fac[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float pv[4][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float sv[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int key = key0 + g + 8 * i;
                            const bool legal = key >= rlo[nt][e] && key < rhi[nt][e];
                            sv[i] = legal ? sacc[i >> 1][nt][2 * (i & 1) + e] * kscale[i] * rowf[nt][e] : -INFINITY;
                        }
                        float mx = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float mnew = fmaxf(m[nt][e], mx);
                        const float mref = mnew == -INFINITY ? 0.f : mnew;  // no key yet: keep zeros
                        const float alpha = exp2f(m[nt][e] - mref);
                        m[nt][e] = mnew;
                        fac[nt][e] = alpha * ru;
                        rescale |= alpha != 1.f;
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float pe = exp2f(sv[i] - (mref - kPOff));
                            sum += pe;
                            // (a scale that is no number counts only where its key does)
                            pv[i][e] = sv[i] == -INFINITY ? 0.f : pe * vw[i];
                        }
                        l[nt][e] = l[nt][e] * alpha + sum;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        pb[i >> 1][nt][i & 1] = movmatrix_trans(MmaOp<__half>::pack(pv[i][0], pv[i][1]));
                }
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
                    for (int mt = 0; mt < DP / 16; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            oacc[mt][nt][0] *= fac[nt][0];
                            oacc[mt][nt][1] *= fac[nt][1];
                            oacc[mt][nt][2] *= fac[nt][0];
                            oacc[mt][nt][3] *= fac[nt][1];
                        }
                }

                // O^T += V^T P^T: rows g and g + 8 of a 16-column step are its
                // columns 2 g and 2 g + 1
#pragma unroll
                for (int cc = 0; cc < DP / 16; cc += 2) {
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt) {
                        uint32_t r[4];
                        ldmatrix_x4_trans(r, vs + chunk_at<DP>(kw0 + kt * 16 + (lane & 15), cc + (lane >> 4)));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t f[4] = {Op::even(r[2 * h]), Op::odd(r[2 * h]),
                                                   Op::even(r[2 * h + 1]), Op::odd(r[2 * h + 1])};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                MmaOp<__half>::run(oacc[cc + h][nt], f, pb[kt][nt][0], pb[kt][nt][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(empty + 8 * s);
        }
    }
    __syncthreads();  // ring drained (or given up): reuse it as the merge buffer
    if (*abort_flag) return;

    // Merge the four warps' states: [warp][row][dv], then (m, l, u) a warp and row.
    float *obuf = reinterpret_cast<float *>(smem);
    float *mbuf = obuf + 4 * R * OPITCH, *lbuf = mbuf + 4 * R, *ubuf = lbuf + 4 * R;
    if (warp < 4) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float ls = l[nt][e];
                ls += __shfl_xor_sync(0xffffffffu, ls, 4);
                ls += __shfl_xor_sync(0xffffffffu, ls, 8);
                ls += __shfl_xor_sync(0xffffffffu, ls, 16);
                const int row = nt * 8 + 2 * tig + e;
                if (g == 0) {
                    mbuf[warp * R + row] = m[nt][e];
                    lbuf[warp * R + row] = ls;
                    ubuf[warp * R + row] = u * Op::kUnit;
                }
#pragma unroll
                for (int mt = 0; mt < DP / 16; ++mt)
                    *reinterpret_cast<float2 *>(obuf + (warp * R + row) * OPITCH + mt * 16 + 2 * g) =
                        make_float2(oacc[mt][nt][e], oacc[mt][nt][2 + e]);
            }
    }
    __syncthreads();

    const int C4 = p.Dv / 4;
    for (int idx = tid; idx < nrows * C4; idx += kThreads) {
        const int row = idx / C4, c = (idx - row * C4) * 4;
        int lo = 0, hi = 0;
        if (row < nvalid) legal_range(row / G, si.Qb, si.Kb, p.window, p.mask, lo, hi);
        const SplitSpan sp = split_span(lo, hi, p.split_len);
        if (sp.direct ? sp.first != split : (split < sp.first || split > sp.last)) continue;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) M = fmaxf(M, mbuf[w * R + row]);
        const float mref = M == -INFINITY ? 0.f : M;
        float L_ = 0.f, f[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            f[w] = exp2f(mbuf[w * R + row] - mref);
            L_ += lbuf[w * R + row] * f[w];
        }
        // a row without keys: +0 and -inf; one with a NaN key: NaN
        const float inv = L_ == 0.f ? 0.f : 1.f / L_;
        float o4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 v = *reinterpret_cast<const float4 *>(obuf + (w * R + row) * OPITCH + c);
            const float k = f[w] * inv, uw = ubuf[w * R + row];
            o4[0] += v.x * k * uw;
            o4[1] += v.y * k * uw;
            o4[2] += v.z * k * uw;
            o4[3] += v.w * k * uw;
        }
        const bool nan = L_ != L_;
        const float lse = nan ? L_ : L_ > 0.f ? (M - kPOff + __log2f(L_)) * kLn2 : -INFINITY;
        const int qi = row / G, h = kvh * G + row % G;
        if (sp.direct) {
            const long long at = ((si.q_off + qi) * p.Hq + h) * (long long)p.Dv + c;
            uint2 w;
            if (a.bf16) {
                w.x = MmaOp<__nv_bfloat16>::pack(o4[0], o4[1]);
                w.y = MmaOp<__nv_bfloat16>::pack(o4[2], o4[3]);
            } else {
                w.x = MmaOp<__half>::pack(o4[0], o4[1]);
                w.y = MmaOp<__half>::pack(o4[2], o4[3]);
            }
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + at) = w;
            if (c == 0 && p.lse) p.lse[(si.q_off + qi) * p.Hq + h] = lse;
        } else {
            const long long prow = (((long long)split * p.B + b) * p.Q + qi) * p.Hq + h;
            *reinterpret_cast<float4 *>(p.part_o + prow * p.Dv + c) = make_float4(o4[0], o4[1], o4[2], o4[3]);
            // (+inf, so that the merge's maximum does not pass a NaN by)
            if (c == 0) p.part_lse[prow] = nan ? INFINITY : lse;
        }
    }
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

template <int CODE, int DP, int NT>
int launch_t(const Q8Args &a, cudaStream_t stream) {
    using L = Ring<DP>;
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)a.p.num_pages * a.p.page_size;
    int rc = pool_map(&tk, a.c.k, a.p.D, a.p.Hkv, rows, L::HALF, a.box_rows);
    if (rc == 0) rc = pool_map(&tv, a.c.v, a.p.Dv, a.p.Hkv, rows, L::HALF, a.box_rows);
    if (rc) return rc;
    auto kern = q8_decode_kernel<CODE, DP, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) {
        set_error("8-bit decode kernel: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 3;
    }
    const dim3 grid((unsigned)a.p.nsplit, (unsigned)(a.p.B * a.p.Hkv));
    kern<<<grid, kThreads, L::SMEM, stream>>>(a, tk, tv);
    e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("8-bit decode kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <int CODE, int DP> int launch_nt(const Q8Args &a, cudaStream_t stream) {
    return a.p.Q * a.p.G <= 8 ? launch_t<CODE, DP, 1>(a, stream) : launch_t<CODE, DP, 2>(a, stream);
}

template <int CODE> int launch_code(const Q8Args &a, cudaStream_t stream) {
    const int w = a.p.D > a.p.Dv ? a.p.D : a.p.Dv;
    if (w <= 64) return launch_nt<CODE, 64>(a, stream);
    if (w <= 128) return launch_nt<CODE, 128>(a, stream);
    return launch_nt<CODE, 256>(a, stream);
}

}  // namespace

bool q8_decode_supported(const AttnParams &p, int dtype) {
    if (dtype != 1 && dtype != 2) return false;
    // TMA copies rows of D bytes from 16-byte boundaries, and whole 8-row swizzle atoms
    if (p.D % 16 || p.Dv % 16 || p.D > 256 || p.Dv > 256 || p.page_size < 8) return false;
    if ((long long)p.Q * p.G > 16 || p.Q < 1) return false;
    return (long long)p.B * p.Hkv <= 65535;
}

int q8_decode_split_len(const AttnParams &p, int nsm) {
    if (nsm < 1) nsm = 1;
    const long long units = (long long)p.B * p.Hkv;
    long long len = ((long long)p.K * units + 4LL * nsm - 1) / (4LL * nsm);
    len = (len + kTile - 1) / kTile * kTile;
    if (len < kTile) len = kTile;
    if (len > 1024) len = 1024;
    return (int)len;
}

int launch_q8_decode(const AttnParams &p, const Q8Cache &c, int dtype, cudaStream_t stream) {
    if (p.nsplit > 0x7fffffff / 2) {
        set_error("8-bit decode kernel: too many splits");
        return 2;
    }
    Q8Args a;
    a.p = p;
    a.c = c;
    a.bf16 = dtype == 2;
    a.box_rows = p.page_size < 64 ? p.page_size : 64;
    a.box_shift = 0;
    while ((1 << a.box_shift) < a.box_rows) ++a.box_shift;
    return c.code == kCodeE4m3 ? launch_code<kCodeE4m3>(a, stream) : launch_code<kCodeInt8>(a, stream);
}

}  // namespace attn
