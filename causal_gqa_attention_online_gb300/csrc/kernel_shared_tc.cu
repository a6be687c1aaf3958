// kernel_shared_tc.cu -- attention of a batch whose sequences begin alike (bf16 /
// fp16), on the 5th-generation tensor cores: each group's shared keys are read once
// for all of its members, whose rows then fill the tensor cores' tiles.
//
// The work is cut into equal shares (shared.cuh); two kernels:
//
// shared_tc_kernel.  One CTA an SM takes its share piece by piece.  A piece is a tile
// range of one job: up to two tiles of 128 rows, a row being a (query token, head of
// the KV group) pair.  With two tiles of rows both use each tile of 128 keys; with one,
// the key tiles alternate between two chains of their own (S, O, maximum and sum), so
// that while one chain runs its softmax the tensor core works for the other, and each
// leaves a partial result.  Either way step x of a piece belongs to chain x & 1, and
// the roles are the same:
//   warps 0-3, 4-7  softmax of chain 0 / 1 (TMEM lane = row = thread)
//   warp 8          issues all MMAs:  S(0) S(1) [ PV(x) S(x + 2) ] ...
//   warp 10         finds the pieces and pages, and loads Q, K and V by TMA (a box of a
//                   page, or of 128 rows of it)
//   warps 12-15     write finished O out of TMEM to the partials
// Pieces are handed to the roles through a ring of descriptors, so that loads of the
// next piece run ahead.  K/V tiles stream through a ring of shared-memory stages.
//
// shared_join_kernel.  One warp a row adds up the row's partials (at most two chains of
// each CTA that its jobs' shares touch) in a fixed order: results do not depend on
// timing.
//
// Bound: HBM for the keys while a group has few rows (a tile of 128 keys for both K and
// V, D = 128, is 64 KB: 1.5 us of an SM's share of the bandwidth), the softmax and the
// tensor core from about 256 rows on.
#include <cuda.h>

#include <cmath>
#include <cstring>

#include "common.cuh"
#include "launch.h"
#include "shared.cuh"
#include "sm100_ptx.cuh"
#include "tc_softmax.cuh"

namespace attn {
namespace {

using namespace sm100;
using namespace tcfwd;

constexpr int kThreads = 512;
constexpr int kMmaWarp = 8, kLoadWarp = 10, kEpiWarp0 = 12;
// registers a lane: 2 x 184 (softmax) + 72 + 72 = 512, what 512 threads at 128 have
constexpr uint32_t kRegsSoftmax = 184, kRegsOther = 72;
static_assert(2 * kRegsSoftmax + 2 * kRegsOther <= 4 * (65536 / kThreads), "register split");
constexpr uint32_t kChunkBytes = 128 * 128;  // 128 rows of 128 bytes (64 columns)
constexpr int kPieces = 4;                   // descriptors in flight

struct Piece {
    int nx;          // steps; 0: the end
    int two;         // two tiles of rows
    int qslot;       // one tile: where Q is
    int kind, b0, tok0, nrows;
    int lo, end;     // keys of the entity / of this piece's rows
    int key0;        // first key of the piece's first tile
    int key_end;     // end of the keys of the piece
    int pad;
    long long base;  // first row of its partials
};
static_assert(sizeof(Piece) == 56, "descriptor");

template <int D, int DV> struct Layout {
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int KTILE = 128 * D * 2, VTILE = 128 * DV * 2;
    static constexpr int STAGE = KTILE > VTILE ? KTILE : VTILE;
    static constexpr int TAIL = 1024;  // barriers, descriptors, scan
    static constexpr int NS_FIT = (227 * 1024 - 1024 - TAIL - 2 * QTILE) / STAGE;
    static constexpr int NS = NS_FIT > 10 ? 10 : NS_FIT;
    static constexpr int KV_OFF = 2 * QTILE;
    static constexpr int TAIL_OFF = KV_OFF + NS * STAGE;
    static constexpr int SMEM = 1024 + TAIL_OFF + TAIL;
    static constexpr int O_COL = 256;  // TMEM columns: S0 S1 | O0 O1
    static_assert(NS >= 4 && O_COL + 2 * DV <= 512, "budget");
};

enum : int {
    B_DESC_FULL = 0,   // [kPieces]
    B_DESC_EMPTY = 4,  // [kPieces]
    B_Q_FULL = 8,      // [2] tiles of Q
    B_Q_EMPTY = 10,    // [2]
    B_S_FULL = 12,     // [2] chains
    B_P_READY = 14,    // [2]
    B_O_FULL = 16,     // [2]
    B_O_EMPTY = 18,    // [2]
    B_TEARDOWN = 20,
    B_KV_FULL = 21,    // [NS] full, [NS] empty
};
constexpr int kBarBytes = (B_KV_FULL + 20) * 8;  // 328
constexpr int kDescOff = 336, kScanOff = kDescOff + kPieces * (int)sizeof(Piece);  // 560
static_assert(kBarBytes <= kDescOff && kScanOff + 16 * 8 + 64 <= 1024, "tail of shared memory");

template <typename T, int D, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    shared_tc_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmOwn,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
    using L = Layout<D, DV>;
    constexpr int NS = L::NS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // the 128-byte-swizzle atoms
    uint8_t *gbase = smem_raw + (base - raw);
    uint8_t *tail = gbase + L::TAIL_OFF;
    const uint32_t bars = base + L::TAIL_OFF;
    auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
    Piece *desc = reinterpret_cast<Piece *>(tail + kDescOff);
    long long *scan = reinterpret_cast<long long *>(tail + kScanOff);        // [16] warps' sums
    long long *found = scan + 16;                                            // entity's first cost
    int *found_e = reinterpret_cast<int *>(found + 1);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(found + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const AttnParams &p = a.p;
    const uint64_t wl = p.wait_ns;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the join (a programmatic dependent launch) may be scheduled; it waits for this grid
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(B_DESC_FULL + i), 1);
            mbar_init(bar(B_DESC_EMPTY + i), 13);  // the MMA warp, 8 softmax and 4 epilogue warps
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(B_Q_FULL + t), 1);
            mbar_init(bar(B_Q_EMPTY + t), 1);
            mbar_init(bar(B_S_FULL + t), 1);
            mbar_init(bar(B_P_READY + t), 128);
            mbar_init(bar(B_O_FULL + t), 1);
            mbar_init(bar(B_O_EMPTY + t), 128);
        }
        mbar_init(bar(B_TEARDOWN), 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar(B_KV_FULL + s), 1);
            mbar_init(bar(B_KV_FULL + NS + s), 1);
        }
        *abort_flag = 0;
        *found_e = a.N + p.B;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(tmem_slot), 512);
        tmem_relinquish();
    }
    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmOwn);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }

    // ---- the share: sums of the entities' costs, a run of them a thread
    const int E = a.N + p.B, run = (E + kThreads - 1) / kThreads;
    const int e0 = min(tid * run, E), e1 = min(e0 + run, E);
    long long mine = 0;
    for (int e = e0; e < e1; ++e) {
        const int n = e >= a.N ? shared_group_of(a, e - a.N) : -1;
        const SharedEntity x = shared_entity(a, e, n);
        mine += (long long)x.jobs * x.cj;
        if (blockIdx.x == 0 && e >= a.N) a.group[e - a.N] = n;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long before = incl - mine, W = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scan[w];
        W += scan[w];
    }
    const long long x0 = shared_bound(W, blockIdx.x, a.ctas), x1 = shared_bound(W, blockIdx.x + 1, a.ctas);
    const bool here = x0 < x1 && before <= x0 && x0 < before + mine;
    if (here || blockIdx.x == 0) {
        long long at = before;
        for (int e = e0; e < e1; ++e) {
            const int n = e >= a.N ? shared_group_of(a, e - a.N) : -1;
            const SharedEntity x = shared_entity(a, e, n);
            const long long c = (long long)x.jobs * x.cj;
            if (here && at <= x0 && x0 < at + c) {
                *found = at;
                *found_e = e;
            }
            if (blockIdx.x == 0) a.start[e] = at;
            at += c;
        }
        if (blockIdx.x == 0 && tid == 0) a.start[E] = W;
    }
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    auto kv_full = [&](int s) { return bar(B_KV_FULL + s); };
    auto kv_empty = [&](int s) { return bar(B_KV_FULL + NS + s); };
    auto stage = [&](int s) { return base + L::KV_OFF + (uint32_t)s * L::STAGE; };

    if (warp >= 8 && warp < kEpiWarp0) {
        regs_decrease<kRegsOther>();
        if (warp == kLoadWarp) {
            // ------------------------------------------------- pieces and loads
            SharedWalker wk(a, x0, x1, *found, *found_e);
            const int page = p.page_size, box = min(page, 128);  // rows of a box of keys
            constexpr int KC = D / 64, VC = DV / 64;             // boxes of 64 columns
            uint32_t it = 0;      // fills of the ring
            uint32_t nq[2] = {0, 0};  // fills of either Q tile
            uint32_t armed = 0;   // ring slots that were filled
            int qslot = 0;
            bool ok = true;
            for (uint32_t np = 0; ok; ++np) {
                SharedJob k;
                int t0 = 0, t1 = 0;
                const bool more = wk.next(k, t0, t1);
                const int slot = (int)(np % kPieces);
                if (!warp_wait(bar(B_DESC_EMPTY + slot), ((np / kPieces) & 1u) ^ 1u, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                const bool two = more && k.ntok > a.tile_tokens;
                const int key0 = wk.x.kv_start + t0 * 128;
                const int key_end = min(k.end, wk.x.kv_start + t1 * 128);
                if (more && !two) qslot ^= 1;
                if (lane == 0) {
                    Piece d = {};
                    if (more) {
                        d.nx = two ? 2 * (t1 - t0) : t1 - t0;
                        d.two = two;
                        d.qslot = qslot;
                        d.kind = wk.x.kind;
                        d.b0 = wk.x.b0;
                        d.tok0 = k.tok0;
                        d.nrows = k.ntok * p.G;
                        d.lo = wk.x.lo;
                        d.end = wk.x.end;
                        d.key0 = key0;
                        d.key_end = key_end;
                        d.base = shared_base(k.row0, blockIdx.x);
                    }
                    desc[slot] = d;
                    mbar_arrive(bar(B_DESC_FULL + slot));
                }
                __syncwarp();
                if (!more) break;
                // Q: a box of a tile's tokens with the heads of the group
                const CUtensorMap *tq = wk.x.kind == 0 ? &tmQ : &tmOwn;
                const int qtok = wk.x.kind == 0 ? a.tile_tokens : min(p.Q, a.tile_tokens);
                for (int t = 0; t < (two ? 2 : 1) && ok; ++t) {
                    const int qs = two ? t : qslot;
                    if (!warp_wait(bar(B_Q_EMPTY + qs), (nq[qs] & 1u) ^ 1u, abort_flag, wl)) {
                        ok = false;
                        break;
                    }
                    ++nq[qs];
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar(B_Q_FULL + qs), (uint32_t)(qtok * p.G * 128 * KC));
                        for (int c = 0; c < KC; ++c)
                            tma_load_4d(base + qs * L::QTILE + c * kChunkBytes, tq, bar(B_Q_FULL + qs),
                                        c * 64, k.kvh * p.G, k.tok0 + t * a.tile_tokens, 0);
                    }
                    __syncwarp();
                }
                // K and V: lane l's box of a tile is page l / columns, columns l % columns
                const int32_t *table = p.block_table + (long long)wk.x.b0 * p.max_pages;
                auto entry = [&](int j, int pages) -> int {
                    const int key = key0 + j * 128 + pages * box;
                    if (key >= key_end) return 0;
                    return min(max(__ldg(table + (key >> p.page_shift)), 0), p.num_pages - 1);
                };
                int pk = entry(0, lane / KC), pv = KC == VC ? pk : entry(0, lane / VC);
                for (int j = 0; j < t1 - t0 && ok; ++j) {
                    const int k0 = key0 + j * 128;
                    const int nb = (min(128, key_end - k0) + box - 1) / box;  // boxes of rows
                    const int inpage = k0 & (page - 1);
                    const int krow = (pk << p.page_shift) + inpage, vrow = (pv << p.page_shift) + inpage;
                    if (j + 1 < t1 - t0) {
                        pk = entry(j + 1, lane / KC);
                        pv = KC == VC ? pk : entry(j + 1, lane / VC);
                    }
#pragma unroll
                    for (int which = 0; which < 2; ++which, ++it) {
                        const int s = (int)(it % NS);
                        const int nc = which ? VC : KC;
                        if (!warp_wait(kv_empty(s), ((it / NS) & 1u) ^ 1u, abort_flag, wl)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(kv_full(s), (uint32_t)(nb * box * 128 * nc));
                        __syncwarp();
                        armed |= 1u << s;
                        const int pg = lane / nc, c = lane - pg * nc;
                        if (pg < nb)
                            tma_load_4d(stage(s) + c * kChunkBytes + pg * box * 128, which ? &tmV : &tmK,
                                        kv_full(s), c * 64, k.kvh, which ? vrow : krow, 0);
                        __syncwarp();
                    }
                }
            }
            if (!ok && lane == 0) raise_abort(abort_flag, p.status, kStatusTimeoutShared);
            // every copy this warp issued has landed before the CTA gives up its memory
            if (lane == 0) {
                for (int t = 0; t < 2; ++t)
                    if (nq[t]) mbar_wait_drain(bar(B_Q_FULL + t), (nq[t] - 1) & 1u);
                for (int s = 0; s < NS; ++s)
                    if (armed & (1u << s)) {
                        const uint32_t last = (it - 1 - (uint32_t)s) / NS;  // its last fill
                        mbar_wait_drain(kv_full(s), last & 1u);
                    }
            }
        } else if (warp == kMmaWarp) {
            // ------------------------------------------------------ MMA issuer
            uint32_t kv = 0;  // fills used
            uint32_t q_ph = 0, p_ph = 0, oe_ph = 0;  // parities, a bit a tile / chain
            bool ok = true;
            for (uint32_t np = 0; ok; ++np) {
                const int slot = (int)(np % kPieces);
                if (!warp_wait(bar(B_DESC_FULL + slot), (np / kPieces) & 1u, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                const volatile Piece *d = desc + slot;
                const int nx = d->nx, two = d->two, qslot = d->qslot, key0 = d->key0, key_end = d->key_end;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_DESC_EMPTY + slot));
                if (nx == 0) break;
                for (int t = 0; t < (two ? 2 : 1); ++t) {
                    const int qs = two ? t : qslot;
                    if (!warp_wait(bar(B_Q_FULL + qs), (q_ph >> qs) & 1u, abort_flag, wl)) ok = false;
                    q_ph ^= 1u << qs;
                }
                if (!ok) break;
                auto tile_of = [&](int x) { return two ? x >> 1 : x; };
                // S of step x into its chain's columns; the last user of K releases it
                auto issue_s = [&](int x) -> bool {
                    const int t = x & 1, j = tile_of(x);
                    const uint32_t f = kv + 2u * (uint32_t)j;
                    const int s = (int)(f % NS);
                    if (!(two && t == 1) && !warp_wait(kv_full(s), (f / NS) & 1u, abort_flag, wl)) return false;
                    tc_fence_after();
                    if (lane == 0) {
                        const int qs = two ? t : qslot;
                        const uint64_t qd = sw128_desc(base + qs * L::QTILE, 16, 1024);
                        const uint64_t kd = sw128_desc(stage(s), 16, 1024);
                        // only the key columns in use, in sixteens; the softmax masks
                        // what is stale behind them
                        const uint32_t ncols = (uint32_t)((min(128, key_end - (key0 + j * 128)) + 15) & ~15);
                        const uint32_t idesc = (a.idesc_s & ~(0x3Fu << 17)) | ((ncols >> 3) << 17);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk / 4) * kChunkBytes + (kk % 4) * 32) >> 4;
                            mma_ss(tmem + (uint32_t)t * 128u, qd + off, kd + off, idesc, kk > 0);
                        }
                        mma_commit(bar(B_S_FULL + t));
                        if (!two || t == 1) mma_commit(kv_empty(s));
                        if (two ? x >= nx - 2 : x == nx - 1) mma_commit(bar(B_Q_EMPTY + qs));
                    }
                    __syncwarp();
                    return true;
                };
                ok = issue_s(0) && (nx < 2 || issue_s(1));
                for (int x = 0; x < nx && ok; ++x) {
                    const int t = x & 1, j = tile_of(x);
                    const uint32_t f = kv + 2u * (uint32_t)j + 1u;
                    const int s = (int)(f % NS);
                    const int nvalid = min(128, key_end - (key0 + j * 128));
                    const int ksteps = (nvalid + 15) / 16;
                    if (!(two && t == 1)) {
                        if (!warp_wait(kv_full(s), (f / NS) & 1u, abort_flag, wl)) {
                            ok = false;
                            break;
                        }
                        // V rows behind the last key may hold anything: zeros, so that
                        // their P = 0 adds 0
                        const int nzero = ksteps * 16 - nvalid;
                        if (nzero > 0) {
                            uint8_t *vt = gbase + (stage(s) - base) + nvalid * 128;
#pragma unroll
                            for (int c = 0; c < DV / 64; ++c)
                                for (int i = lane; i < nzero * 8; i += 32)
                                    *reinterpret_cast<uint4 *>(vt + c * kChunkBytes + i * 16) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                    }
                    if (x < 2) {  // the chain's O of the last piece has been read
                        if (!warp_wait(bar(B_O_EMPTY + t), ((oe_ph >> t) & 1u) ^ 1u, abort_flag, wl)) {
                            ok = false;
                            break;
                        }
                        oe_ph ^= 1u << t;
                    }
                    if (!warp_wait(bar(B_P_READY + t), (p_ph >> t) & 1u, abort_flag, wl)) {
                        ok = false;
                        break;
                    }
                    p_ph ^= 1u << t;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t vd = sw128_desc(stage(s), kChunkBytes, 1024);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            if (kk < ksteps)
                                mma_ts(tmem + (uint32_t)(L::O_COL + t * DV), tmem + (uint32_t)t * 128u + kk * 8,
                                       vd + (kk * 2048 >> 4), a.idesc_o, (x >= 2 || kk > 0) ? 1u : 0u);
                        if (!two || t == 1) mma_commit(kv_empty(s));
                        if (x + 2 >= nx) mma_commit(bar(B_O_FULL + t));
                    }
                    __syncwarp();
                    // S(x + 2) overwrites P(x): issued behind PV(x) by the same thread
                    if (x + 2 < nx) ok = issue_s(x + 2);
                }
                kv += 2u * (uint32_t)(two ? nx / 2 : nx);
            }
            if (!ok && lane == 0) raise_abort(abort_flag, p.status, kStatusTimeoutShared);
            if (lane == 0) {  // all MMAs have completed before TMEM is released
                mma_commit(bar(B_TEARDOWN));
                mbar_wait_drain(bar(B_TEARDOWN), 0);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ------------------------------------------------- softmax warpgroups
        regs_increase<kRegsSoftmax>();
        const int t = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + (uint32_t)(t * 128);
        const uint32_t tO = tmem + lane_off + (uint32_t)(L::O_COL + t * DV);
        const int tile_rows = a.tile_tokens * p.G;
        const float c = a.c_scale;
        uint32_t s_ph = 0;
        bool ok = true;
        for (uint32_t np = 0; ok; ++np) {
            const int slot = (int)(np % kPieces);
            if (!warp_wait(bar(B_DESC_FULL + slot), (np / kPieces) & 1u, abort_flag, wl)) {
                ok = false;
                break;
            }
            const volatile Piece *d = desc + slot;
            const int nx = d->nx, two = d->two, key0 = d->key0, lo = d->lo, kind = d->kind;
            const int first = two ? t * tile_rows : 0;  // row of the piece in lane 0
            const int nrows = min(d->nrows - first, tile_rows);
            const long long at = d->base + (two ? first : t * d->nrows) + r;
            // the row's keys [lo, hi)
            const bool valid = r < nrows;
            int hi = 0;
            if (valid && nx > 0) {
                const int token = d->tok0 + (first + r) / p.G;
                const int b = token / p.Q, i = token - b * p.Q;
                const int len = clamp_len(__ldg(p.seqlens_k + b), p.K);
                const int Qb = p.seqlens_q ? clamp_len(__ldg(p.seqlens_q + b), p.Q) : p.Q;
                if (i < Qb) hi = min(len - Qb + i + 1, d->end);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DESC_EMPTY + slot));
            if (nx == 0) break;
            const bool idle = !__any_sync(0xffffffffu, valid);  // no row in this warp
            float m_run = -INFINITY, l_run = 0.f;
            for (int x = t; x < nx; x += 2) {
                if (!warp_wait(bar(B_S_FULL + t), s_ph, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                s_ph ^= 1u;
                if (idle) {
                    mbar_arrive(bar(B_P_READY + t));
                    continue;
                }
                tc_fence_after();
                const int k0 = key0 + (two ? x >> 1 : x) * 128;
                if (!__all_sync(0xffffffffu, !valid || (lo <= k0 && hi >= k0 + 128))) {
                    // keys outside [lo, hi) become -inf in TMEM, in chunks of 32
#pragma unroll 1
                    for (int cc = 0; cc < 4; ++cc) {
                        const int a0 = min(max(lo - k0 - cc * 32, 0), 32);
                        const int b0 = min(max(hi - k0 - cc * 32, 0), 32);
                        const uint32_t below_b = b0 >= 32 ? 0xffffffffu : (1u << b0) - 1u;
                        const uint32_t below_a = a0 >= 32 ? 0xffffffffu : (1u << a0) - 1u;
                        const uint32_t keep = below_b & ~below_a;
                        if (__all_sync(0xffffffffu, keep == 0xffffffffu)) continue;
                        uint32_t v[32];
                        tmem_ld32(tS + cc * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = ((keep >> i) & 1u) ? v[i] : 0xff800000u;
                        tmem_st32(tS + cc * 32, v);
                    }
                    tmem_st_wait();
                }
                uint32_t sr[4][32];
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + cc * 32, sr[cc]);
                tmem_ld_wait();
                float mc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mc[i] = -INFINITY;
#pragma unroll
                for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        mc[i & 7] = fmax3(mc[i & 7], __uint_as_float(sr[cc][2 * i]),
                                          __uint_as_float(sr[cc][2 * i + 1]));
                const float mx = fmax3(fmax3(mc[0], mc[1], mc[2]), fmax3(mc[3], mc[4], mc[5]),
                                       fmaxf(mc[6], mc[7]));
                const float m_tile = mx * c;
                // O is rescaled only when the maximum grows by more than 2^8: a stale
                // one serves as well, it is what the sum and the partial refer to
                float alpha = 1.f;
                bool rescale = false;
                if (m_run == -INFINITY) {
                    m_run = m_tile;
                } else if (m_tile > m_run + 8.f) {
                    alpha = ex2(m_run - m_tile);
                    m_run = m_tile;
                    rescale = true;
                }
                const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
                if (__any_sync(0xffffffffu, rescale)) {
                    // every PV of this chain before S(x) is in O, none after
#pragma unroll
                    for (int cc = 0; cc < DV / 16; ++cc) {
                        uint32_t ov[16];
                        tmem_ld16(tO + cc * 16, ov);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st16(tO + cc * 16, ov);
                    }
                }
                const uint64_t c2 = f2pack(c, c), nm2 = f2pack(neg_m, neg_m);
                uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
#pragma unroll
                    for (int cc = 2 * half; cc < 2 * half + 2; ++cc)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint64_t x2 = ffma2(f2pack(__uint_as_float(sr[cc][2 * i]),
                                                             __uint_as_float(sr[cc][2 * i + 1])), c2, nm2);
                            float f0, f1;
                            f2unpack(x2, f0, f1);
                            const float p0 = ex2(f0), p1 = ex2(f1);
                            acc2[i & 3] = fadd2(acc2[i & 3], f2pack(p0, p1));
                            // P is rounded to the storage type, as the MMA takes it; the
                            // sum is over the unrounded values
                            pk[(cc & 1) * 16 + i] = pack2<T>(p0, p1);
                        }
                    tmem_st32(tS + 32 * half, pk);
                }
                float sa[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) f2unpack(acc2[i], sa[2 * i], sa[2 * i + 1]);
                l_run = l_run * alpha + (((sa[0] + sa[1]) + (sa[2] + sa[3])) + ((sa[4] + sa[5]) + (sa[6] + sa[7])));
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(B_P_READY + t));
            }
            if (ok && valid && t < nx) a.part_ml[kind][at] = make_float2(m_run, l_run);
        }
        if (!ok && lane == 0) raise_abort(abort_flag, p.status, kStatusTimeoutShared);
    } else {
        // ------------------------------------------------ epilogue warpgroup
        regs_decrease<kRegsOther>();
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const int tile_rows = a.tile_tokens * p.G;
        uint32_t o_ph = 0;
        bool ok = true;
        for (uint32_t np = 0; ok; ++np) {
            const int slot = (int)(np % kPieces);
            if (!warp_wait(bar(B_DESC_FULL + slot), (np / kPieces) & 1u, abort_flag, wl)) {
                ok = false;
                break;
            }
            const volatile Piece *d = desc + slot;
            const int nx = d->nx, two = d->two, all = d->nrows, kind = d->kind;
            const long long at = d->base;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DESC_EMPTY + slot));
            if (nx == 0) break;
            for (int t = 0; t < 2 && t < nx; ++t) {
                if (!warp_wait(bar(B_O_FULL + t), (o_ph >> t) & 1u, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                o_ph ^= 1u << t;
                tc_fence_after();
                const int first = two ? t * tile_rows : 0;
                const bool valid = r < min(all - first, tile_rows);
                if (__any_sync(0xffffffffu, valid)) {
                    float *to = a.part_o[kind] + (at + (two ? first : t * all) + r) * p.Dv;
                    const uint32_t tO = tmem + lane_off + (uint32_t)(L::O_COL + t * DV);
#pragma unroll
                    for (int cc = 0; cc < DV / 32; ++cc) {
                        uint32_t ov[32];
                        tmem_ld32(tO + cc * 32, ov);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (valid && cc * 32 + i * 4 < p.Dv)
                                *reinterpret_cast<uint4 *>(to + cc * 32 + i * 4) =
                                    make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
                    }
                }
                tc_fence_before();
                mbar_arrive(bar(B_O_EMPTY + t));
            }
        }
        if (!ok && lane == 0) raise_abort(abort_flag, p.status, kStatusTimeoutShared);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ the join

constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) shared_join_kernel(const __grid_constant__ SharedArgs a) {
    const AttnParams &p = a.p;
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (row >= (long long)p.B * p.Q * p.Hq) return;
    const int token = (int)(row / p.Hq), h = (int)(row - (long long)token * p.Hq);
    const int b = token / p.Q;
    const long long W = a.start[a.N + p.B];
    const int n = a.group[b];
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool mine = lane * 4 < p.Dv;
    for (int kind = n >= 0 ? 0 : 1; kind < 2; ++kind) {
        const int e = kind == 0 ? n : a.N + b;
        const SharedRow r = shared_row(a, e, n, a.start[e], W, token, h);
        if (r.x.nt == 0) continue;
        const int slots = 2 * (r.c1 - r.c0 + 1);  // two chains of each CTA
        for (int s0 = 0; s0 < slots; s0 += 32) {
            const int s = s0 + lane;
            float m = -INFINITY, l = 0.f;
            long long at = s < slots ? shared_partial(a, r, W, r.c0 + (s >> 1), s & 1) : -1;
            if (at >= 0) {
                const float2 ml = a.part_ml[kind][at];
                m = ml.x;
                l = ml.y;
                if (l == 0.f) at = -1;  // no key of this row (NaN stays)
            }
            uint32_t todo = __ballot_sync(0xffffffffu, at >= 0);
            if (todo == 0) continue;
            const float mnew = fmaxf(M, warp_max(at >= 0 ? m : -INFINITY));
            const float keep = M == -INFINITY ? (L == 0.f ? 0.f : 1.f) : exp2f(M - mnew);
            M = mnew;
            acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
            // (a sum that is NaN with no maximum poisons the row)
            const float w = at >= 0 ? (m == -INFINITY ? 1.f : exp2f(m - M)) : 0.f;
            L = L * keep + warp_sum(at >= 0 ? w * l : 0.f);
            while (todo) {
                float4 v[4];
                float ws[4];
                int cnt = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (todo) {
                        const int src = __ffs(todo) - 1;
                        todo &= todo - 1;
                        ws[u] = __shfl_sync(0xffffffffu, w, src);
                        const long long from = __shfl_sync(0xffffffffu, at, src);
                        if (mine) v[u] = *reinterpret_cast<const float4 *>(a.part_o[kind] + from * p.Dv + lane * 4);
                        cnt = u + 1;
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (u < cnt && mine) {
                        acc.x = fmaf(ws[u], v[u].x, acc.x);
                        acc.y = fmaf(ws[u], v[u].y, acc.y);
                        acc.z = fmaf(ws[u], v[u].z, acc.z);
                        acc.w = fmaf(ws[u], v[u].w, acc.w);
                    }
            }
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (mine) {
        uint2 o;
        o.x = pack2<T>(L == 0.f ? 0.f : acc.x * inv, L == 0.f ? 0.f : acc.y * inv);
        o.y = pack2<T>(L == 0.f ? 0.f : acc.z * inv, L == 0.f ? 0.f : acc.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.o) + row * p.Dv + lane * 4) = o;
    }
    if (lane == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------ host

unsigned long long round256(unsigned long long x) { return (x + 255) / 256 * 256; }

// Lays the workspace out; returns its bytes (`ws` may be null).
unsigned long long layout(SharedArgs &a, void *ws) {
    const AttnParams &p = a.p;
    char *at = static_cast<char *>(ws);
    unsigned long long n = 0;
    auto take = [&](unsigned long long bytes) {
        char *q = at + n;
        n += round256(bytes);
        return q;
    };
    a.start = reinterpret_cast<long long *>(take(8ull * (a.N + (long long)p.B + 1)));
    a.group = reinterpret_cast<int32_t *>(take(4ull * p.B));
    const unsigned long long rows = (unsigned long long)shared_rows(p, a.ctas);
    for (int k = 0; k < 2; ++k) {
        a.part_ml[k] = reinterpret_cast<float2 *>(take(8ull * rows));
        a.part_o[k] = reinterpret_cast<float *>(take(4ull * rows * p.Dv));
    }
    return n;
}

void fill(SharedArgs &a, const AttnParams &p, const int32_t *cu_groups, const int32_t *shared_lens, int N,
          int nsm) {
    a.p = p;
    a.cu_groups = cu_groups;
    a.shared_lens = shared_lens;
    a.N = N;
    a.tile_tokens = 128 / p.G;
    a.own_blocks = (p.Q + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
    a.tile_align = p.page_size < 128 ? p.page_size : 128;
    a.ctas = nsm > 0 ? nsm : 1;
}

template <typename T, int D, int DV>
int launch_t(SharedArgs &a, bool bf16, cudaStream_t stream) {
    using L = Layout<D, DV>;
    const AttnParams &p = a.p;
    a.idesc_s = idesc_f16(bf16, 128, 128, false, p.scale < 0.f);
    a.idesc_o = idesc_f16(bf16, 128, DV, true, false);
    CUtensorMap tq, town, tk, tv;
    const uint64_t tokens = (uint64_t)p.B * p.Q, keys = (uint64_t)p.num_pages * p.page_size;
    const uint32_t box = p.page_size < 128 ? p.page_size : 128;
    int rc = make_tma_map_4d(&tq, p.q, bf16, p.D, p.Hq, tokens, 1, p.G, a.tile_tokens);
    if (rc == 0) rc = make_tma_map_4d(&town, p.q, bf16, p.D, p.Hq, tokens, 1, p.G,
                                      p.Q < a.tile_tokens ? p.Q : a.tile_tokens);
    if (rc == 0) rc = make_tma_map_4d(&tk, p.k, bf16, p.D, p.Hkv, keys, 1, 1, box);
    if (rc == 0) rc = make_tma_map_4d(&tv, p.v, bf16, p.Dv, p.Hkv, keys, 1, 1, box);
    if (rc) return rc;
    auto kern = shared_tc_kernel<T, D, DV>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) {
        set_error("shared-prefix kernel: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 3;
    }
    kern<<<a.ctas, kThreads, L::SMEM, stream>>>(a, tq, town, tk, tv);
    e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("shared-prefix kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    const long long rows = (long long)p.B * p.Q * p.Hq, blocks = (rows + kJoinWarps - 1) / kJoinWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, shared_join_kernel<T>, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("shared-prefix join launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <typename T> int launch_dtype(SharedArgs &a, bool bf16, cudaStream_t stream) {
    const bool d128 = a.p.D > 64, dv128 = a.p.Dv > 64;  // tiles padded to 64 or 128 columns
    if (d128 && dv128) return launch_t<T, 128, 128>(a, bf16, stream);
    if (!d128 && !dv128) return launch_t<T, 64, 64>(a, bf16, stream);
    if (d128) return launch_t<T, 128, 64>(a, bf16, stream);
    return launch_t<T, 64, 128>(a, bf16, stream);
}

}  // namespace

bool shared_tc_supported(const AttnParams &p, int dtype) {
    if (dtype != 1 && dtype != 2) return false;
    if (p.D < 64 || p.D > 128 || p.D % 16 || p.Dv < 64 || p.Dv > 128 || p.Dv % 16) return false;
    // a tile of rows holds whole tokens; a box of a page fills whole swizzle atoms
    if (p.G > 128 || p.page_size < 8) return false;
    // rows and tokens are counted in 32 bits, two partials of each
    return (long long)p.B * p.Q * p.Hq < (1LL << 30);
}

unsigned long long shared_tc_workspace(const AttnParams &p, int N, int nsm) {
    SharedArgs a = {};
    fill(a, p, nullptr, nullptr, N, nsm);
    return layout(a, nullptr);
}

int launch_shared_tc(const AttnParams &p, const int32_t *cu_groups, const int32_t *shared_lens, int N,
                     int dtype, int nsm, void *ws, cudaStream_t stream) {
    SharedArgs a = {};
    fill(a, p, cu_groups, shared_lens, N, nsm);
    layout(a, ws);
    a.c_scale = (p.scale == 0.f ? 1e-30f : fabsf(p.scale)) * kLog2e;
    if (dtype == 2) return launch_dtype<__nv_bfloat16>(a, true, stream);
    return launch_dtype<__half>(a, false, stream);
}

}  // namespace attn
