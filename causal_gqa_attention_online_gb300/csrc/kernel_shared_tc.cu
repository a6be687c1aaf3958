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
//   warps 11, 10    issue the MMAs of chain 0 / 1:  S(x) [ PV(x) S(x + 2) ] ...
//   warp 8          finds the pieces
//   warp 9          loads Q, K and V by TMA (a box of a page, or of 128 rows of it)
//   warps 12-15     write finished O out of TMEM to the partials
// Pieces are handed to the roles through a ring of descriptors, so that loads of the
// next piece run ahead.  K/V tiles stream through a ring of shared-memory stages.
//
// Where few query rows attend to a sequence's own keys, the decode's kernel takes these
// (kernel_shared_own.cu), as a programmatic dependent.
//
// shared_join_kernel adds up each row's partials (at most two chains of each CTA that its
// jobs' shares touch) in a fixed order: results do not depend on timing.
//
// Bound: HBM for the keys while a group has few rows (a tile of 128 keys for both K and
// V, D = 128, is 64 KB: 1.5 us of an SM's share of the bandwidth); from about 256 rows on
// the chain S -> maximum -> exponentials -> P -> PV -> next S, which is serial in each of the
// two chains: neither the tensor core nor the exponentials are busy for half of it.  32 groups
// of 8 over up to 8192 keys of 8 heads of 128: 140 us, 5.8 TB/s.  64 sequences of 4 rows over
// 32768: 47 us at 1.94 GHz; an SM's CTA runs for 80000 cycles, for 13.5 tiles of keys by two of
// rows, and its tensor core for 27600.  21 sequences of 4 tokens, 64-wide heads of 4 rows, over
// 100000: 72 us, 125000 cycles for 20.6 tiles of keys by three of rows, 31600 of tensor core.
// 24 sequences of 130 tokens, 6 rows each, over 4096 + 700: 162 us, 270000 cycles of 317000 (the
// CTAs do not end together), the tensor core busy for 46%.
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
// The MMA warps share their schedulers with the softmax's warps of rows 96 .. 127 and
// 64 .. 95, which have nothing to do while a group has few rows.
constexpr int kFindWarp = 8, kLoadWarp = 9, kMmaWarp1 = 10, kMmaWarp = 11, kEpiWarp0 = 12;
// registers a lane: 2 x 176 (softmax) + 104 (MMA, loads, pieces) + 56 (epilogue) = 512,
// what 512 threads at 128 have
constexpr uint32_t kRegsSoftmax = 176, kRegsOther = 104, kRegsEpi = 56;
static_assert(2 * kRegsSoftmax + kRegsOther + kRegsEpi <= 4 * (65536 / kThreads), "register split");
constexpr uint32_t kChunkBytes = 128 * 128;  // 128 rows of 128 bytes (64 columns)
constexpr int kPieces = 4;                   // descriptors in flight

struct Piece {
    int nx;          // steps; 0: the end
    int two;         // two tiles of rows
    int qslot;       // one tile: where Q is
    int chain0;      // chain of the first step (short pieces take turns)
    int kind, b0, kvh, tok0, nrows;
    int lo, end;     // keys of the entity
    int Qb;          // a sequence's query tokens
    int key0;        // first key of the piece's first tile
    int key_end;     // end of the keys of the piece
    long long base;  // first row of its partials
    int pages[2][32];  // lanes' pages of the first tile: K, V
};
static_assert(sizeof(Piece) == 320, "descriptor");

template <int D, int DV> struct Layout {
    static constexpr int QTILE = 128 * D * 2;
    static constexpr int KTILE = 128 * D * 2, VTILE = 128 * DV * 2;
    static constexpr int STAGE = KTILE > VTILE ? KTILE : VTILE;
    static constexpr int TAIL = 2048;  // barriers, descriptors, scan
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
    B_P_READY = 14,    // [2] x [2] halves of a tile's keys
    B_O_FULL = 18,     // [2]
    B_O_EMPTY = 20,    // [2]
    B_TEARDOWN = 22,   // [2]
    B_ORDER = 24,      // [2] the other chain's MMAs of a tile are issued (two tiles of rows)
    B_KV_FULL = 26,    // [NS] full, [NS] empty
};
constexpr int kBarBytes = (B_KV_FULL + 20) * 8;  // 368
constexpr int kDescOff = 368, kScanOff = kDescOff + kPieces * (int)sizeof(Piece);  // 1648
constexpr int kBeginOff = kScanOff + 16 * 8, kSlotOff = kBeginOff + (int)sizeof(SharedBegin);
static_assert(kBarBytes <= kDescOff && kSlotOff + 8 <= 2048, "tail of shared memory");
// Lengths that are copied to shared memory (in place of the first tiles) while the shares
// are found.
constexpr int kCopied = 2048;

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
    long long *scan = reinterpret_cast<long long *>(tail + kScanOff);  // [16] warps' sums
    SharedBegin *begin = reinterpret_cast<SharedBegin *>(tail + kBeginOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail + kSlotOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const AttnParams &p = a.p;
    const uint64_t wl = p.wait_ns;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the join (a programmatic dependent launch) may be scheduled; it waits for this grid
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid < B_KV_FULL + 2 * NS) {
        // arrivals: descriptors go to the load warp, 2 MMA, 8 softmax and 4 epilogue warps;
        // Q and the ring's slots come back from both MMA warps
        const int i = tid;
        const uint32_t n = i < B_DESC_EMPTY ? 1 : i < B_Q_FULL ? 15 : i < B_Q_EMPTY ? 1 : i < B_S_FULL ? 2
                         : i < B_P_READY ? 1 : i < B_O_FULL ? 4 : i < B_O_EMPTY ? 1 : i < B_TEARDOWN ? 4
                         : i < B_KV_FULL + NS ? 1 : 2;
        mbar_init(bar(i), n);
        fence_mbar_init();
    }
    if (tid == 0) {
        *abort_flag = 0;
        begin->e = a.entities;
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

    // ---- the share: sums of the entities' costs, a run of them a thread.  The lengths
    // are copied first: what an entity costs hangs on several loads, one after the other.
    const int E = a.entities, run = (E + kThreads - 1) / kThreads;
    SharedLens z = shared_lens_of(a);
    if (a.N < kCopied && p.B <= kCopied) {
        int32_t *to = reinterpret_cast<int32_t *>(gbase + L::KV_OFF);
        // (without groups both of their arrays may be null)
        for (int i = tid; a.N > 0 && i <= a.N; i += kThreads) {
            to[i] = z.cu[i];
            if (i < a.N) to[kCopied + i] = z.shared[i];
        }
        for (int i = tid; i < p.B; i += kThreads) {
            to[2 * kCopied + i] = z.k[i];
            if (z.q) to[3 * kCopied + i] = z.q[i];
        }
        z = {to, to + kCopied, to + 2 * kCopied, z.q ? to + 3 * kCopied : nullptr};
        __syncthreads();
    }
    const int e0 = min(tid * run, E), e1 = min(e0 + run, E);
    long long mine = 0;
    int n = -1;
    for (int e = e0; e < e1; ++e) {
        n = e >= a.N ? shared_group_of(a, z, e - a.N) : -1;
        const SharedEntity x = shared_entity(a, z, e, n);
        mine += x.jobs * x.cj;
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
    const int shares = shared_ctas(W, a.ctas);
    const long long x0 = shared_bound(W, blockIdx.x, shares), x1 = shared_bound(W, blockIdx.x + 1, shares);
    if (x0 < x1 && before <= x0 && x0 < before + mine) {  // the share begins in this thread's run
        long long at = before;
        int e = e0;
        if (run > 1)
            for (;; ++e) {
                n = e >= a.N ? shared_group_of(a, z, e - a.N) : -1;
                const SharedEntity x = shared_entity(a, z, e, n);
                const long long c = x.jobs * x.cj;
                if (x0 < at + c) break;
                at += c;
            }
        *begin = shared_begin(a, z, e, n, at);
    }
    fence_proxy_async_smem();  // the copies' place is the loads' from here on
    __syncthreads();
    const uint32_t tmem = *tmem_slot;
    auto kv_full = [&](int s) { return bar(B_KV_FULL + s); };
    auto kv_empty = [&](int s) { return bar(B_KV_FULL + NS + s); };
    auto stage = [&](int s) { return base + L::KV_OFF + (uint32_t)s * L::STAGE; };

    if (warp >= 8 && warp < kEpiWarp0) {
        regs_decrease<kRegsOther>();
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ loads
            const int page = p.page_size, box = min(page, 128);  // rows of a box of keys
            constexpr int KC = D / 64, VC = DV / 64;             // boxes of 64 columns
            uint32_t it = 0;          // fills of the ring
            uint32_t nq[2] = {0, 0};  // fills of either Q tile
            uint32_t armed = 0;       // ring slots that were filled
            bool ok = true;
            for (uint32_t np = 0; ok; ++np) {
                const int slot = (int)(np % kPieces);
                if (!warp_wait(bar(B_DESC_FULL + slot), (np / kPieces) & 1u, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                const volatile Piece *d = desc + slot;
                const int nx = d->nx, two = d->two, qslot = d->qslot, kind = d->kind, kvh = d->kvh, tok0 = d->tok0;
                const int key0 = d->key0, key_end = d->key_end, nt = two ? nx >> 1 : nx;
                const int32_t *table = p.block_table + (long long)d->b0 * p.max_pages;
                int pk = d->pages[0][lane], pv = d->pages[1][lane];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_DESC_EMPTY + slot));
                if (nx == 0) break;
                // Q: a box of a tile's tokens with the heads of the group
                const int qtok = kind == 0 ? a.tile_tokens : min(p.Q, a.tile_tokens);
                for (int t = 0; t < (two ? 2 : 1) && ok; ++t) {
                    const int qs = two ? t : qslot;
                    if (!warp_wait(bar(B_Q_EMPTY + qs), (nq[qs] & 1u) ^ 1u, abort_flag, wl)) {
                        ok = false;
                        break;
                    }
                    ++nq[qs];
                    if (lane == 0) mbar_arrive_expect_tx(bar(B_Q_FULL + qs), (uint32_t)(qtok * p.G * 128 * KC));
                    __syncwarp();
                    if (lane < KC)
                        tma_load_4d(base + qs * L::QTILE + lane * kChunkBytes, kind == 0 ? &tmQ : &tmOwn,
                                    bar(B_Q_FULL + qs), lane * 64, kvh * p.G, tok0 + t * a.tile_tokens, 0);
                    __syncwarp();
                }
                // K and V: lane l's box of a tile is page l / columns, columns l % columns
                auto entry = [&](int j, int pages) -> int {
                    const int key = key0 + j * 128 + pages * box;
                    if (key >= key_end) return 0;
                    return min(max(__ldg(table + (key >> p.page_shift)), 0), p.num_pages - 1);
                };
                for (int j = 0; j < nt && ok; ++j) {
                    const int k0 = key0 + j * 128;
                    const int nb = (min(128, key_end - k0) + box - 1) / box;  // boxes of rows
                    const int inpage = k0 & (page - 1);
                    const int krow = (pk << p.page_shift) + inpage, vrow = (pv << p.page_shift) + inpage;
                    if (j + 1 < nt) {
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
                                        kv_full(s), c * 64, kvh, which ? vrow : krow, 0);
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
        } else if (warp == kFindWarp) {
            // ------------------------------------------------------------ pieces
            constexpr int KC = D / 64, VC = DV / 64;
            const int box = min(p.page_size, 128);
            SharedWalker wk(a, x0, x1, *begin);
            int qslot = 0, chain = 0;
            for (uint32_t np = 0;; ++np) {
                SharedJob k;
                int t0 = 0, t1 = 0;
                const bool more = wk.next(k, t0, t1);
                const int key0 = wk.s.x.kv_start + t0 * 128, key_end = min(k.end, wk.s.x.kv_start + t1 * 128);
                int pk = 0, pv = 0;
                if (more) {  // the first tile's pages; every entry of a key before key_end is there
                    const int32_t *table = p.block_table + (long long)wk.s.x.b0 * p.max_pages;
                    const int ka = key0 + lane / KC * box, va = key0 + lane / VC * box;
                    if (ka < key_end) pk = min(max(__ldg(table + (ka >> p.page_shift)), 0), p.num_pages - 1);
                    if (KC == VC) pv = pk;
                    else if (va < key_end) pv = min(max(__ldg(table + (va >> p.page_shift)), 0), p.num_pages - 1);
                }
                const int slot = (int)(np % kPieces);
                if (!warp_wait(bar(B_DESC_EMPTY + slot), ((np / kPieces) & 1u) ^ 1u, abort_flag, wl)) {
                    if (lane == 0) raise_abort(abort_flag, p.status, kStatusTimeoutShared);
                    break;
                }
                Piece &d = desc[slot];
                d.pages[0][lane] = pk;
                d.pages[1][lane] = pv;
                const bool two = more && k.ntok > a.tile_tokens;
                if (more && !two) qslot ^= 1;
                if (lane == 0) {
                    d.nx = !more ? 0 : two ? 2 * (t1 - t0) : t1 - t0;
                    if (more) {
                        d.two = two;
                        d.qslot = qslot;
                        d.chain0 = two ? 0 : chain;
                        d.kind = wk.s.x.kind;
                        d.b0 = wk.s.x.b0;
                        d.kvh = k.kvh;
                        d.tok0 = k.tok0;
                        d.nrows = k.ntok * p.G;
                        d.lo = wk.s.x.lo;
                        d.end = wk.s.x.end;
                        d.Qb = wk.s.x.Qb;
                        d.key0 = key0;
                        d.key_end = key_end;
                        d.base = shared_base(k.at, p.G, blockIdx.x);
                        int2 *sp = a.span[wk.s.x.kind] + k.at;
                        if (t0 == 0) sp->x = blockIdx.x;
                        if (t1 == k.nt) sp->y = blockIdx.x;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_DESC_FULL + slot));
                if (!more) break;
                if (!two) chain ^= (t1 - t0) & 1;
            }
        } else if (warp == kMmaWarp || warp == kMmaWarp1) {
            // -------------------------------------- MMA issuers, one a chain
            // The chain is  S(j) [softmax] PV(j) S(j')  ...: P comes in two halves, so that the
            // product with the first one runs while the softmax is at the second.  (S in
            // halves of 64 keys and two buffers, always one ahead, is slower: an MMA of 64
            // columns takes as long as one of 128, the rows of Q have to be read for either.)
            // What a tile needs beside P is waited for while the softmax runs.  Of the key
            // tiles that belong to the other chain alone a warp only sees that they landed,
            // and gives up its half of their slots.
            const int t = warp == kMmaWarp ? 0 : 1;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t s_tm = tm + (uint32_t)t * 128u, o_tm = tm + (uint32_t)(L::O_COL + t * DV);
            uint32_t kv = 0;  // fills of the pieces before
            uint32_t q_ph = 0, p_ph = 0, oe_ph = 0;  // parities (a bit a tile of Q, a half)
            uint32_t turn = 0;
            bool ok = true;
            for (uint32_t np = 0; ok; ++np) {
                const int slot = (int)(np % kPieces);
                if (!warp_wait(bar(B_DESC_FULL + slot), (np / kPieces) & 1u, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                const volatile Piece *d = desc + slot;
                // (shuffles: the compiler sees that the warp's values are one)
                const int nx = __shfl_sync(0xffffffffu, d->nx, 0), two = __shfl_sync(0xffffffffu, d->two, 0);
                const int qslot = __shfl_sync(0xffffffffu, d->qslot, 0), key0 = __shfl_sync(0xffffffffu, d->key0, 0);
                const int key_end = __shfl_sync(0xffffffffu, d->key_end, 0);
                const int chain0 = __shfl_sync(0xffffffffu, d->chain0, 0);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_DESC_EMPTY + slot));
                if (nx == 0) break;
                const int nj = two ? nx >> 1 : nx;  // key tiles
                const int qs = two ? t : qslot;
                const uint64_t qd = sw128_desc(base + qs * L::QTILE, 16, 1024);
                auto landed = [&](uint32_t f) -> bool {
                    return warp_wait(kv_full((int)(f % NS)), (f / NS) & 1u, abort_flag, wl);
                };
                auto pass = [&](uint32_t f) -> bool {  // K or V of a tile of the other chain
                    if (!landed(f)) return false;
                    if (lane == 0) mbar_arrive(kv_empty((int)(f % NS)));
                    return true;
                };
                // S of the keys in the ring's slot s.  Only the columns in use, in sixteens; the
                // softmax masks what is stale behind them.
                auto issue_s = [&](int s, int keys) {
                    tc_fence_after();
                    const uint32_t ncols = (uint32_t)((keys + 15) & ~15);
                    warp_mma_ss<D / 16>(s_tm, qd, sw128_desc(stage(s), 16, 1024),
                                        (a.idesc_s & ~(0x3Fu << 17)) | ((ncols >> 3) << 17));
                };
                // PV of a half, whose P is waited for
                auto issue_pv = [&](int s, int half, int keys, uint32_t accumulate) -> bool {
                    if (!warp_wait(bar(B_P_READY + 2 * t + half), (p_ph >> half) & 1u, abort_flag, wl)) return false;
                    p_ph ^= 1u << half;
                    tc_fence_after();
                    const uint64_t vd = sw128_desc(stage(s) + half * 64 * 128, kChunkBytes, 1024);
                    if (keys > 48) {
                        warp_mma_ts4(o_tm, s_tm + half * 32, vd, a.idesc_o, accumulate);
                    } else {
                        for (int kk = 0; kk * 16 < keys; ++kk)
                            warp_mma_ts(o_tm, s_tm + half * 32 + kk * 8, vd + (kk * 2048 >> 4), a.idesc_o,
                                        accumulate | (kk > 0));
                    }
                    return true;
                };
                // V rows behind the last key may hold anything: zeros, so that their P = 0
                // adds 0 (with two tiles of rows either warp writes the same ones)
                auto zero_tail = [&](int s, int nvalid) {
                    const int nzero = ((nvalid + 15) & ~15) - nvalid;
                    if (nzero == 0) return;
                    uint8_t *vt = gbase + (stage(s) - base) + nvalid * 128;
#pragma unroll
                    for (int c = 0; c < DV / 64; ++c)
                        for (int i = lane; i < nzero * 8; i += 32)
                            *reinterpret_cast<uint4 *>(vt + c * kChunkBytes + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                };
                auto keys_of = [&](int j) { return min(128, key_end - (key0 + j * 128)); };
                auto o_free = [&]() -> bool {  // the chain's O of the last piece has been read
                    const bool w = warp_wait(bar(B_O_EMPTY + t), oe_ph ^ 1u, abort_flag, wl);
                    oe_ph ^= 1u;
                    return w;
                };
                if (!warp_wait(bar(B_Q_FULL + qs), (q_ph >> qs) & 1u, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                q_ph ^= two ? 3u : 1u << qs;  // (with two tiles each warp waits for its own)
                const int step = two ? 1 : 2, j0 = two ? 0 : t ^ chain0;
                if (j0 == 1 && (!pass(kv) || !pass(kv + 1u))) ok = false;
                if (j0 >= nj && lane == 0) mbar_arrive(bar(B_Q_EMPTY + qs));  // no tile of ours
                // S of tile j, which has landed, and what it lets go of
                auto step_s = [&](int j) {
                    const int s = (int)((kv + 2u * (uint32_t)j) % NS);
                    issue_s(s, keys_of(j));
                    warp_mma_commit(bar(B_S_FULL + t));
                    warp_mma_commit(kv_empty(s));
                    if (j + step >= nj) {  // the last use of Q, whose barriers count two
                        warp_mma_commit(bar(B_Q_EMPTY + qs));
                        if (two) warp_mma_commit(bar(B_Q_EMPTY + qs));
                    }
                };
                if (ok && j0 < nj) {
                    ok = landed(kv + 2u * (uint32_t)j0);
                    if (ok) step_s(j0);
                }
                for (int j = j0; j < nj && ok; j += step) {
                    const uint32_t f = kv + 2u * (uint32_t)j;
                    const int sv = (int)((f + 1u) % NS), keys = keys_of(j);
                    const bool last = j + step >= nj;
                    if ((!two && j + 1 < nj && !pass(f + 2u)) || !landed(f + 1u) || (j == j0 && !o_free()) ||
                        (two && !last && !landed(f + 2u))) {
                        ok = false;
                        break;
                    }
                    zero_tail(sv, keys);
                    if (keys > 64) ok = issue_pv(sv, 0, 64, j > j0);
                    // With two tiles of rows the warps take turns at what closes a tile, so
                    // that the chains stay half a tile apart: where their MMAs mix, both get
                    // their S late and then run their softmax at the same time.
                    if (ok && two) {
                        ok = warp_wait(bar(B_ORDER + t), (turn & 1u) ^ (t == 0 ? 1u : 0u), abort_flag, wl);
                        ++turn;
                    }
                    if (ok) ok = keys > 64 ? issue_pv(sv, 1, keys - 64, 1u) : issue_pv(sv, 0, keys, j > j0);
                    if (!ok) break;
                    // The next K has landed: its S goes right behind PV, and V is released
                    // after both.
                    if (two) {
                        if (!last) step_s(j + step);
                        if (lane == 0) mbar_arrive(bar(B_ORDER + (t ^ 1)));
                    }
                    warp_mma_commit(kv_empty(sv));
                    if (last) warp_mma_commit(bar(B_O_FULL + t));
                    if (two) continue;
                    if (j + 1 < nj && !pass(f + 3u)) ok = false;
                    if (ok && !last) {
                        ok = landed(f + 4u);
                        if (ok) step_s(j + step);
                    }
                }
                kv += 2u * (uint32_t)nj;
            }
            if (!ok && lane == 0) raise_abort(abort_flag, p.status, kStatusTimeoutShared);
            warp_mma_commit(bar(B_TEARDOWN + t));  // all MMAs have completed before TMEM is released
            mbar_wait_drain(bar(B_TEARDOWN + t), 0);
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
            const int rel = two ? t : t ^ d->chain0;    // step of the chain's first tile
            const int first = two ? t * tile_rows : 0;  // row of the piece in lane 0
            const int nrows = min(d->nrows - first, tile_rows), key_end = d->key_end;
            const long long at = d->base + (two ? first : rel * d->nrows) + r;
            // the row's keys [lo, hi)
            const bool valid = r < nrows;
            int hi = 0;
            if (valid && nx > 0) {
                const int token = d->tok0 + (first + r) / p.G;
                const int b = p.Q == 1 ? token : token / p.Q, i = token - b * p.Q;
                int len = d->end, Qb = d->Qb;
                if (kind == 0) {
                    len = clamp_len(__ldg(p.seqlens_k + b), p.K);
                    Qb = p.seqlens_q ? clamp_len(__ldg(p.seqlens_q + b), p.Q) : p.Q;
                }
                if (i < Qb) hi = min(len - Qb + i + 1, d->end);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DESC_EMPTY + slot));
            if (nx == 0) break;
            const bool idle = !__any_sync(0xffffffffu, valid);  // no row in this warp
            float m_run = -INFINITY, l_run = 0.f;
            // A tile's maximum: the factor for what was summed before, and minus the maximum
            // to exponentiate with.  O is rescaled only when the maximum grows by more than
            // 2^8: a stale one serves as well, the partial refers to it.
            auto step_max = [&](float m_tile, float &neg_m) -> float {
                float alpha = 1.f;
                bool rescale = false;
                if (m_run == -INFINITY) {
                    m_run = m_tile;
                } else if (m_tile > m_run + 8.f) {
                    alpha = ex2(m_run - m_tile);
                    m_run = m_tile;
                    rescale = true;
                }
                neg_m = m_run == -INFINITY ? 0.f : -m_run;
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
                return alpha;
            };
            auto p_ready = [&](int half) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P_READY + 2 * t + half));
            };
            for (int x = rel; x < nx; x += 2) {
                const int k0 = key0 + (two ? x >> 1 : x) * 128, keys = min(128, key_end - k0);
                if (!warp_wait(bar(B_S_FULL + t), s_ph, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                s_ph ^= 1u;
                tc_fence_after();
                if (idle) {  // nothing to do for these rows
                    p_ready(0);
                    if (keys > 64) p_ready(1);
                } else if (__all_sync(0xffffffffu, !valid || (lo <= k0 && hi >= k0 + 128))) {
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
                    float neg_m;
                    const float alpha = step_max(mx * c, neg_m);
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
                        p_ready(half);
                    }
                    float sa[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) f2unpack(acc2[i], sa[2 * i], sa[2 * i + 1]);
                    l_run = l_run * alpha + (((sa[0] + sa[1]) + (sa[2] + sa[3])) + ((sa[4] + sa[5]) + (sa[6] + sa[7])));
                } else {
                    // A tile that ends before 128 keys, or where a row's keys do: 32 keys at a
                    // time, those outside [lo, hi) as -inf, and none past the last that the
                    // product with V takes.
                    const int nch = (keys + 31) / 32;
                    auto load = [&](int cc, uint32_t (&v)[32]) {
                        const int a0 = min(max(lo - k0 - cc * 32, 0), 32);
                        const int b0 = min(max(hi - k0 - cc * 32, 0), 32);
                        const uint32_t below_b = b0 >= 32 ? 0xffffffffu : (1u << b0) - 1u;
                        const uint32_t below_a = a0 >= 32 ? 0xffffffffu : (1u << a0) - 1u;
                        const uint32_t keep = below_b & ~below_a;
                        tmem_ld32(tS + cc * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = ((keep >> i) & 1u) ? v[i] : 0xff800000u;
                    };
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int cc = 0; cc < nch; ++cc) {
                        uint32_t v[32];
                        load(cc, v);
                        float m4[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) m4[i] = mx;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            m4[i & 3] = fmax3(m4[i & 3], __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
                    }
                    float neg_m;
                    const float alpha = step_max(mx * c, neg_m);
                    float sum = 0.f;
#pragma unroll 1
                    for (int cc = 0; cc < nch; ++cc) {
                        uint32_t v[32], pk[16];
                        load(cc, v);
                        float s2[2] = {0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float p0 = ex2(fmaf(__uint_as_float(v[2 * i]), c, neg_m));
                            const float p1 = ex2(fmaf(__uint_as_float(v[2 * i + 1]), c, neg_m));
                            s2[i & 1] += p0 + p1;
                            pk[i] = pack2<T>(p0, p1);
                        }
                        sum += s2[0] + s2[1];
                        tmem_st16(tS + 16 * cc, pk);  // over keys that have been read
                        if (cc == 3 || cc == nch - 1) p_ready(cc >> 1);
                        else if (cc == 1) p_ready(0);
                    }
                    l_run = l_run * alpha + sum;
                }
            }
            // (a chain without a step says so)
            if (ok && valid) a.part_ml[kind][at] = make_float2(m_run, l_run);
        }
        if (!ok && lane == 0) raise_abort(abort_flag, p.status, kStatusTimeoutShared);
    } else {
        // ------------------------------------------------ epilogue warpgroup
        regs_decrease<kRegsEpi>();
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const int tile_rows = a.tile_tokens * p.G;
        if (blockIdx.x == 0) {  // for the join, while the first tiles are on their way
            const SharedLens z = shared_lens_of(a);
            for (int b = tid - kEpiWarp0 * 32; b < p.B; b += 128) {
                const int n = shared_group_of(a, z, b);
                int g0 = b, s = 1, keys = 0;
                if (n >= 0) {
                    shared_group(a, z, n, g0, s);
                    keys = shared_keys(a, z, n, g0, s);
                }
                a.info[b] = make_int4(g0, s, keys, 0);
            }
        }
        uint32_t o_ph = 0;
        bool ok = true;
        for (uint32_t np = 0; ok; ++np) {
            const int slot = (int)(np % kPieces);
            if (!warp_wait(bar(B_DESC_FULL + slot), (np / kPieces) & 1u, abort_flag, wl)) {
                ok = false;
                break;
            }
            const volatile Piece *d = desc + slot;
            const int nx = d->nx, two = d->two, all = d->nrows, kind = d->kind, chain0 = d->chain0;
            const long long at = d->base;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DESC_EMPTY + slot));
            if (nx == 0) break;
            for (int rel = 0; rel < 2 && rel < nx; ++rel) {
                const int t = rel ^ chain0;
                if (!warp_wait(bar(B_O_FULL + t), (o_ph >> t) & 1u, abort_flag, wl)) {
                    ok = false;
                    break;
                }
                o_ph ^= 1u << t;
                tc_fence_after();
                const int first = two ? t * tile_rows : 0;
                const bool valid = r < min(all - first, tile_rows);
                if (__any_sync(0xffffffffu, valid)) {
                    // (a warp's 32 rows lie side by side: every store is a run of 512 bytes)
                    const long long row = at + (two ? first : rel * all) + r;
                    float *to = a.part_o[kind] + (row >> 5) * 32 * p.Dv + (row & 31) * 4;
                    const uint32_t tO = tmem + lane_off + (uint32_t)(L::O_COL + t * DV);
#pragma unroll
                    for (int cc = 0; cc < DV / 32; ++cc) {
                        uint32_t ov[32];
                        tmem_ld32(tO + cc * 32, ov);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (valid && cc * 32 + i * 4 < p.Dv)
                                *reinterpret_cast<uint4 *>(to + (cc * 8 + i) * 128) =
                                    make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_O_EMPTY + t));
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

// A block joins R rows.  Its first warp finds and weighs their partials, 32 / R lanes a row,
// and leaves a list of them; then warp w adds up columns 16 w .. 16 w + 15 of all rows, four
// lanes a row, so that a load of the partials (rows side by side) is four runs of 128
// bytes.  What a block takes is latency, of the chain from the lengths to the partials
// (4 us), so many rows want blocks of 32 of them, few rows and many partials blocks of 8
// (74880 rows: 41 us and 61; 10500 rows of 2 x 12 sequences, the whole call, 38.0 and 43.2, 6300
// rows 44.6 and 34.5).
constexpr int kJoinMost = 8;  // partials a lane finds at a time

struct JoinEntry {
    const float *o;
    float w;
    int chunk;         // floats from one chunk of four columns to the next
};

template <typename T, int R>
__global__ void __launch_bounds__(256, R == 8 ? 2 : 4) shared_join_kernel(const __grid_constant__ SharedArgs a) {
    constexpr int kLanes = 32 / R, kList = kLanes * kJoinMost, kUnroll = R == 8 ? 12 : 3;
    __shared__ JoinEntry list[R][kList];
    __shared__ float max_of[R], sum_of[R];
    __shared__ int live_of[R], most_all;
    const AttnParams &p = a.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long rows = (long long)p.B * p.Q * p.Hq, row_base = (long long)blockIdx.x * R;
    const bool own = a.own_splits > 0;
    // the first warp's: partials s < n0 of the shared keys, s < all of both
    const int mine = lane / kLanes, part = lane % kLanes;
    int n0 = 0, all = 0, most = 0, two0 = 0, two1 = 0;
    long long at0 = 0, at1 = row_base + mine;
    float M = -INFINITY, sum = 0.f;
    auto place = [&](int s) -> long long {
        if (s < n0) return at0 + (two0 ? (s >> 1) * 256LL + (s & 1) * two0 : s * 256LL);
        s -= n0;
        if (own) return at1 + s * rows;
        return at1 + (two1 ? (s >> 1) * 256LL + (s & 1) * two1 : s * 256LL);
    };
    auto weigh = [&](int s) -> float2 {
        return s < all ? (s < n0 ? a.part_ml[0] : a.part_ml[1])[place(s)] : make_float2(0.f, 0.f);
    };
    if (warp == 0) {
        const long long row = row_base + mine;
        int len = 0, Qb = 0, b = 0, i = 0, h = 0;
        if (row < rows) {  // (before the wait: what the caller gave)
            const int token = rows >> 31 ? (int)(row / p.Hq) : (int)((uint32_t)row / (uint32_t)p.Hq);
            h = (int)(row - (long long)token * p.Hq);
            b = (int)((uint32_t)token / (uint32_t)p.Q);
            i = token - b * p.Q;
            len = clamp_len(__ldg(p.seqlens_k + b), p.K);
            Qb = p.seqlens_q ? clamp_len(__ldg(p.seqlens_q + b), p.Q) : p.Q;
        }
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        if (row < rows) {
            const int4 in = a.info[b];
            // where the partials of a job are: chains (one or two) of CTAs [x, y]
            auto find = [&](int kind, int &two, long long &at) -> int {
                const SharedRow r = shared_row(a, kind, in.x, in.y, in.z, b, i, h, len, Qb);
                if (!r.some) return 0;
                int2 c = a.span[kind][r.at];
                // (a launch that gave up leaves them unwritten: never past the partials)
                c.x = max(c.x, 0), c.y = min(c.y, a.ctas - 1);
                two = r.ntok > a.tile_tokens ? 0 : r.ntok * p.G;  // rows between the chains, or 0
                at = shared_base(r.at, p.G, c.x) + r.lr;
                return max(c.y - c.x + 1, 0) << (two ? 1 : 0);
            };
            n0 = find(0, two0, at0);
            if (!own) {
                all = n0 + find(1, two1, at1);
            } else if (i < Qb && len > in.z) {  // parts of the sequence's own keys, from the other kernel
                all = n0 + own_parts(in.z, len, a.own_splits);
            } else {
                all = n0;
            }
        }
        most = __reduce_max_sync(0xffffffffu, all);
        if (lane == 0) most_all = most;
    }
    float4 acc[R / 8];
#pragma unroll
    for (int g = 0; g < R / 8; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int quarter = lane & 3, chunk = warp * 4 + quarter;  // columns 4 chunk ..
    for (int s0 = 0; s0 == 0 || s0 < most; s0 += kList) {
        if (warp == 0) {
            float2 ml[kJoinMost];
#pragma unroll
            for (int k = 0; k < kJoinMost; ++k) ml[k] = weigh(s0 + part + k * kLanes);
            if (s0 == 0) {  // the largest maximum of all
#pragma unroll
                for (int k = 0; k < kJoinMost; ++k)
                    if (ml[k].y != 0.f) M = fmaxf(M, ml[k].x);
                for (int s = kList + part; s < all; s += kLanes) {
                    const float2 x = weigh(s);
                    if (x.y != 0.f) M = fmaxf(M, x.x);
                }
#pragma unroll
                for (int x = 1; x < kLanes; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
                if (part == 0) max_of[mine] = M;
            }
            int live = 0;
#pragma unroll
            for (int k = 0; k < kJoinMost; ++k) {
                const int s = s0 + part + k * kLanes;
                const bool some = ml[k].y != 0.f;  // (0: no key of this row; NaN stays)
                const uint32_t bits = (__ballot_sync(0xffffffffu, some) >> (lane - part)) & ((1u << kLanes) - 1u);
                if (some) {
                    const bool flat = s >= n0 && own;
                    const long long x = place(s);
                    JoinEntry e;
                    e.o = flat ? a.part_o[1] + x * p.Dv
                               : (s < n0 ? a.part_o[0] : a.part_o[1]) + (x >> 5) * 32 * p.Dv + (x & 31) * 4;
                    e.chunk = flat ? 4 : 128;
                    // (a sum that is NaN without a maximum poisons the row)
                    e.w = ml[k].x == -INFINITY ? 1.f : exp2f(ml[k].x - M);
                    list[mine][live + __popc(bits & ((1u << part) - 1u))] = e;
                    sum = fmaf(e.w, ml[k].y, sum);
                }
                live += __popc(bits);
            }
            float l = sum;
#pragma unroll
            for (int x = 1; x < kLanes; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
            if (part == 0) {
                live_of[mine] = live;
                sum_of[mine] = l;
            }
        }
        __syncthreads();
        most = most_all;
        int live[R / 8], longest = 0;
#pragma unroll
        for (int g = 0; g < R / 8; ++g) {
            live[g] = live_of[g * 8 + (lane >> 2)];
            longest = max(longest, live[g]);
        }
#pragma unroll 1
        for (int k0 = 0; k0 < longest; k0 += kUnroll) {
            float4 v[kUnroll][R / 8];
            float w[kUnroll][R / 8];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
#pragma unroll
                for (int g = 0; g < R / 8; ++g) {
                    v[k][g] = make_float4(0.f, 0.f, 0.f, 0.f);
                    w[k][g] = 0.f;
                    if (k0 + k >= live[g]) continue;
                    const JoinEntry e = list[g * 8 + (lane >> 2)][k0 + k];
                    w[k][g] = e.w;
                    v[k][g] = *reinterpret_cast<const float4 *>(e.o + chunk * e.chunk);
                }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k)
#pragma unroll
                for (int g = 0; g < R / 8; ++g) {
                    acc[g].x = fmaf(w[k][g], v[k][g].x, acc[g].x);
                    acc[g].y = fmaf(w[k][g], v[k][g].y, acc[g].y);
                    acc[g].z = fmaf(w[k][g], v[k][g].z, acc[g].z);
                    acc[g].w = fmaf(w[k][g], v[k][g].w, acc[g].w);
                }
        }
        if (s0 + kList < most) __syncthreads();
    }
#pragma unroll
    for (int g = 0; g < R / 8; ++g) {
        const int r = g * 8 + (lane >> 2);
        const long long row = row_base + r;
        if (row >= rows) continue;
        const float L = sum_of[r], inv = L == 0.f ? 0.f : 1.f / L;
        const float4 x = acc[g];
        uint2 o;
        o.x = pack2<T>(L == 0.f ? 0.f : x.x * inv, L == 0.f ? 0.f : x.y * inv);
        o.y = pack2<T>(L == 0.f ? 0.f : x.z * inv, L == 0.f ? 0.f : x.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.o) + row * p.Dv + chunk * 4) = o;
        if (chunk == 0 && p.lse) p.lse[row] = L == 0.f ? -INFINITY : (max_of[r] + log2f(L)) * kLn2;
    }
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
    a.info = reinterpret_cast<int4 *>(take(16ull * p.B));
    for (int k = 0; k < 2; ++k) a.span[k] = reinterpret_cast<int2 *>(take(8ull * p.B * p.Q * p.Hkv));
    const unsigned long long rows = ((unsigned long long)shared_rows(p, a.ctas) + 31) / 32 * 32;
    for (int k = 0; k < 2; ++k) {
        const bool own = k == 1 && a.own_splits > 0;
        const unsigned long long r = own ? (unsigned long long)a.own_splits * p.B * p.Q * p.Hq : rows;
        a.part_ml[k] = reinterpret_cast<float2 *>(take(8ull * r));
        a.part_o[k] = reinterpret_cast<float *>(take(4ull * r * p.Dv));
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
    a.tile_align = p.page_size < 128 ? p.page_size : 128;
    a.ctas = nsm > 0 ? nsm : 1;
    // A sequence's own keys for few rows: the decode's way (keys on M, four warps a unit)
    // needs a fifth of the time of a tile of 128 rows that are nearly all empty, and none of
    // its set-up (64 x 250 keys of 8 heads took 12 us more there; 74 sequences over 4096 shared
    // keys and up to 250 of their own 83 us, now 68).  It is a launch more: 4 x 4 sequences of
    // 320 + 40 keys 31 us a call for 29, on the GPU 18 either way.
    a.own_splits = 0;
    if (own_decode_supported(p)) {
        const long long units = (long long)p.B * p.Hkv, want = (4LL * a.ctas + units - 1) / units;
        const long long most = (p.K + kOwnKeys - 1) / kOwnKeys + 1;
        a.own_splits = (int)(want < 1 ? 1 : want > 64 ? 64 : want);
        if (a.own_splits > most) a.own_splits = (int)most;
    }
    a.entities = a.own_splits > 0 ? N : N + p.B;
    a.cost_one = p.D > 64 || p.Dv > 64 ? kCostTile128 : kCostTile64;
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
    if (a.own_splits > 0) {
        rc = launch_own_decode(a, bf16, stream);
        if (rc) return rc;
    }
    const long long rows = (long long)p.B * p.Q * p.Hq;
    const bool many = rows >= 64LL * a.ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(many ? (rows + 31) / 32 : (rows + 7) / 8));
    cfg.blockDim = dim3(p.Dv * 2);  // Dv / 16 warps
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, many ? shared_join_kernel<T, 32> : shared_join_kernel<T, 8>, a);
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
    // rows, tokens and keys are counted in 32 bits, two partials of each row
    return (long long)p.B * p.Q * p.Hq < (1LL << 30) && p.K < (1 << 30);
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
