// kernel_pages.cu -- management of a paged cache's pages: copying pages of
// several pools, the next version of a block table (fork), and compaction.
//
// Block tables and reference counts are versions: an operation reads one and
// writes the next, so a call that does not fit its pool leaves the caller's
// version as it was, and every call can be captured into a graph.  The integer
// work is latency bound (a few thousand entries); it runs as one cluster of
// kPlanCtas blocks that meet at cluster barriers, so a plan is one launch
// whatever its phases.  Per-page counts live in the cluster's shared memory where
// they fit (fork: 65536 pages, compaction: 136528), and there is no workspace then; where few bytes
// can move (kSmallBytes) the cluster copies them itself, otherwise a second launch
// does, which finds the pairs in the new version.  Larger pools, and calls that can
// move more than kListBytes, keep counts and lists in a workspace, and the table
// follows in the second launch, too.
//
// Page numbers are handed out lowest first and the results do not depend on
// the order of any atomic: counts and minima only.
//
// Measured: plan of 256 slots of 129 entries 19 us, of 16 slots of 6 entries 13 (a
// cluster barrier is about a microsecond, the rest chains of dependent loads).
//
// Copies move 2 bytes for each byte of a page.  A warp moves a chunk of a page
// with 16-byte loads, all issued before the first store, and the chunks of all
// pools form one index space, so that small pools (scales) and large ones fill
// the same launch.  500 pages of 64 KB in random order, eight layers: 175 us, 6.0
// TB/s, 0.88 of a plain copy.
#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace attn {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanCtas = 8;       // blocks of the planning cluster (the portable size)
constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kChunk = 4096;       // bytes a warp moves at a time: 8 x 16 bytes a lane

struct PoolTable {
    const uint8_t *src[kMaxPools];
    uint8_t *dst[kMaxPools];
    long long bytes[kMaxPools];      // bytes of a page
    int first_chunk[kMaxPools + 1];  // chunks of a page before this pool's
    int n;
};

// ------------------------------------------------------------------- copies

template <typename V> __device__ __forceinline__ void copy_units(uint8_t *dst, const uint8_t *src, int n, int lane) {
    constexpr int U = kChunk / 32 / 16;  // units a lane keeps in flight
    const V *s = reinterpret_cast<const V *>(src);
    V *d = reinterpret_cast<V *>(dst);
    for (int i0 = 0; i0 < n; i0 += 32 * U) {
        V v[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i * 32 + lane < n) v[i] = __ldcs(s + i0 + i * 32 + lane);
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i * 32 + lane < n) __stcs(d + i0 + i * 32 + lane, v[i]);
    }
}

// Chunk r of a page's (over all pools): page sp -> dp, by a warp.
__device__ __forceinline__ void copy_chunk(const PoolTable &t, int sp, int dp, int r) {
    int pool = 0;
    while (r >= t.first_chunk[pool + 1]) ++pool;
    const long long off = (long long)(r - t.first_chunk[pool]) * kChunk;
    const long long bytes = t.bytes[pool];
    const int len = (int)min((long long)kChunk, bytes - off), lane = threadIdx.x & 31;
    const uint8_t *s = t.src[pool] + sp * bytes + off;
    uint8_t *d = t.dst[pool] + dp * bytes + off;
    const uintptr_t low = reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(d) | (uintptr_t)len;
    if ((low & 15) == 0) copy_units<uint4>(d, s, len / 16, lane);
    else if ((low & 3) == 0) copy_units<uint32_t>(d, s, len / 4, lane);
    else copy_units<uint8_t>(d, s, len, lane);
}

// Pages pair(i).x -> pair(i).y of every pool for i < n, by warp `first`, first +
// step, ....  Pairs outside the pools are skipped.
template <typename F>
__device__ __forceinline__ void copy_pairs(const PoolTable &t, int n, int src_pages, int dst_pages,
                                           long long first, long long step, F pair) {
    const int per_page = t.first_chunk[t.n];
    const long long total = (long long)n * per_page;
    int2 next = first < total ? pair((int)(first / per_page)) : make_int2(-1, -1);
    for (long long c = first; c < total; c += step) {
        const int i = (int)(c / per_page), r = (int)(c - (long long)i * per_page);
        const int sp = next.x, dp = next.y;
        if (c + step < total) next = pair((int)((c + step) / per_page));  // under way during the copy
        if (sp < 0 || sp >= src_pages || dp < 0 || dp >= dst_pages) continue;
        copy_chunk(t, sp, dp, r);
    }
}

// Pages src[i] -> dst[i] (src_back: src[n - 1 - i] -> dst[i]), by the warps of the
// grid.
__device__ __forceinline__ void copy_pages(const PoolTable &t, const int32_t *src, const int32_t *dst, int n,
                                           int src_pages, int dst_pages, bool src_back = false) {
    const int warps = blockDim.x / 32;
    copy_pairs(t, n, src_pages, dst_pages, (long long)blockIdx.x * warps + (threadIdx.x >> 5),
               (long long)gridDim.x * warps, [&](int i) {
        return make_int2(__ldcg(src + (src_back ? n - 1 - i : i)), __ldcg(dst + i));
    });
}

__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const __grid_constant__ PoolTable t, const int32_t *src, const int32_t *dst,
                      int n, int src_pages, int dst_pages) {
    copy_pages(t, src, dst, n, src_pages, dst_pages);
}

// The same with the number of pages, and whether src runs from the back,
// decided by an earlier kernel.
__global__ void __launch_bounds__(kCopyThreads)
    copy_counted_kernel(const __grid_constant__ PoolTable t, const int32_t *src, const int32_t *dst,
                        const int32_t *count, int pages, bool src_back) {
    copy_pages(t, src, dst, __ldcg(count), pages, pages, src_back);
}

// --------------------------------------------------------------- block scans

// Exclusive sum of v over the block's NW warps; *total gets the block's sum.
// `warps`: 32 ints of shared memory.
template <int NW = 32> __device__ __forceinline__ int block_scan(int v, int *warps, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = lane < NW ? warps[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warps[lane] = w;
    }
    __syncthreads();
    *total = warps[31];
    return incl - v + (warp > 0 ? warps[warp - 1] : 0);
}

// --------------------------------------------------------------------- fork

struct ForkArgs {
    const int32_t *table, *lens, *refs, *parents, *grow;
    int S, M, P, N, page_shift;
    int32_t *table_out, *lens_out, *refs_out, *status;
    // workspace: per page, references by the old table, by full entries of the
    // new one, the lowest claiming entry, and whether an entry holds it
    int32_t *was, *full, *held;
    unsigned long long *claim;
    int32_t *need;       // pages each slot takes
    int32_t *list;       // the free pages, in ascending order
    int32_t *src, *dst;  // pages to copy (N at most)
    int32_t *count;      // [0] pages to copy
};

struct Slot {
    int parent;       // row of the old table, -1: empty
    int len;          // tokens
    long long want;   // table entries of the new version
    int nfull;        // of them, pages full of tokens (shared)
};

__device__ __forceinline__ Slot slot_of(const ForkArgs &a, int i) {
    Slot s;
    s.parent = __ldg(a.parents + i);
    s.len = 0;
    s.want = 0;
    s.nfull = 0;
    if (s.parent < 0 || s.parent >= a.S) {
        s.parent = -1;
        return s;
    }
    const long long cap = (long long)a.M << a.page_shift;
    s.len = (int)min(max((long long)__ldg(a.lens + s.parent), 0LL), cap);
    const long long grow = a.grow ? max(__ldg(a.grow + i), 0) : 0;
    s.want = (s.len + grow + (1LL << a.page_shift) - 1) >> a.page_shift;
    s.nfull = s.len >> a.page_shift;
    return s;
}

__device__ __forceinline__ int cand_of(const ForkArgs &a, const Slot &s, int j) {
    return __ldg(a.table + (long long)s.parent * a.M + j);
}

// Whether entry j (not full) of slot i keeps its parent's page: the page is
// live, no full entry and nobody outside the tables holds it, and this entry is
// the first that wants it.
__device__ __forceinline__ bool keeps(const ForkArgs &a, int i, int j, int c) {
    if (c < 0 || c >= a.P) return false;
    const int refs = __ldg(a.refs + c);
    return refs > 0 && __ldcg(a.full + c) == 0 && refs <= __ldcg(a.was + c) &&
           __ldcg(a.claim + c) == (unsigned long long)i * a.M + j;
}

// f(0), f(1), ... for the entries first, first + step, ... below end of an array,
// four loads at a time.
template <typename F>
__device__ __forceinline__ void for_entries(const int32_t *v, long long first, long long end, long long step, F f) {
    for (; first < end; first += 4 * step) {
        int c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = first + k * step < end ? __ldg(v + first + k * step) : -1;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (first + k * step < end) f(first + k * step, c[k]);
    }
}

// Four phases, each spread over the whole cluster; the dependent loads of a slot
// (parent, length, entry, the entry's page) are what they cost, so a warp takes a
// slot and every warp has as few as can be.  Slots and pages are dealt out in
// contiguous parts, so that a part's place in the order is the sum of the parts
// before it, read through distributed shared memory.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    fork_plan_kernel(const __grid_constant__ ForkArgs a) {
    __shared__ int warps[32];
    __shared__ int part_free;  // free pages of this block's part
    __shared__ int part_wide;  // slots of its part that do not fit the table
    __shared__ unsigned long long part_need;  // pages its slots take
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gt = blockIdx.x * kPlanThreads + tid;
    const int gn = kPlanCtas * kPlanThreads;
    constexpr int NW = kPlanThreads / 32;
    // the finish grid (a programmatic dependent launch) may be scheduled now
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    // 1. clear the per-page workspace
    for (int p = gt; p < a.P; p += gn) {
        a.was[p] = 0;
        a.full[p] = 0;
        a.held[p] = 0;
        a.claim[p] = ~0ull;
    }
    if (gt == 0) a.count[0] = 0;
    if (tid == 0) {
        part_free = 0;
        part_wide = 0;
        part_need = 0;
    }
    const int per_s = (int)(((long long)a.N + kPlanCtas - 1) / kPlanCtas);
    const int s0 = (int)min((long long)blockIdx.x * per_s, (long long)a.N), s1 = min(s0 + per_s, a.N);
    Slot mine;  // the warp's first slot, kept over the phases
    mine.parent = -1;
    mine.len = mine.nfull = 0;
    mine.want = 0;
    if (s0 + warp < s1) mine = slot_of(a, s0 + warp);
    auto slot = [&](int i) -> Slot { return i == s0 + warp ? mine : slot_of(a, i); };
    // (a cluster barrier orders what the blocks write, in global memory too)
    cluster.sync();
    // 2. references by the old table; full entries and claims of the new one; free
    // pages of each part
    for_entries(a.table, gt, (long long)a.S * a.M, gn, [&](long long, int c) {
        if (c >= 0 && c < a.P) atomicAdd(a.was + c, 1);
    });
    for (int i = s0 + warp; i < s1; i += NW) {
        const Slot s = slot(i);
        if (s.parent < 0) continue;
        if (lane == 0 && s.want > a.M) atomicAdd(&part_wide, 1);
        for_entries(a.table + (long long)s.parent * a.M, lane, min(s.want, (long long)a.M), 32, [&](long long j, int c) {
            if (c < 0 || c >= a.P) return;
            if (j < s.nfull) atomicAdd(a.full + c, 1);
            else atomicMin(a.claim + c, (unsigned long long)i * a.M + j);
        });
    }
    const int per_p = (a.P + kPlanCtas - 1) / kPlanCtas;
    const int p0 = (int)min((long long)blockIdx.x * per_p, (long long)a.P);
    const int p1 = (int)min((long long)p0 + per_p, (long long)a.P);
    int nfree = 0;
    for (int p = p0 + tid; p < p1; p += kPlanThreads) nfree += __ldg(a.refs + p) == 0;
    nfree = __reduce_add_sync(0xffffffffu, nfree);
    if (lane == 0 && nfree) atomicAdd(&part_free, nfree);
    cluster.sync();
    // 3. how many pages each slot takes; the free pages in ascending order
    for (int i = s0 + warp; i < s1; i += NW) {
        const Slot s = slot(i);
        const int last = s.parent < 0 ? 0 : (int)min(s.want, (long long)a.M);
        int cnt = 0;
        for (int j = s.nfull + lane; j < last; j += 32) cnt += !keeps(a, i, j, cand_of(a, s, j));
        cnt = __reduce_add_sync(0xffffffffu, cnt);
        if (lane == 0) {
            a.need[i] = cnt;
            if (cnt) atomicAdd(&part_need, (unsigned long long)cnt);
        }
    }
    int free_before = 0, all_free = 0, wide = 0;
#pragma unroll
    for (int r = 0; r < kPlanCtas; ++r) {
        const int f = *cluster.map_shared_rank(&part_free, r);
        if (r < (int)blockIdx.x) free_before += f;
        all_free += f;
        wide += *cluster.map_shared_rank(&part_wide, r);
    }
    for (long long q = p0; q < p1; q += 8 * kPlanThreads) {  // eight pages a thread
        const long long p = q + 8 * tid;
        unsigned f = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (p + k < p1 && __ldg(a.refs + p + k) == 0) f |= 1u << k;
        int tot;
        int at = free_before + block_scan(__popc(f), warps, &tot);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if ((f >> k) & 1u) a.list[at++] = (int)(p + k);
        free_before += tot;
    }
    cluster.sync();
    // 4. entries that need a page take the free ones in the order of slots and
    // entries, when there are enough
    unsigned long long before = 0, total = 0;
#pragma unroll
    for (int r = 0; r < kPlanCtas; ++r) {
        const unsigned long long x = *cluster.map_shared_rank(&part_need, r);
        if (r < (int)blockIdx.x) before += x;
        total += x;
    }
    const long long missing = (long long)total - all_free;
    const bool fine = missing <= 0 && wide == 0;
    if (gt == 0) {
        a.status[0] = missing > 0 ? (int)min(missing, (long long)INT_MAX) : 0;
        a.status[1] = wide;
        a.status[2] = fine ? (int)total : 0;
        if (!fine) a.status[3] = 0;
    }
    if (fine) {
        int taken = (int)before;
        for (int i0 = s0; i0 < s1; i0 += NW) {
            const int i = i0 + warp;
            Slot s;
            s.parent = -1;
            s.nfull = s.len = 0;
            s.want = 0;
            if (i < s1) s = slot(i);
            const int last = s.parent < 0 ? 0 : (int)min(s.want, (long long)a.M);
            int tot;
            int at = block_scan(lane == 0 && i < s1 ? __ldcg(a.need + i) : 0, warps, &tot);
            at = taken + __shfl_sync(0xffffffffu, at, 0);
            taken += tot;
            for (int j0 = s.nfull; j0 < last; j0 += 32) {
                const int j = j0 + lane;
                int c = -1;
                bool get = false;
                if (j < last) {
                    c = cand_of(a, s, j);
                    get = !keeps(a, i, j, c);
                }
                const unsigned m = __ballot_sync(0xffffffffu, get);
                int pg = c;
                if (get) pg = __ldcg(a.list + at + __popc(m & ((1u << lane) - 1u)));
                at += __popc(m);
                if (j < last) {
                    a.table_out[(long long)i * a.M + j] = pg;
                    a.held[pg] = 1;
                    if (get && c >= 0 && c < a.P && j == s.nfull && (s.len & ((1 << a.page_shift) - 1))) {
                        const int k = atomicAdd(a.count, 1);
                        a.src[k] = c;
                        a.dst[k] = pg;
                    }
                }
            }
        }
    }
    cluster.sync();  // (every part's sums are read, and every copy is counted)
    if (gt == 0 && fine) a.status[3] = __ldcg(a.count);
}

// The new version's remaining entries, lengths and counts, and the page copies.
__global__ void __launch_bounds__(kCopyThreads)
    fork_finish_kernel(const __grid_constant__ ForkArgs a, const __grid_constant__ PoolTable t) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const bool fine = __ldcg(a.status) == 0 && __ldcg(a.status + 1) == 0;
    const long long gt = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long gn = (long long)gridDim.x * blockDim.x;
    for (long long p = gt; p < a.P; p += gn) {
        const int r = __ldg(a.refs + p);
        a.refs_out[p] = fine ? r - __ldcg(a.was + p) + __ldcg(a.full + p) + __ldcg(a.held + p) : r;
    }
    const int lane = threadIdx.x & 31;
    for (long long i = gt >> 5; i < a.N; i += gn >> 5) {
        const Slot s = slot_of(a, (int)i);
        if (lane == 0) a.lens_out[i] = fine ? s.len : 0;
        const int last = fine ? (int)min(s.want, (long long)a.M) : 0;
        for (int j = lane; j < a.M; j += 32) {
            int v = -1;
            if (fine && j < s.nfull) {
                const int c = cand_of(a, s, j);
                v = c >= 0 && c < a.P ? c : -1;
            } else if (j < last) {
                continue;  // the plan wrote it
            }
            a.table_out[i * a.M + j] = v;
        }
    }
    if (t.n > 0) copy_pages(t, a.src, a.dst, __ldcg(a.count), a.P, a.P);
}

// The whole of a small fork by one cluster.  The per-page counts live in the shared
// memory of the block that has the page's part (parts of 2^part_shift pages), the
// free pages of a part in a list of its own, and each block copies the pages of
// its own slots.
struct SmallFork {
    ForkArgs a;
    int part_shift;
};

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    fork_small_kernel(const __grid_constant__ SmallFork sf, const __grid_constant__ PoolTable t) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ int warps[32];
    __shared__ int part_free, part_wide, part_copies;
    __shared__ unsigned long long part_need;
    const ForkArgs &a = sf.a;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gt = blockIdx.x * kPlanThreads + tid;
    const int gn = kPlanCtas * kPlanThreads;
    constexpr int NW = kPlanThreads / 32;
    const int per_p = 1 << sf.part_shift, pmask = per_p - 1;
    const int per_s = (a.N + kPlanCtas - 1) / kPlanCtas;
    // (entries are numbered in 32 bits here: the 64-bit minimum on another block's
    // shared memory was seen to lose updates; the cause was not found)
    int2 *moves = reinterpret_cast<int2 *>(dyn);                   // [per_s] pages to copy
    unsigned *claim = reinterpret_cast<unsigned *>(moves + per_s);  // [per_p]
    int *was = reinterpret_cast<int *>(claim + per_p), *full = was + per_p, *held = full + per_p;
    int *list = held + per_p;                   // [per_p] free pages of the part
    int *need = list + per_p;                   // [per_s]
    // page c's entry of an array
    auto of = [&](auto *arr, int c) { return cluster.map_shared_rank(arr, c >> sf.part_shift) + (c & pmask); };
    auto keep = [&](int i, int j, int c) -> bool {
        if (c < 0 || c >= a.P) return false;
        const int refs = __ldg(a.refs + c);
        return refs > 0 && *of(full, c) == 0 && refs <= *of(was, c) &&
               *of(claim, c) == (unsigned)(i * a.M + j);
    };
    // the copy grid (a programmatic dependent launch) may be scheduled now
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int p0 = min(blockIdx.x << sf.part_shift, (unsigned)a.P), p1 = min(p0 + per_p, a.P);
    const int s0 = min((int)blockIdx.x * per_s, a.N), s1 = min(s0 + per_s, a.N);
    // 1. clear; the free pages of the part, in ascending order
    for (int p = tid; p < per_p; p += kPlanThreads) {
        was[p] = 0;
        full[p] = 0;
        held[p] = 0;
        claim[p] = ~0u;
    }
    if (tid == 0) {
        part_wide = 0;
        part_copies = 0;
        part_need = 0;
    }
    int nf = 0;
    for (int q = p0; q < p1; q += kPlanThreads) {
        const int p = q + tid;
        const int f = p < p1 && __ldg(a.refs + p) == 0;
        int tot;
        const int at = nf + block_scan(f, warps, &tot);
        if (f) list[at] = p;
        nf += tot;
    }
    if (tid == 0) part_free = nf;
    Slot mine;  // the warp's first slot, kept over the phases
    mine.parent = -1;
    mine.len = mine.nfull = 0;
    mine.want = 0;
    if (s0 + warp < s1) mine = slot_of(a, s0 + warp);
    auto slot = [&](int i) -> Slot { return i == s0 + warp ? mine : slot_of(a, i); };
    cluster.sync();
    // 2. references by the old table; full entries and claims of the new one
    for_entries(a.table, gt, (long long)a.S * a.M, gn, [&](long long, int c) {
        if (c >= 0 && c < a.P) atomicAdd(of(was, c), 1);
    });
    for (int i = s0 + warp; i < s1; i += NW) {
        const Slot s = slot(i);
        if (lane == 0) a.lens_out[i] = s.len;
        if (s.parent < 0) continue;
        if (lane == 0 && s.want > a.M) atomicAdd(&part_wide, 1);
        for_entries(a.table + (long long)s.parent * a.M, lane, min(s.want, (long long)a.M), 32, [&](long long j, int c) {
            if (c < 0 || c >= a.P) return;
            if (j < s.nfull) atomicAdd(of(full, c), 1);
            else atomicMin(of(claim, c), (unsigned)(i * a.M + (int)j));
        });
    }
    cluster.sync();
    // 3. how many pages each slot takes
    for (int i = s0 + warp; i < s1; i += NW) {
        const Slot s = slot(i);
        const int last = s.parent < 0 ? 0 : (int)min(s.want, (long long)a.M);
        int cnt = 0;
        for (int j = s.nfull + lane; j < last; j += 32) cnt += !keep(i, j, cand_of(a, s, j));
        cnt = __reduce_add_sync(0xffffffffu, cnt);
        if (lane == 0) {
            need[i - s0] = cnt;
            if (cnt) atomicAdd(&part_need, (unsigned long long)cnt);
        }
    }
    cluster.sync();
    // 4. entries that need a page take the free ones in the order of slots and entries
    unsigned long long before = 0, total = 0;
    int wide = 0, free_end[kPlanCtas], all_free = 0;
#pragma unroll
    for (int r = 0; r < kPlanCtas; ++r) {
        const unsigned long long x = *cluster.map_shared_rank(&part_need, r);
        if (r < (int)blockIdx.x) before += x;
        total += x;
        wide += *cluster.map_shared_rank(&part_wide, r);
        all_free += *cluster.map_shared_rank(&part_free, r);
        free_end[r] = all_free;
    }
    auto free_page = [&](int k) -> int {  // the k-th free page
        int r = 0, first = 0;
#pragma unroll
        for (int x = 0; x < kPlanCtas - 1; ++x)
            if (k >= free_end[x]) {
                r = x + 1;
                first = free_end[x];
            }
        return cluster.map_shared_rank(list, r)[k - first];
    };
    const long long missing = (long long)total - all_free;
    const bool fine = missing <= 0 && wide == 0;
    if (gt == 0) {
        a.status[0] = missing > 0 ? (int)min(missing, (long long)INT_MAX) : 0;
        a.status[1] = wide;
        a.status[2] = fine ? (int)total : 0;
    }
    int taken = (int)before;
    for (int i0 = s0; i0 < s1; i0 += NW) {
        const int i = i0 + warp;
        Slot s;
        s.parent = -1;
        s.nfull = s.len = 0;
        s.want = 0;
        if (i < s1 && fine) s = slot(i);
        const int last = s.parent < 0 ? 0 : (int)min(s.want, (long long)a.M);
        int tot;
        int at = block_scan(lane == 0 && i < s1 ? need[i - s0] : 0, warps, &tot);
        at = taken + __shfl_sync(0xffffffffu, at, 0);
        taken += tot;
        if (i >= s1) continue;
        if (!fine && lane == 0) a.lens_out[i] = 0;
        for (int j0 = 0; j0 < a.M; j0 += 32) {
            const int j = j0 + lane;
            const int c = j < last ? cand_of(a, s, j) : -1;
            const bool get = j < last && j >= s.nfull && !keep(i, j, c);
            const unsigned m = __ballot_sync(0xffffffffu, get);
            int pg = c >= 0 && c < a.P ? c : -1;
            if (get) pg = free_page(at + __popc(m & ((1u << lane) - 1u)));
            at += __popc(m);
            if (j < a.M) a.table_out[(long long)i * a.M + j] = pg;
            if (j < last && j >= s.nfull) *of(held, pg) = 1;
            if (get && c >= 0 && c < a.P && j == s.nfull && (s.len & ((1 << a.page_shift) - 1)))
                moves[atomicAdd(&part_copies, 1)] = make_int2(c, pg);
        }
    }
    cluster.sync();
    // 5. the counts of the part's pages, and the block's copies
    for (int p = p0 + tid; p < p1; p += kPlanThreads) {
        const int r = __ldg(a.refs + p), k = p - p0;
        a.refs_out[p] = fine ? r - was[k] + full[k] + held[k] : r;
    }
    if (gt == 0) {
        int copies = 0;
#pragma unroll
        for (int r = 0; r < kPlanCtas; ++r) copies += *cluster.map_shared_rank(&part_copies, r);
        a.status[3] = copies;
    }
    if (t.n > 0) copy_pairs(t, part_copies, a.P, a.P, warp, NW, [&](int i) { return moves[i]; });
    cluster.sync();  // every block's sums are read before it exits
}

// The copies of a fork whose plan kept no list: slot i's partly filled page, where
// its entry is not its parent's.  Every block lists the pairs (kSlotsMax at most),
// in slot order, in shared memory first.
constexpr int kSlotsMax = 2048;

__global__ void __launch_bounds__(kCopyThreads)
    fork_copy_kernel(const __grid_constant__ ForkArgs a, const __grid_constant__ PoolTable t) {
    __shared__ int2 moves[kSlotsMax];
    __shared__ int warps[32];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (__ldcg(a.status + 3) == 0) return;  // (0 as well where the call did not fit)
    int count = 0;
    for (int i0 = 0; i0 < a.N; i0 += kCopyThreads) {
        const int i = i0 + threadIdx.x;
        int2 m = make_int2(-1, -1);
        if (i < a.N) {
            const Slot s = slot_of(a, i);
            if (s.parent >= 0 && s.nfull < a.M && (s.len & ((1 << a.page_shift) - 1)) != 0) {
                const int c = cand_of(a, s, s.nfull), d = __ldcg(a.table_out + (long long)i * a.M + s.nfull);
                if (c >= 0 && c < a.P && c != d) m = make_int2(c, d);
            }
        }
        int tot;
        const int at = count + block_scan<kCopyThreads / 32>(m.x >= 0, warps, &tot);
        if (m.x >= 0) moves[at] = m;
        count += tot;
    }
    __syncthreads();
    constexpr int W = kCopyThreads / 32;
    copy_pairs(t, count, a.P, a.P, (long long)blockIdx.x * W + (threadIdx.x >> 5), (long long)gridDim.x * W,
               [&](int i) { return moves[i]; });
}

// ------------------------------------------------------------------ compact

struct CompactArgs {
    const int32_t *table, *refs;
    int S, M, P;
    int32_t *table_out, *refs_out, *remap, *n_live;
    int32_t *src, *dst;  // pages to move (src from the back) and the holes they fill
    int32_t *count;      // [0] pages to move
};

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const __grid_constant__ CompactArgs a) {
    // the finish grid (a programmatic dependent launch) may be scheduled now
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    __shared__ int warps[32];
    __shared__ int mine;  // live pages of this block's part
    cg::cluster_group cluster = cg::this_cluster();
    const int per = (a.P + kPlanCtas - 1) / kPlanCtas;
    const int p0 = min(blockIdx.x * per, (unsigned)a.P), p1 = min(p0 + per, a.P);
    int cnt = 0;
    for (int p = p0 + threadIdx.x; p < p1; p += kPlanThreads) cnt += __ldg(a.refs + p) > 0;
    int tot;
    block_scan(cnt, warps, &tot);
    if (threadIdx.x == 0) mine = tot;
    cluster.sync();
    int before = 0, n = 0;
#pragma unroll
    for (int r = 0; r < kPlanCtas; ++r) {
        const int c = *cluster.map_shared_rank(&mine, r);
        if (r < (int)blockIdx.x) before += c;
        n += c;
    }
    // Holes (free pages before n) take the live pages at or behind n, both in
    // ascending order.  A hole's rank is its index less the live pages before
    // it; a mover's is counted from the back (n - 1 less the live pages before
    // it), so that one scan ranks both.
    int live_before = before;
    for (int q0 = p0; q0 < p1; q0 += kPlanThreads) {
        const int p = q0 + threadIdx.x;
        const bool in = p < p1;
        const int r = in ? __ldg(a.refs + p) : 0;
        const int live = r > 0;
        const int at = live_before + block_scan(live, warps, &tot);
        if (in) {
            if (p == n) a.count[0] = n - at;  // pages to move
            if (live && p >= n) a.src[n - 1 - at] = p;
            if (!live && p < n) a.dst[p - at] = p;
            // (a mover's number and a hole's count follow below)
            if (!live || p < n) a.remap[p] = live ? p : -1;
            if (live || p >= n) a.refs_out[p] = p < n ? r : 0;
        }
        live_before += tot;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.n_live = n;
        if (n == a.P) a.count[0] = 0;  // no hole
    }
    cluster.sync();  // (also: every block has read `mine` before any leaves)
    const int moves = __ldcg(a.count);
    for (int k = blockIdx.x * kPlanThreads + threadIdx.x; k < moves; k += kPlanCtas * kPlanThreads) {
        const int d = __ldcg(a.dst + k), s = __ldcg(a.src + moves - 1 - k);
        a.remap[s] = d;
        a.refs_out[d] = __ldg(a.refs + s);
    }
}

// The whole of a small compaction by one cluster: a block has a part of the pages,
// lists the live ones at or behind the live count (movers) and fills the holes
// before it from the parts' lists, in ascending order both.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    compact_small_kernel(const __grid_constant__ CompactArgs a, const __grid_constant__ PoolTable t) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ int warps[32];
    __shared__ int part_live, part_movers, part_holes;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5;
    const int per = (a.P + kPlanCtas - 1) / kPlanCtas;
    const int p0 = min((int)blockIdx.x * per, a.P), p1 = min(p0 + per, a.P);
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    int2 *moves = reinterpret_cast<int2 *>(dyn);       // [per] {page, hole}: the holes of this part
    int *movers = reinterpret_cast<int *>(moves + per);  // [per]
    int cnt = 0;
    for (int p = p0 + tid; p < p1; p += kPlanThreads) cnt += __ldg(a.refs + p) > 0;
    int tot;
    block_scan(cnt, warps, &tot);
    if (tid == 0) part_live = tot;
    cluster.sync();
    int n = 0;
#pragma unroll
    for (int r = 0; r < kPlanCtas; ++r) n += *cluster.map_shared_rank(&part_live, r);
    int nm = 0, nh = 0;
    for (int q = p0; q < p1; q += kPlanThreads) {
        const int p = q + tid;
        const int r = p < p1 ? __ldg(a.refs + p) : 0;
        const int mover = p < p1 && r > 0 && p >= n, hole = p < p1 && r <= 0 && p < n;
        const int at_m = nm + block_scan(mover, warps, &tot);
        nm += tot;
        const int at_h = nh + block_scan(hole, warps, &tot);
        nh += tot;
        if (mover) movers[at_m] = p;
        if (hole) moves[at_h].y = p;
        if (p < p1) {
            // (a mover's number and a hole's count follow below)
            if (!mover) a.remap[p] = r > 0 ? p : -1;
            if (!hole) a.refs_out[p] = p < n ? r : 0;
        }
    }
    if (tid == 0) {
        part_movers = nm;
        part_holes = nh;
        if (blockIdx.x == 0) *a.n_live = n;
    }
    cluster.sync();
    int before = 0, end[kPlanCtas], holes_end[kPlanCtas], sum = 0, holes = 0;
#pragma unroll
    for (int r = 0; r < kPlanCtas; ++r) {
        if (r == (int)blockIdx.x) before = holes;
        holes += *cluster.map_shared_rank(&part_holes, r);
        sum += *cluster.map_shared_rank(&part_movers, r);
        holes_end[r] = holes;
        end[r] = sum;
    }
    for (int k = tid; k < nh; k += kPlanThreads) {
        int r = 0, first = 0;
#pragma unroll
        for (int x = 0; x < kPlanCtas - 1; ++x)
            if (before + k >= end[x]) {
                r = x + 1;
                first = end[x];
            }
        const int p = cluster.map_shared_rank(movers, r)[before + k - first], d = moves[k].y;
        moves[k].x = p;
        a.remap[p] = d;
        a.refs_out[d] = __ldg(a.refs + p);
    }
    cluster.sync();
    for (long long e = blockIdx.x * kPlanThreads + tid; e < (long long)a.S * a.M; e += kPlanCtas * kPlanThreads) {
        const int c = __ldg(a.table + e);
        a.table_out[e] = c >= 0 && c < a.P ? __ldcg(a.remap + c) : -1;
    }
    // (the holes lie in the first parts: the copies are spread over all blocks)
    if (t.n > 0)
        copy_pairs(t, holes_end[kPlanCtas - 1], a.P, a.P, blockIdx.x * (kPlanThreads / 32) + warp,
                   kPlanCtas * (kPlanThreads / 32), [&](int i) {
            int r = 0, first = 0;
#pragma unroll
            for (int x = 0; x < kPlanCtas - 1; ++x)
                if (i >= holes_end[x]) {
                    r = x + 1;
                    first = holes_end[x];
                }
            return cluster.map_shared_rank(moves, r)[i - first];
        });
    cluster.sync();  // every block's lists are read before it exits
}

// The copies of a compaction whose plan kept no list: page p at or behind the live
// count goes to remap[p].
__global__ void __launch_bounds__(kCopyThreads)
    compact_copy_kernel(const __grid_constant__ CompactArgs a, const __grid_constant__ PoolTable t) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int n = __ldcg(a.n_live), warps = kCopyThreads / 32;
    copy_pairs(t, a.P - n, a.P, a.P, (long long)blockIdx.x * warps + (threadIdx.x >> 5), (long long)gridDim.x * warps,
               [&](int i) { return make_int2(n + i, __ldcg(a.remap + n + i)); });
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_finish_kernel(const __grid_constant__ CompactArgs a, const __grid_constant__ PoolTable t) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const long long gt = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long gn = (long long)gridDim.x * blockDim.x;
    for (long long e = gt; e < (long long)a.S * a.M; e += gn) {
        const int c = __ldg(a.table + e);
        a.table_out[e] = c >= 0 && c < a.P ? __ldcg(a.remap + c) : -1;
    }
    if (t.n > 0) copy_pages(t, a.src, a.dst, __ldcg(a.count), a.P, a.P, true);
}

// --------------------------------------------------------------------- host

// 0, or 2 when a page has more chunks than the index holds.
int fill_pools(PoolTable &t, const void *const *src, void *const *dst, const long long *bytes,
               int n) {
    long long chunks = 0;
    t.n = n;
    for (int i = 0; i < n; ++i) {
        t.src[i] = static_cast<const uint8_t *>(src[i]);
        t.dst[i] = static_cast<uint8_t *>(dst[i]);
        t.bytes[i] = bytes[i];
        t.first_chunk[i] = (int)chunks;
        chunks += (bytes[i] + kChunk - 1) / kChunk;
        if (chunks >= (1LL << 30)) {
            set_error("pages: a page of more than 2^30 chunks");
            return 2;
        }
    }
    t.first_chunk[n] = (int)chunks;
    return 0;
}

// Blocks for `chunks` warps' worth of copies beside `other` threads' worth of
// table work: four blocks an SM at most.
unsigned grid_for(long long chunks, long long other) {
    int dev = 0;
    cudaGetDevice(&dev);
    const int nsm = sm_count(dev);
    const long long most = 4LL * (nsm < 1 ? 1 : nsm);
    long long want = (chunks + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    const long long w2 = (other + kCopyThreads - 1) / kCopyThreads;
    want = want > w2 ? want : w2;
    return (unsigned)(want < 1 ? 1 : want > most ? most : want);
}

int launched(const char *what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s launch: %s", what, cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

// A finish kernel as the programmatic dependent of its plan.
template <typename A>
int launch_finish(void (*kern)(A, PoolTable), unsigned blocks, const A &a, const PoolTable &t, const char *what,
                  cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, t);
    if (e != cudaSuccess) {
        set_error("%s launch: %s", what, cudaGetErrorString(e));
        return 3;
    }
    return launched(what);
}

// The pools past the first kMaxPools, in launches of their own.
template <typename F> int for_pool_groups(const void *const *src, void *const *dst, const long long *bytes, int n, F f) {
    int rc = 0;
    int at = 0;
    do {
        PoolTable t;
        const int m = n - at < kMaxPools ? n - at : kMaxPools;
        rc = fill_pools(t, src + at, dst + at, bytes + at, m);
        if (rc == 0) rc = f(t, at == 0);
        at += m;
    } while (rc == 0 && at < n);
    return rc;
}


// What a cluster moves by itself: 8 SMs copy about 1 TB/s, so up to here the second
// launch costs more than it saves.
constexpr long long kSmallBytes = 4LL << 20;
constexpr int kSmallShared = 200 * 1024;  // dynamic shared memory a block

template <typename A>
int launch_small(void (*kern)(A, PoolTable), const A &a, const PoolTable &t, size_t smem, const char *what,
                 cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
        set_error("%s: cudaFuncSetAttribute: %s", what, cudaGetErrorString(e));
        return 3;
    }
    kern<<<kPlanCtas, kPlanThreads, smem, stream>>>(a, t);
    return launched(what);
}

long long page_total(const long long *bytes, int n) {
    long long x = 0;
    for (int i = 0; i < n; ++i) x += bytes[i];
    return x;
}

// log2 of the pages of a block's part, and the shared memory that a small fork
// takes.
int fork_part_shift(int P) {
    int k = 0;
    while ((8LL << k) < P) ++k;
    return k;
}
size_t fork_small_shared(int N, int P) {
    const size_t per_s = (N + kPlanCtas - 1) / kPlanCtas;
    return ((size_t)20 << fork_part_shift(P)) + per_s * 12;
}
size_t compact_small_shared(int P) { return (size_t)((P + kPlanCtas - 1) / kPlanCtas) * 12; }

constexpr long long kSmallEntries = 1 << 17;  // of a table

// Bytes from which on a plan with lists in a workspace is worth its allocation (4 us
// of host time): a copy launch that looks the pairs up is slower by 7 to 11%.  Of the
// GPU's time, with lists and without: a fork of 32 x 8 candidates of up to 8192 keys
// 42.8 and 47.6 us, a compaction of 4096 pages, half of them holes, 183.1 and 196.2 us
// (4 layers of K and V each).
constexpr double kListBytes = 64.0 * (1 << 20);

// Whether a plan goes without a workspace: its counts fit the cluster's shared
// memory, its table is not so large that a whole grid has to write it, and not
// much can move; and whether the cluster copies as well.
bool fork_fits(const long long *bytes, int npools, int N, int M, int P) {
    return (long long)N * M <= kSmallEntries && N <= kSlotsMax && P <= (1 << 20) &&
           fork_small_shared(N, P) <= kSmallShared && (double)N * page_total(bytes, npools) <= kListBytes;
}
bool fork_copies(const long long *bytes, int npools, int N) {
    return npools <= kMaxPools && (double)N * page_total(bytes, npools) <= kSmallBytes;
}
bool compact_fits(const long long *bytes, int npools, int S, int M, int P) {
    return (long long)S * M <= kSmallEntries && P <= (1 << 20) && compact_small_shared(P) <= kSmallShared &&
           0.5 * P * page_total(bytes, npools) <= kListBytes;
}
bool compact_copies(const long long *bytes, int npools, int P) {  // (at most half of the pages move)
    return npools <= kMaxPools && 0.5 * P * page_total(bytes, npools) <= kSmallBytes;
}

}  // namespace

int launch_pages_copy(const void *const *src_pools, void *const *dst_pools, const long long *bytes,
                      int npools, int src_pages, int dst_pages, const int32_t *src,
                      const int32_t *dst, int n, cudaStream_t stream) {
    return for_pool_groups(src_pools, dst_pools, bytes, npools, [&](const PoolTable &t, bool) {
        const long long chunks = (long long)n * t.first_chunk[t.n];
        if (chunks == 0) return 0;
        copy_pages_kernel<<<grid_for(chunks, 0), kCopyThreads, 0, stream>>>(t, src, dst, n, src_pages,
                                                                           dst_pages);
        return launched("page copy kernel");
    });
}

unsigned long long pages_fork_workspace(const long long *bytes, int npools, int N, int M, int P) {
    return fork_fits(bytes, npools, N, M, P) ? 0 : 8ull * P + 4ull * (4ull * P + 3ull * N + 1ull);
}

int launch_pages_fork(void *const *pools, const long long *bytes, int npools,
                      const int32_t *block_table, const int32_t *seqlens, const int32_t *refcount,
                      int S, int M, int P, int page_shift, const int32_t *parents,
                      const int32_t *new_tokens, int N, int32_t *table_out, int32_t *seqlens_out,
                      int32_t *refcount_out, int32_t *status, void *ws, cudaStream_t stream) {
    ForkArgs a = {};
    a.table = block_table;
    a.lens = seqlens;
    a.refs = refcount;
    a.parents = parents;
    a.grow = new_tokens;
    a.S = S;
    a.M = M;
    a.P = P;
    a.N = N;
    a.page_shift = page_shift;
    a.table_out = table_out;
    a.lens_out = seqlens_out;
    a.refs_out = refcount_out;
    a.status = status;
    if (fork_fits(bytes, npools, N, M, P)) {
        PoolTable none;
        none.n = 0;
        none.first_chunk[0] = 0;
        const bool all = fork_copies(bytes, npools, N);
        int rc = 0;
        if (all) rc = fill_pools(none, pools, pools, bytes, npools);
        if (rc == 0)
            rc = launch_small(fork_small_kernel, SmallFork{a, fork_part_shift(P)}, none, fork_small_shared(N, P),
                              "page fork kernel", stream);
        if (rc || all) return rc;
        return for_pool_groups(pools, pools, bytes, npools, [&](const PoolTable &t, bool first) {
            const unsigned blocks = grid_for((long long)N * t.first_chunk[t.n], 0);
            if (first) return launch_finish(fork_copy_kernel, blocks, a, t, "page copy kernel", stream);
            fork_copy_kernel<<<blocks, kCopyThreads, 0, stream>>>(a, t);
            return launched("page copy kernel");
        });
    }
    a.claim = static_cast<unsigned long long *>(ws);
    a.was = reinterpret_cast<int32_t *>(a.claim + P);
    a.full = a.was + P;
    a.held = a.full + P;
    a.list = a.held + P;
    a.need = a.list + P;
    a.src = a.need + N;
    a.dst = a.src + N;
    a.count = a.dst + N;
    fork_plan_kernel<<<kPlanCtas, kPlanThreads, 0, stream>>>(a);
    int rc = launched("page fork kernel");
    if (rc) return rc;
    return for_pool_groups(pools, pools, bytes, npools, [&](const PoolTable &t, bool first) {
        const long long chunks = (long long)N * t.first_chunk[t.n];
        if (!first) {
            copy_counted_kernel<<<grid_for(chunks, 0), kCopyThreads, 0, stream>>>(t, a.src, a.dst, a.count, P, false);
            return launched("page copy kernel");
        }
        const long long other = (long long)N * 32 > P ? (long long)N * 32 : P;
        return launch_finish(fork_finish_kernel, grid_for(chunks, other), a, t, "page fork kernel", stream);
    });
}

unsigned long long pages_compact_workspace(const long long *bytes, int npools, int S, int M, int P) {
    return compact_fits(bytes, npools, S, M, P) ? 0 : 4ull * (2ull * P + 1ull);
}

int launch_pages_compact(void *const *pools, const long long *bytes, int npools,
                         const int32_t *block_table, const int32_t *refcount, int S, int M, int P,
                         int32_t *table_out, int32_t *refcount_out, int32_t *remap,
                         int32_t *n_live, void *ws, cudaStream_t stream) {
    CompactArgs a = {};
    a.table = block_table;
    a.refs = refcount;
    a.S = S;
    a.M = M;
    a.P = P;
    a.table_out = table_out;
    a.refs_out = refcount_out;
    a.remap = remap;
    a.n_live = n_live;
    if (compact_fits(bytes, npools, S, M, P)) {
        PoolTable none;
        none.n = 0;
        none.first_chunk[0] = 0;
        const bool all = compact_copies(bytes, npools, P);
        int rc = 0;
        if (all) rc = fill_pools(none, pools, pools, bytes, npools);
        if (rc == 0)
            rc = launch_small(compact_small_kernel, a, none, compact_small_shared(P), "page compact kernel", stream);
        if (rc || all) return rc;
        return for_pool_groups(pools, pools, bytes, npools, [&](const PoolTable &t, bool first) {
            const unsigned blocks = grid_for((long long)(P / 2) * t.first_chunk[t.n], 0);
            if (first) return launch_finish(compact_copy_kernel, blocks, a, t, "page copy kernel", stream);
            compact_copy_kernel<<<blocks, kCopyThreads, 0, stream>>>(a, t);
            return launched("page copy kernel");
        });
    }
    a.src = static_cast<int32_t *>(ws);
    a.dst = a.src + P;
    a.count = a.dst + P;
    compact_plan_kernel<<<kPlanCtas, kPlanThreads, 0, stream>>>(a);
    int rc = launched("page compact kernel");
    if (rc) return rc;
    return for_pool_groups(pools, pools, bytes, npools, [&](const PoolTable &t, bool first) {
        // at most half of the pages move
        const long long chunks = (long long)(P / 2) * t.first_chunk[t.n];
        if (!first) {
            copy_counted_kernel<<<grid_for(chunks, 0), kCopyThreads, 0, stream>>>(t, a.src, a.dst, a.count, P, true);
            return launched("page copy kernel");
        }
        return launch_finish(compact_finish_kernel, grid_for(chunks, (long long)S * M), a, t,
                             "page compact kernel", stream);
    });
}

}  // namespace attn
