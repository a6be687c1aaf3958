// kernel_rope_q8.cu -- the position rotation of new rows on their way into the 8-bit
// paged cache, and of the queries beside them, in one launch.
//
// What a block of tokens gets is what kernel_q8_append.cu writes (scale: the smallest
// power of two that holds the block's largest magnitude; earlier rows rounded again
// where it grows), for keys that are turned first (rope.cuh).  A turned key stays in
// fp32 until it is a code: rounding it to 16 bits in between would add up to half a
// 16-bit step to the half code step that is lost anyway.
//
// Bound: one read of the rows, one write of the codes and of the turned queries; the
// single-token call is launch latency.
//
// rope_q8_kernel: a unit is one block of one head of K or V by one or four warps, as in
// the append kernel; a thread keeps what it turned (64 floats, of single elements 16: eight
// items) between the maximum and the codes, and turns again (from L2) what is left over.
// The blocks behind the units turn the queries.
//
// rope_q8_stream_kernel, for many tokens in 16-byte vectors: a unit of 64 tokens is 16 KB and
// some 1000 instructions a warp behind a chain of three loads (length, page, rows), 5 us of
// latency that registers for 16 warps an SM do not hide.  So a block of threads stays with
// a block of tokens and walks its heads, the next ones' rows on their way into shared
// memory and the angles there once: 73 us where the units alone took 150 (16 x up to 4096
// tokens of 8 heads of 128).  That leaves the memory idle for the better part, and the
// queries (rope_stream.cuh), which use little but memory, run beside it: two blocks of each
// SM's three turn queries first (173 us together; with one of three 223, with all three
// 189, one kernel after the other 209).
#include "launch.h"
#include "q8_append.cuh"
#include "rope_stream.cuh"

namespace attn {
namespace {

using namespace sm100;

constexpr int kKeepFloats = 64;           // a thread keeps, in eight items at most
constexpr int kTileRows = 128;            // of a block of tokens, at most
constexpr int kTileBytes = 68 * 1024;     // of a block of threads: three an SM

struct RopeQ8Args {
    RopeArgs r;         // ko, vo: the pools of codes; q rows beside them
    float *scales[2];
    int nblk, blk_shift;
    int touch;          // blocks a sequence's new rows can touch
    int items_k, items_v;
    int stage;          // bytes of a stage of rows
    unsigned q_blocks;  // blocks in front that turn the queries
    StreamShape stream; // of these
    unsigned unit_blocks;
    RopeShape shape;    // of the queries' blocks
};

// VEC codes of values already divided by the scale.
template <int CODE, int VEC> __device__ __forceinline__ void put_codes(uint8_t *to, const float *y) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint2 *>(to) = make_uint2(code4<CODE>(y[0], y[1], y[2], y[3]),
                                                    code4<CODE>(y[4], y[5], y[6], y[7]));
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint32_t *>(to) = code4<CODE>(y[0], y[1], y[2], y[3]);
    } else {
        *to = CodeOps<CODE>::code(y[0]);
    }
}

// The largest of a, |b| and |c|; NaN if any is.
__device__ __forceinline__ float largest(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One block of head h of K or V (which: 0, 1), by TG threads: keep() turns its rows and
// finds the largest magnitude, put() writes their codes.
template <typename T, int CODE, int TG, int VEC, bool ADJ> struct RopeQ8Unit {
    using Op = CodeOps<CODE>;
    // items (32 single ones: 29 us become 47 in the case at launch_size)
    static constexpr int kKeep = kKeepFloats / (2 * VEC) < 8 ? kKeepFloats / (2 * VEC) : 8;
    struct Place {
        int r, c;
    };
    const RopeArgs &a;
    const RopeSeq &sq;
    const AppendSpan &span;
    int tid, rows, W, rot, per_row, lanes, rstep, r0, c0, pitch;
    float *sp;
    uint8_t *page_base;
    bool old_rows;
    float s_old;
    float y[kKeep][2 * VEC];

    __device__ __forceinline__ RopeQ8Unit(const RopeQ8Args &g, const RopeSeq &seq, const AppendSpan &sn, int page,
                                          int which, int h)
        : a(g.r), sq(seq), span(sn) {
        tid = threadIdx.x % TG;
        rows = (int)(span.last - span.first);
        W = which ? a.Dv : a.D;
        rot = which ? 0 : a.rot;
        sp = g.scales[which] + ((long long)page * g.nblk + span.sub) * a.Hkv + h;
        pitch = a.Hkv * W;
        page_base = static_cast<uint8_t *>(which ? a.vo : a.ko) +
                    (((long long)page << a.page_shift) * a.Hkv + h) * (long long)W;
        old_rows = span.start < sq.len;
        s_old = old_rows ? __ldcg(sp) : 0.f;
        // a thread's items: one column, or every lanes-th, of every rstep-th row
        per_row = which ? g.items_v : g.items_k;
        lanes = per_row < TG ? per_row : TG;
        rstep = TG / lanes;
        r0 = tid / lanes;
        c0 = tid - r0 * lanes;
    }
    __device__ __forceinline__ Place start() const { return {r0 < rstep ? r0 : rows, c0}; }
    __device__ __forceinline__ void next(Place &p) const {
        p.c += lanes;
        if (p.c >= per_row) {
            p.c = c0;
            p.r += rstep;
        }
    }
    // `src`, `stride`: the head's first new row; trig(row, pair, angles): its angles
    template <typename F>
    __device__ __forceinline__ void fetch(const Place &p, const T *src, long long stride, F trig,
                                          float (&to)[2 * VEC]) {
        const RopeItem<VEC> it = rope_item<VEC, ADJ>(p.c, rot);
        RowVec<T, VEC> x, w;
        x.load(src + p.r * stride + it.a);
        w.load(src + p.r * stride + it.b);
        Trig<VEC> tr;
        if (it.trig >= 0) trig(p.r, it.trig, tr);
        turn_item<T, VEC, ADJ>(it, x, w, tr, to);
    }
    template <typename F> __device__ __forceinline__ uint32_t keep(const T *src, long long stride, F trig) {
        float mx = 0.f;
        Place p = start();
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            if (p.r < rows) {
                fetch(p, src, stride, trig, y[k]);
            } else {
#pragma unroll
                for (int e = 0; e < 2 * VEC; ++e) y[k][e] = 0.f;
            }
            next(p);
        }
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
#pragma unroll
            for (int e = 0; e < 2 * VEC; e += 2) mx = largest(mx, y[k][e], y[k][e + 1]);
        for (; p.r < rows; next(p)) {
            float z[2 * VEC];
            fetch(p, src, stride, trig, z);
#pragma unroll
            for (int e = 0; e < 2 * VEC; e += 2) mx = largest(mx, z[e], z[e + 1]);
        }
        return __float_as_uint(mx) & 0x7fffffffu;
    }
    template <typename F> __device__ __forceinline__ void put(uint32_t mx, const T *src, long long stride, F trig) {
        const float nan = __int_as_float(0x7fc00000);
        float s = mx >= Bits<float>::kInf ? nan : append_scale(__uint_as_float(mx), CODE);
        if (old_rows) s = s_old != s_old || s != s ? nan : fmaxf(s_old, s);
        if (tid == 0 && !(old_rows && s == s_old)) *sp = s;
        // x / s: a multiplication where s is a power of two (always, unless the caller's
        // own scales are not); a NaN scale: codes 0
        const bool pow2 = (__float_as_uint(s) & 0x807fffffu) == 0u && s > 0.f && s < 1e38f;
        const float inv = pow2 ? 1.f / s : 0.f;
        uint8_t *dst = page_base + (long long)((int)span.first & ((1 << a.page_shift) - 1)) * pitch;
        auto codes = [&](const Place &at, float (&z)[2 * VEC]) {
            const RopeItem<VEC> it = rope_item<VEC, ADJ>(at.c, rot);
            if (pow2) {
#pragma unroll
                for (int e = 0; e < 2 * VEC; e += 2) mul_f2(z[e], z[e + 1], inv, inv, z[e], z[e + 1]);
            } else {
#pragma unroll
                for (int e = 0; e < 2 * VEC; ++e) z[e] = divided(z[e], s, Op::kMax);
            }
            uint8_t *to = dst + (long long)at.r * pitch;
            put_codes<CODE, VEC>(to + it.a, z);
            if (VEC > 1 || it.trig >= 0) put_codes<CODE, VEC>(to + it.b, z + VEC);
        };
        Place p = start();
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
            if (p.r < rows) codes(p, y[k]);
            next(p);
        }
        for (; p.r < rows; next(p)) {
            float z[2 * VEC];
            fetch(p, src, stride, trig, z);
            codes(p, z);
        }
        // earlier rows of a block whose scale has grown
        if (old_rows && !(s == s_old)) {
            const int from = (int)span.start;
            uint8_t *ob = page_base + (long long)(from & ((1 << a.page_shift) - 1)) * pitch;
            const int n_old = (sq.len - from) * W;
            const float ratio = __fdiv_rn(s_old, s);
            for (int i = tid; i < n_old; i += TG) {
                uint8_t *c = ob + (long long)(i / W) * pitch + i % W;
                float z = Op::one(*c) * ratio;
                z = fabsf(z) <= 3.402823466e38f ? z : 0.f;
                *c = Op::code(z);
            }
        }
    }
};

// What new rows block t of sequence ub gets, and its page: false where there is none.
__device__ __forceinline__ bool rope_q8_place(const RopeQ8Args &g, int t, uint32_t ub, RopeSeq &sq,
                                              AppendSpan &span, int &page) {
    const RopeArgs &a = g.r;
    if (t >= g.touch || ub >= (uint32_t)a.B) return false;
    const int b = (int)ub;
    sq = rope_seq(a, b);
    span = append_span(sq.len, sq.n, (long long)a.max_pages << a.page_shift, t, a.page_shift, g.blk_shift);
    if (span.last <= span.first) return false;
    page = __ldg(a.block_table + (long long)b * a.max_pages + span.entry);
    return page >= 0 && page < a.num_pages;
}

template <typename T, int CODE, int TG, int VEC, bool ADJ>
__global__ void __launch_bounds__(128) rope_q8_kernel(const __grid_constant__ RopeQ8Args g) {
    __shared__ uint32_t red[4];
    const RopeArgs &a = g.r;
    const uint32_t ub = blockIdx.y + blockIdx.z * gridDim.y;
    if (blockIdx.x >= g.unit_blocks) {
        RopeArgs q = a;
        q.ko = nullptr;
        q.v = nullptr;
        rope_rows<T, VEC, ADJ, false>(q, g.shape, blockIdx.x - g.unit_blocks, ub);
        return;
    }
    const uint32_t u = blockIdx.x * (128 / TG) + threadIdx.x / TG;
    const int which = (int)(u & 1u);
    const int t = (int)((u >> 1) / (uint32_t)a.Hkv), h = (int)((u >> 1) - (uint32_t)t * (uint32_t)a.Hkv);
    RopeSeq sq;
    AppendSpan span;
    int page;
    if (!rope_q8_place(g, t, ub, sq, span, page)) return;
    RopeQ8Unit<T, CODE, TG, VEC, ADJ> unit(g, sq, span, page, which, h);
    const long long stride = which ? a.v_stride : a.k_stride;
    const int i0 = (int)span.first - sq.len;  // of the sequence's new rows
    const T *src = static_cast<const T *>(which ? a.v : a.k) + (sq.row0 + i0) * stride + (long long)h * unit.W;
    auto trig = [&](int r, int pair, Trig<VEC> &tr) { tr.load(a, rope_position(a, sq, i0 + r), pair); };
    const uint32_t mx = group_max<TG>(unit.keep(src, stride, trig), red);
    unit.put(mx, src, stride, trig);
}

// The same by blocks that stay with a block of tokens: all heads of K, or of V, one after
// the other (four at a time where TG is 32).
template <typename T, int CODE, int TG, int VEC, bool ADJ>
__global__ void __launch_bounds__(128, 3) rope_q8_stream_kernel(const __grid_constant__ RopeQ8Args g) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t red[8];  // (of two units in turn)
    __shared__ alignas(8) uint64_t full[3];  // of the two stages, and of the angles
    __shared__ int pos[kTileRows];
    __shared__ StreamToken token[4][kStreamMost][32];
    __shared__ alignas(8) uint64_t q_full[4][kStreamMost];
    constexpr int kHeads = 128 / TG;
    const RopeArgs &a = g.r;
    if (blockIdx.x < g.q_blocks) {
        RopeArgs q = a;
        q.k = q.v = nullptr;
        q.ko = q.vo = nullptr;
        rope_stream<T, VEC, ADJ, false>(q, g.stream, smem, token, q_full, blockIdx.x, g.q_blocks);
        return;
    }
    const uint32_t u = (blockIdx.x - g.q_blocks) >> 1, ub = u / (uint32_t)g.touch;
    const int t = (int)(u - ub * g.touch), which = (int)((blockIdx.x - g.q_blocks) & 1u), lane = threadIdx.x & 31;
    RopeSeq sq;
    AppendSpan span;
    int page;
    if (!rope_q8_place(g, t, ub, sq, span, page)) return;
    const int rows = (int)(span.last - span.first), i0 = (int)span.first - sq.len;
    const int W = which ? a.Dv : a.D, half = which ? 0 : a.rot >> 1;
    const uint32_t sbase = smem_addr(smem);
    auto bar = [&](int s) { return smem_addr(full + s); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < 3; ++s) mbar_init(bar(s), 128);
        fence_mbar_init();
    }
    __syncthreads();
    const int count = (a.Hkv + kHeads - 1) / kHeads;
    const long long stride = which ? a.v_stride : a.k_stride;
    const T *src = static_cast<const T *>(which ? a.v : a.k) + (sq.row0 + i0) * stride;
    // a thread brings in row r0 (the warps share them: a copy's issue is some 40 cycles)
    const int r0 = (lane << 2) + (threadIdx.x >> 5);
    auto load = [&](int n) {  // heads n * kHeads .. of all rows
        const int heads = min(kHeads, a.Hkv - n * kHeads), bytes = heads * W * (int)sizeof(T);
        mbar_arrive_expect_tx(bar(n & 1), r0 < rows ? (uint32_t)bytes : 0u);
        if (r0 < rows)
            bulk_load(sbase + (n & 1) * g.stage + r0 * bytes, src + r0 * stride + (long long)n * kHeads * W, bytes,
                      bar(n & 1));
    };
    load(0);
    if (half > 0) {
        int p = -1;
        if (r0 < rows) pos[r0] = p = rope_position(a, sq, i0 + r0);
        mbar_arrive_expect_tx(bar(2), p >= 0 ? half * 8 : 0);
        if (p >= 0) {
            const uint32_t at = sbase + 2 * g.stage + r0 * half * 8;
            bulk_load(at, a.cos + (long long)p * half, half * 4, bar(2));
            bulk_load(at + half * 4, a.sin + (long long)p * half, half * 4, bar(2));
        }
    }
    if (count > 1) load(1);
    __syncthreads();  // pos
    const float *angles = reinterpret_cast<const float *>(smem + 2 * g.stage);
    auto trig = [&](int r, int pair, Trig<VEC> &tr) {
        const float *c = angles + r * half * 2 + pair;
        if (pos[r] >= 0) tr.load_from(c, c + half, 1.f);
        else tr.set_nan();
    };
    bool ok = half == 0 || mbar_wait_within(bar(2), 0, a.wait_ns);
    int n = 0;
    for (; n < count; ++n) {
        const int h = n * kHeads + (int)threadIdx.x / TG, heads = min(kHeads, a.Hkv - n * kHeads);
        ok &= mbar_wait_within(bar(n & 1), (uint32_t)(n >> 1) & 1u, a.wait_ns);
        RopeQ8Unit<T, CODE, TG, VEC, ADJ> unit(g, sq, span, page, which, h < a.Hkv ? h : 0);
        const T *tile = reinterpret_cast<const T *>(smem + (n & 1) * g.stage) + (int)threadIdx.x / TG * W;
        uint32_t mx = 0;
        if (h < a.Hkv) mx = unit.keep(tile, heads * W, trig);
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (TG > 32 && lane == 0) red[4 * (n & 1) + (threadIdx.x >> 5)] = mx;
        // the stage is read: the one after the next goes there
        if (!__syncthreads_and(ok)) break;
        if (n + 2 < count) load(n + 2);
        if (TG > 32)
            for (int w = 0; w < 4; ++w) mx = max(mx, red[4 * (n & 1) + w]);
        if (h < a.Hkv) unit.put(mx, tile, heads * W, trig);
    }
    if (n < count) {  // a wait that ran out: what is on its way lands before the block ends
        if (threadIdx.x == 0) report_status(a.status, kStatusTimeoutRope);
        if (half > 0) mbar_wait_drain(bar(2), 0);
        for (int m = n; m < count && m < n + 2; ++m) mbar_wait_drain(bar(m & 1), (uint32_t)(m >> 1) & 1u);
    }
}

int launched() {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("rotating append kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <typename T, int CODE, int TG, int VEC> int launch_t(RopeQ8Args g, int nsm, cudaStream_t stream) {
    const RopeArgs &a = g.r;
    const long long units = 2LL * g.touch * a.Hkv, per = 128 / TG;
    RopeArgs q = a;
    q.ko = nullptr;
    q.vo = nullptr;
    g.shape = rope_shape<VEC>(q, a.N == 1, 128);
    long long qb = a.qo ? ((long long)a.N + g.shape.tokens - 1) / g.shape.tokens : 0;
    if (units + qb >= (1LL << 31)) {
        set_error("attn_rope_append_q8: 2^31 or more blocks of rows in a sequence");
        return 2;
    }
    g.items_k = rope_items<VEC>(a.D, a.rot);
    g.items_v = rope_items<VEC>(a.Dv, 0);
    const unsigned by = a.B < 65535 ? a.B : 65535;
    if constexpr (VEC * sizeof(T) == 16) {
        // Blocks of tokens that a block of threads can keep, and enough of them for the
        // device: 16 x 1024 tokens of 32 and 8 heads of 128 take 60 us this way and 63 the
        // other (in blocks of 16 tokens 68 and 85), 16 x 4096 173 and 222, but 2 x 4096,
        // 260 blocks, 50 and 44.
        const long long blk = 1LL << g.blk_shift, wide = a.D > a.Dv ? a.D : a.Dv;
        const long long stage = blk * per * wide * (long long)sizeof(T);
        const long long lanes_k = g.items_k < TG ? g.items_k : TG, lanes_v = g.items_v < TG ? g.items_v : TG;
        const long long most_k = (blk + TG / lanes_k - 1) / (TG / lanes_k) * ((g.items_k + lanes_k - 1) / lanes_k);
        const long long most_v = (blk + TG / lanes_v - 1) / (TG / lanes_v) * ((g.items_v + lanes_v - 1) / lanes_v);
        constexpr int kKeep = RopeQ8Unit<T, CODE, TG, VEC, false>::kKeep;
        const long long bytes = 2 * stage + blk * a.rot * 4;
        const long long tiles = 2LL * g.touch * a.B;
        if (most_k <= kKeep && most_v <= kKeep && blk <= kTileRows && bytes <= kTileBytes && tiles >= 2 * nsm &&
            tiles < (1LL << 30) && (a.qo == nullptr || stream_shape<T, VEC>(q, kTileBytes, 4, 2 * nsm, g.stream))) {
            auto kern = a.adjacent ? rope_q8_stream_kernel<T, CODE, TG, VEC, true>
                                   : rope_q8_stream_kernel<T, CODE, TG, VEC, false>;
            size_t smem = (size_t)bytes;
            g.stage = (int)stage;
            g.q_blocks = 0;
            if (a.qo != nullptr) {
                const long long per_block = (long long)g.stream.tokens * g.stream.warps;
                const long long most = (g.stream.rows + per_block - 1) / per_block;
                g.q_blocks = (unsigned)(most < 2 * nsm ? most : 2 * nsm);
                const size_t rings = (size_t)g.stream.row * g.stream.tokens * g.stream.stages * g.stream.warps;
                if (rings > smem) smem = rings;
            }
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileBytes);
            if (e != cudaSuccess) {
                set_error("rotating append kernel: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
                return 3;
            }
            kern<<<(unsigned)(tiles + g.q_blocks), 128, smem, stream>>>(g);
            return launched();
        }
    }
    // many queries go by themselves, through the kernel for many rows (a second launch is
    // 2 us; that kernel moves 6 TB/s, the blocks behind the units 4.5)
    RopeArgs alone = q;
    alone.k = alone.v = nullptr;
    alone.vo = nullptr;
    alone.block_table = nullptr;
    if (a.qo != nullptr && (a.cu ? a.total : (long long)a.B * a.N) * a.Hq * a.D * (long long)sizeof(T) >= 8LL << 20) {
        const int rc = launch_rope(alone, std::is_same_v<T, float> ? 0 : std::is_same_v<T, __half> ? 1 : 2, stream);
        if (rc) return rc;
        g.r.q = nullptr;
        g.r.qo = nullptr;
        qb = 0;
    }
    g.unit_blocks = (unsigned)((units + per - 1) / per);
    const dim3 grid((unsigned)(g.unit_blocks + qb), by, (a.B + by - 1) / by);
    if (a.adjacent) rope_q8_kernel<T, CODE, TG, VEC, true><<<grid, 128, 0, stream>>>(g);
    else rope_q8_kernel<T, CODE, TG, VEC, false><<<grid, 128, 0, stream>>>(g);
    return launched();
}

template <typename T, int CODE, int VEC> int launch_size(const RopeQ8Args &g, int nsm, cudaStream_t stream) {
    // One warp a unit while its rows fit half of what one warp keeps, four otherwise.  (Of
    // single elements, an item of a plain column is one: with 1024 for them, too, most of a
    // unit was read and turned twice.  16 x 1024 tokens of 8 + 4 heads of 20 in blocks of 32:
    // 29 us, now 20; of 127 in blocks of 8: 136, now 120.)
    constexpr int kWarp = 32 * RopeQ8Unit<T, CODE, 32, VEC, false>::kKeep * (VEC == 1 ? 1 : 2 * VEC);
    const long long most = g.r.N < (1 << g.blk_shift) ? g.r.N : (1 << g.blk_shift);
    const bool small = most * (g.r.D > g.r.Dv ? g.r.D : g.r.Dv) <= kWarp / 2;
    return small ? launch_t<T, CODE, 32, VEC>(g, nsm, stream) : launch_t<T, CODE, 128, VEC>(g, nsm, stream);
}

template <typename T, int CODE> int launch_code(const RopeQ8Args &g, int nsm, cudaStream_t stream) {
    constexpr int kWide = 16 / (int)sizeof(T), kHalf = kWide / 2;
    const int vec = rope_vector(g.r, (int)sizeof(T), 2);
    if (vec == kWide) return launch_size<T, CODE, kWide>(g, nsm, stream);
    if (sizeof(T) == 2 && vec == kHalf) return launch_size<T, CODE, sizeof(T) == 2 ? kHalf : 1>(g, nsm, stream);
    return launch_size<T, CODE, 1>(g, nsm, stream);
}

}  // namespace

int launch_rope_q8(const RopeArgs &a, float *k_scale, float *v_scale, int nblk, int blk_shift,
                   int code, int dtype, cudaStream_t stream) {
    RopeQ8Args g = {};
    g.r = a;
    int dev = 0, rc = current_device(&dev);
    if (rc == 0) rc = status_ptr(dev, &g.r.status);
    g.r.wait_ns = wait_limit_ns();
    if (rc) return rc;
    const int nsm = sm_count(dev);
    g.scales[0] = k_scale;
    g.scales[1] = v_scale;
    g.nblk = nblk;
    g.blk_shift = blk_shift;
    // N rows from any offset in a block
    g.touch = (int)(((long long)a.N - 1 + (1 << blk_shift) - 1) / (1 << blk_shift)) + 1;
    if (code == kCodeE4m3) {
        switch (dtype) {
            case 0: return launch_code<float, kCodeE4m3>(g, nsm, stream);
            case 1: return launch_code<__half, kCodeE4m3>(g, nsm, stream);
            default: return launch_code<__nv_bfloat16, kCodeE4m3>(g, nsm, stream);
        }
    }
    switch (dtype) {
        case 0: return launch_code<float, kCodeInt8>(g, nsm, stream);
        case 1: return launch_code<__half, kCodeInt8>(g, nsm, stream);
        default: return launch_code<__nv_bfloat16, kCodeInt8>(g, nsm, stream);
    }
}

}  // namespace attn
