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
// single-token call is launch latency.  A unit is one block of one head of K or V by
// one or four warps, as in the append kernel; a thread keeps what it turned (64 floats)
// between the maximum and the codes, and turns again (from L2) what is left over.  The
// blocks behind the units turn the queries.
#include "launch.h"
#include "q8_append.cuh"
#include "rope.cuh"

namespace attn {
namespace {

struct RopeQ8Args {
    RopeArgs r;         // ko, vo: the pools of codes; q rows beside them
    float *scales[2];
    int nblk, blk_shift;
    int touch;          // blocks a sequence's new rows can touch
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

template <typename T, int CODE, int TG, int VEC>
__global__ void __launch_bounds__(128) rope_q8_kernel(const __grid_constant__ RopeQ8Args g) {
    using Op = CodeOps<CODE>;
    constexpr int kKeep = 32 / VEC < 8 ? 32 / VEC : 8;  // items a thread keeps
    __shared__ uint32_t red[4];
    const RopeArgs &a = g.r;
    const uint32_t ub = blockIdx.y + blockIdx.z * gridDim.y;
    if (blockIdx.x >= g.unit_blocks) {
        RopeArgs q = a;
        q.ko = nullptr;
        q.v = nullptr;
        rope_rows<T, VEC, false>(q, g.shape, blockIdx.x - g.unit_blocks, ub);
        return;
    }
    const int tid = threadIdx.x % TG;
    const uint32_t u = blockIdx.x * (128 / TG) + threadIdx.x / TG;
    const int which = (int)(u & 1u);
    const int t = (int)((u >> 1) / (uint32_t)a.Hkv), h = (int)((u >> 1) - (uint32_t)t * (uint32_t)a.Hkv);
    if (t >= g.touch || ub >= (uint32_t)a.B) return;
    const int b = (int)ub;
    const RopeSeq sq = rope_seq(a, b);
    const AppendSpan span = append_span(sq.len, sq.n, (long long)a.max_pages << a.page_shift, t,
                                        a.page_shift, g.blk_shift);
    if (span.last <= span.first) return;
    const int page = __ldg(a.block_table + (long long)b * a.max_pages + span.entry);
    if (page < 0 || page >= a.num_pages) return;
    const int first = (int)span.first, rows = (int)(span.last - span.first);
    const int W = which ? a.Dv : a.D, rot = which ? 0 : a.rot;
    float *sp = g.scales[which] + ((long long)page * g.nblk + span.sub) * a.Hkv + h;
    const long long stride = which ? a.v_stride : a.k_stride;
    const T *src = static_cast<const T *>(which ? a.v : a.k) + (sq.row0 + (first - sq.len)) * stride +
                   (long long)h * W;
    const int pitch = a.Hkv * W;
    uint8_t *page_base = static_cast<uint8_t *>(which ? a.vo : a.ko) +
                         (((long long)page << a.page_shift) * a.Hkv + h) * (long long)W;
    uint8_t *dst = page_base + (long long)(first & ((1 << a.page_shift) - 1)) * pitch;
    const bool old_rows = span.start < sq.len;
    const float s_old = old_rows ? __ldcg(sp) : 0.f;

    const int per_row = rope_items<VEC>(W, rot), items = rows * per_row;
    // item i of the unit: its row, its columns, its turned values
    struct Place {
        int r;
        RopeItem<VEC> it;
    };
    auto place = [&](int i) -> Place {
        const int r = i / per_row;
        return {r, rope_item<VEC>(i - r * per_row, rot, a.adjacent)};
    };
    auto fetch = [&](const Place &p, float (&y)[2 * VEC]) {
        RowVec<T, VEC> x, w;
        x.load(src + p.r * stride + p.it.a);
        w.load(src + p.r * stride + p.it.b);
        Trig<VEC> tr;
        if (p.it.trig >= 0) tr.load(a, rope_position(a, sq, first - sq.len + p.r), p.it.trig);
        turn_item<T, VEC>(p.it, x, w, tr, a.adjacent, y);
    };
    float keep[kKeep][2 * VEC];
    uint32_t mx = 0;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int i = tid + k * TG;
        if (i < items) {
            fetch(place(i), keep[k]);
        } else {
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) keep[k][e] = 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) mx = max(mx, __float_as_uint(keep[k][e]) & 0x7fffffffu);
    for (int i = tid + kKeep * TG; i < items; i += TG) {
        float y[2 * VEC];
        fetch(place(i), y);
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) mx = max(mx, __float_as_uint(y[e]) & 0x7fffffffu);
    }
    mx = group_max<TG>(mx, red);

    const float nan = __int_as_float(0x7fc00000);
    float s = mx >= Bits<float>::kInf ? nan : append_scale(__uint_as_float(mx), CODE);
    if (old_rows) s = s_old != s_old || s != s ? nan : fmaxf(s_old, s);
    if (tid == 0 && !(old_rows && s == s_old)) *sp = s;
    // x / s: a multiplication where s is a power of two (always, unless the caller's
    // own scales are not); a NaN scale: codes 0
    const bool pow2 = (__float_as_uint(s) & 0x807fffffu) == 0u && s > 0.f && s < 1e38f;
    const float inv = pow2 ? 1.f / s : 0.f;
    auto put = [&](int i, float (&y)[2 * VEC]) {
        const Place p = place(i);
#pragma unroll
        for (int e = 0; e < 2 * VEC; ++e) y[e] = pow2 ? y[e] * inv : divided(y[e], s, Op::kMax);
        uint8_t *to = dst + (long long)p.r * pitch;
        put_codes<CODE, VEC>(to + p.it.a, y);
        if (VEC > 1 || p.it.trig >= 0) put_codes<CODE, VEC>(to + p.it.b, y + VEC);
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
        if (tid + k * TG < items) put(tid + k * TG, keep[k]);
    for (int i = tid + kKeep * TG; i < items; i += TG) {
        float y[2 * VEC];
        fetch(place(i), y);
        put(i, y);
    }
    // earlier rows of a block whose scale has grown
    if (old_rows && !(s == s_old)) {
        const int start = (int)span.start;
        uint8_t *ob = page_base + (long long)(start & ((1 << a.page_shift) - 1)) * pitch;
        const int n_old = (sq.len - start) * W;
        const float ratio = __fdiv_rn(s_old, s);
        for (int i = tid; i < n_old; i += TG) {
            uint8_t *c = ob + (long long)(i / W) * pitch + i % W;
            float y = Op::one(*c) * ratio;
            y = fabsf(y) <= 3.402823466e38f ? y : 0.f;
            *c = Op::code(y);
        }
    }
}

template <typename T, int CODE, int TG, int VEC> int launch_t(RopeQ8Args g, cudaStream_t stream) {
    const RopeArgs &a = g.r;
    const long long units = 2LL * g.touch * a.Hkv, per = 128 / TG;
    RopeArgs q = a;
    q.ko = nullptr;
    g.shape = rope_shape<VEC>(q);
    const long long qb = a.qo ? ((long long)a.N + g.shape.tokens - 1) / g.shape.tokens : 0;
    if (units + qb >= (1LL << 31)) {
        set_error("attn_rope_append_q8: 2^31 or more blocks of rows in a sequence");
        return 2;
    }
    g.unit_blocks = (unsigned)((units + per - 1) / per);
    const unsigned by = a.B < 65535 ? a.B : 65535;
    rope_q8_kernel<T, CODE, TG, VEC>
        <<<dim3((unsigned)(g.unit_blocks + qb), by, (a.B + by - 1) / by), 128, 0, stream>>>(g);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("rotating append kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <typename T, int CODE, int VEC> int launch_size(const RopeQ8Args &g, cudaStream_t stream) {
    // one warp a unit while its rows fit half of what one warp keeps, four otherwise
    const long long most = g.r.N < (1 << g.blk_shift) ? g.r.N : (1 << g.blk_shift);
    const bool small = most * (g.r.D > g.r.Dv ? g.r.D : g.r.Dv) <= 32 * 32;
    return small ? launch_t<T, CODE, 32, VEC>(g, stream) : launch_t<T, CODE, 128, VEC>(g, stream);
}

template <typename T, int CODE> int launch_code(const RopeQ8Args &g, cudaStream_t stream) {
    constexpr int kWide = 16 / (int)sizeof(T), kHalf = kWide / 2;
    const int vec = rope_vector(g.r, (int)sizeof(T), 2);
    if (vec == kWide) return launch_size<T, CODE, kWide>(g, stream);
    if (sizeof(T) == 2 && vec == kHalf) return launch_size<T, CODE, sizeof(T) == 2 ? kHalf : 1>(g, stream);
    return launch_size<T, CODE, 1>(g, stream);
}

}  // namespace

int launch_rope_q8(const RopeArgs &a, float *k_scale, float *v_scale, int nblk, int blk_shift,
                   int code, int dtype, cudaStream_t stream) {
    RopeQ8Args g = {};
    g.r = a;
    g.scales[0] = k_scale;
    g.scales[1] = v_scale;
    g.nblk = nblk;
    g.blk_shift = blk_shift;
    // N rows from any offset in a block
    g.touch = (int)(((long long)a.N - 1 + (1 << blk_shift) - 1) / (1 << blk_shift)) + 1;
    if (code == kCodeE4m3) {
        switch (dtype) {
            case 0: return launch_code<float, kCodeE4m3>(g, stream);
            case 1: return launch_code<__half, kCodeE4m3>(g, stream);
            default: return launch_code<__nv_bfloat16, kCodeE4m3>(g, stream);
        }
    }
    switch (dtype) {
        case 0: return launch_code<float, kCodeInt8>(g, stream);
        case 1: return launch_code<__half, kCodeInt8>(g, stream);
        default: return launch_code<__nv_bfloat16, kCodeInt8>(g, stream);
    }
}

}  // namespace attn
