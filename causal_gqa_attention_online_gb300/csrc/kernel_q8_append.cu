// kernel_q8_append.cu -- writes new K / V rows into the 8-bit paged cache.
//
// For each (sequence, block of tokens that gets rows, head, K or V):
//
//     a      = max |x| over the block's new rows
//     s_new  = the smallest 2^e >= 2^-100 with a <= qmax * 2^e   (qmax 448 or 127)
//     s      = s_new in a block without earlier rows, else max(s_old, s_new)
//     code   = round-to-nearest-even(x / s)
//     earlier rows, where s > s_old:  code = round(code * s_old / s)
//
// Scales are powers of two, so x / s and s_old / s are exact: a block whose
// scale grows token by token requantises e4m3 codes without loss (down to their
// subnormals), and the roundings of int8 codes sum to at most one step.  A block
// that receives an infinity or a NaN gets the scale NaN and codes 0: every row
// that attends to it is poisoned, as by a NaN key of a 16-bit cache.
//
// Bound: one read of the rows (2 or 4 bytes an element) and one write of the
// codes; the single-token call is launch latency.  A unit is one block of one
// head, so the maximum and the codes come from one read: each thread keeps its
// rows' vectors of eight elements in registers between the two passes, and
// reads again (from L2) only what a block of more than kKeep vectors a thread
// leaves over.  Units of few vectors take one warp, others four.
#include "q8.cuh"
#include "launch.h"

namespace attn {
namespace {

constexpr int kKeep = 8;      // vectors of eight elements a thread keeps

struct AppendArgs {
    const void *x[2];      // K, V rows
    uint8_t *pages[2];
    float *scales[2];
    int width[2];          // D, Dv
    int B, N, Hkv;
    const int32_t *cu;     // packed rows: sequence b owns rows [cu[b], cu[b+1])
    long long total;       // packed rows in all
    const int32_t *seqlens_new, *seqlens_k, *block_table;
    int max_pages, page_shift, num_pages, nblk, blk_shift;
    int touch;             // blocks a sequence's new rows can touch
};

template <typename T> struct Vec8 {
    uint4 r[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ float at(int i) const {
        return to_f32<T>(reinterpret_cast<const T *>(r)[i]);
    }
};

template <int TG> __device__ __forceinline__ float group_max(float a, float *red) {
    a = warp_max(a);
    if (TG == 32) return a;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TG / 32; ++w) a = fmaxf(a, red[w]);
    return a;
}

// |x| with NaN as infinity, so that the maximum carries it
__device__ __forceinline__ float mag(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : INFINITY;
}

// One unit by TG threads.  VEC: rows and codes are moved eight elements at a
// time (width a multiple of 8, aligned rows).
template <typename T, int CODE, int TG, bool VEC>
__global__ void __launch_bounds__(128) append_kernel(const AppendArgs a) {
    using Op = CodeOps<CODE>;
    __shared__ float red[4];
    constexpr int UNITS = 128 / TG;
    const int tid = threadIdx.x % TG;
    long long u = (long long)blockIdx.x * UNITS + threadIdx.x / TG;
    const long long nunits = 2LL * a.B * a.touch * a.Hkv;
    if (u >= nunits) return;
    const int which = (int)(u & 1);
    u >>= 1;
    const int h = (int)(u % a.Hkv);
    u /= a.Hkv;
    const int t = (int)(u % a.touch), b = (int)(u / a.touch);

    const long long cap = (long long)a.max_pages << a.page_shift;
    const int len = clamp_len(__ldg(a.seqlens_k + b), (int)cap);
    long long row0;
    int n;
    if (a.cu != nullptr) {
        row0 = max(0, __ldg(a.cu + b));
        n = clamp_len((int)min((long long)__ldg(a.cu + b + 1), a.total) - (int)row0, a.N);
    } else {
        row0 = (long long)b * a.N;
        n = a.seqlens_new ? clamp_len(__ldg(a.seqlens_new + b), a.N) : a.N;
    }
    const AppendSpan span = append_span(len, n, cap, t, a.page_shift, a.blk_shift);
    if (span.last <= span.first) return;
    const int page = __ldg(a.block_table + (long long)b * a.max_pages + span.entry);
    if (page < 0 || page >= a.num_pages) return;
    const int start = (int)span.start, first = (int)span.first;
    const int rows = (int)(span.last - span.first), sub = span.sub;
    const int W = a.width[which];
    float *sp = a.scales[which] + ((long long)page * a.nblk + sub) * a.Hkv + h;
    const T *src = static_cast<const T *>(a.x[which]) +
                   ((row0 + (first - len)) * a.Hkv + h) * (long long)W;
    const long long pitch = (long long)a.Hkv * W;  // elements between rows, of both sides
    // code row `r` of the page
    uint8_t *page_base = a.pages[which] +
                         (((long long)page << a.page_shift) * a.Hkv + h) * (long long)W;
    uint8_t *dst = page_base + (first & ((1 << a.page_shift) - 1)) * pitch;

    const int per_row = VEC ? W / 8 : W;
    const int items = rows * per_row;
    Vec8<T> keep[VEC ? kKeep : 1];
    float amax = 0.f;
    if (VEC) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int it = tid + i * TG;
            if (it < items) keep[i].load(src + (it / per_row) * pitch + (it % per_row) * 8);
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (tid + i * TG < items)
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = fmaxf(amax, mag(keep[i].at(j)));
        for (int it = tid + kKeep * TG; it < items; it += TG) {
            Vec8<T> v;
            v.load(src + (it / per_row) * pitch + (it % per_row) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, mag(v.at(j)));
        }
    } else {
        for (int it = tid; it < items; it += TG)
            amax = fmaxf(amax, mag(to_f32<T>(src[(it / per_row) * pitch + it % per_row])));
    }
    amax = group_max<TG>(amax, red);

    float s = append_scale(amax, CODE);
    const bool old_rows = start < len;
    float s_old = 0.f;
    if (old_rows) {
        s_old = *sp;
        s = (s_old != s_old || s != s) ? __int_as_float(0x7fc00000) : fmaxf(s_old, s);
    }
    if (TG == 32) __syncwarp(); else __syncthreads();  // every thread has read s_old
    if (tid == 0 && !(old_rows && s == s_old)) *sp = s;

    // x / s: a multiplication where s is a power of two (always, unless the
    // caller's own scales are not)
    const bool pow2 = (__float_as_uint(s) & 0x007fffffu) == 0u && s > 0.f && s < 1e38f;
    const float inv = pow2 ? 1.f / s : 0.f;
    auto code_of = [&](float x) -> uint8_t {
        float y = pow2 ? x * inv : __fdiv_rn(x, s);
        y = fabsf(y) <= 3.402823466e38f ? y : 0.f;
        return Op::code(y);
    };
    if (VEC) {
        auto put = [&](const Vec8<T> &v, int it) {
            uint8_t c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = code_of(v.at(j));
            uint2 w;
            w.x = c[0] | (c[1] << 8) | (c[2] << 16) | ((uint32_t)c[3] << 24);
            w.y = c[4] | (c[5] << 8) | (c[6] << 16) | ((uint32_t)c[7] << 24);
            *reinterpret_cast<uint2 *>(dst + (it / per_row) * pitch + (it % per_row) * 8) = w;
        };
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (tid + i * TG < items) put(keep[i], tid + i * TG);
        for (int it = tid + kKeep * TG; it < items; it += TG) {
            Vec8<T> v;
            v.load(src + (it / per_row) * pitch + (it % per_row) * 8);
            put(v, it);
        }
    } else {
        for (int it = tid; it < items; it += TG)
            dst[(it / per_row) * pitch + it % per_row] =
                code_of(to_f32<T>(src[(it / per_row) * pitch + it % per_row]));
    }

    // earlier rows of a block whose scale has grown
    if (old_rows && !(s == s_old)) {
        uint8_t *ob = page_base + (start & ((1 << a.page_shift) - 1)) * pitch;
        const int n_old = (len - start) * W;
        const float ratio = __fdiv_rn(s_old, s);
        for (int it = tid; it < n_old; it += TG) {
            uint8_t *c = ob + (it / W) * pitch + it % W;
            float y = Op::one(*c) * ratio;
            y = fabsf(y) <= 3.402823466e38f ? y : 0.f;
            *c = Op::code(y);
        }
    }
}

template <typename T, int CODE, int TG, bool VEC>
int launch_t(const AppendArgs &a, cudaStream_t stream) {
    const long long nunits = 2LL * a.B * a.touch * a.Hkv;
    const long long blocks = (nunits + 128 / TG - 1) / (128 / TG);
    if (blocks >= (1LL << 31)) {
        set_error("attn_cache_append: too many blocks of rows");
        return 2;
    }
    append_kernel<T, CODE, TG, VEC><<<(unsigned)blocks, 128, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("append kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

template <typename T, int CODE> int launch_code(const AppendArgs &a, cudaStream_t stream) {
    const bool vec = a.width[0] % 8 == 0 && a.width[1] % 8 == 0;
    // one warp a unit while its rows fit one warp's kept vectors by half, four
    // warps otherwise
    const long long most = a.N < (1 << a.blk_shift) ? a.N : (1 << a.blk_shift);
    const bool small = most * (a.width[0] > a.width[1] ? a.width[0] : a.width[1]) <= 32 * 4 * 8;
    if (vec)
        return small ? launch_t<T, CODE, 32, true>(a, stream)
                     : launch_t<T, CODE, 128, true>(a, stream);
    return small ? launch_t<T, CODE, 32, false>(a, stream)
                 : launch_t<T, CODE, 128, false>(a, stream);
}

}  // namespace

int launch_cache_append(const void *k, const void *v, void *k_pages, void *v_pages, float *k_scale,
                        float *v_scale, int B, int N, int Hkv, int D, int Dv,
                        const int32_t *seqlens_new, const int32_t *cu_new, long long total,
                        const int32_t *seqlens_k, const int32_t *block_table, int max_pages,
                        int page_shift, int num_pages, int nblk, int blk_shift, int code,
                        int dtype, cudaStream_t stream) {
    AppendArgs a = {};
    a.x[0] = k;
    a.x[1] = v;
    a.pages[0] = static_cast<uint8_t *>(k_pages);
    a.pages[1] = static_cast<uint8_t *>(v_pages);
    a.scales[0] = k_scale;
    a.scales[1] = v_scale;
    a.width[0] = D;
    a.width[1] = Dv;
    a.B = B;
    a.N = N;
    a.Hkv = Hkv;
    a.cu = cu_new;
    a.total = total;
    a.seqlens_new = seqlens_new;
    a.seqlens_k = seqlens_k;
    a.block_table = block_table;
    a.max_pages = max_pages;
    a.page_shift = page_shift;
    a.num_pages = num_pages;
    a.nblk = nblk;
    a.blk_shift = blk_shift;
    // N rows from any offset in a block
    a.touch = (int)(((long long)N - 1 + (1 << blk_shift) - 1) / (1 << blk_shift)) + 1;
    if (code == kCodeE4m3) {
        switch (dtype) {
            case 0: return launch_code<float, kCodeE4m3>(a, stream);
            case 1: return launch_code<__half, kCodeE4m3>(a, stream);
            default: return launch_code<__nv_bfloat16, kCodeE4m3>(a, stream);
        }
    }
    switch (dtype) {
        case 0: return launch_code<float, kCodeInt8>(a, stream);
        case 1: return launch_code<__half, kCodeInt8>(a, stream);
        default: return launch_code<__nv_bfloat16, kCodeInt8>(a, stream);
    }
}

}  // namespace attn
