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
// Magnitudes are compared as integers, two 16-bit ones an instruction (infinities
// and NaN come out above every finite value); a whole block whose rows divide the
// threads takes a path without tests and steps by one pointer.  Measured: prompts
// of 16 ragged sequences up to 4096 rows (8 heads, D 128, bf16 to e4m3, 212 MB) 40
// us, 5.4 TB/s, 0.79 of a plain copy; 64 sequences of one row 6 us.
#include <type_traits>

#include "q8_append.cuh"
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
    int row_shift[2];      // log2 of the vectors of a row (-1: no power of two)
    int row_step[2];       // rows that a unit's threads take at a time
};

// Eight elements.
template <typename T> struct Vec8 {
    static constexpr int NW = sizeof(T) * 2;  // 32-bit words
    uint32_t w[NW];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < NW / 4; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NW; ++i) w[i] = 0u;
    }
    // the largest magnitude, added to `m`: two 16-bit maxima in a word, or one
    __device__ __forceinline__ uint32_t max_into(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < NW; ++i)
            m = sizeof(T) == 2 ? __vmaxu2(m, w[i] & 0x7fff7fffu) : max(m, w[i] & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ float at(int i) const {
        return to_f32<T>(reinterpret_cast<const T *>(w)[i]);
    }
};

// One unit by TG threads.  VEC: rows and codes are moved eight elements at a
// time (width a multiple of 8, aligned rows).
template <typename T, int CODE, int TG, bool VEC>
__global__ void __launch_bounds__(128, VEC && sizeof(T) == 2 ? 8 : 3) append_kernel(const __grid_constant__ AppendArgs a) {
    using Op = CodeOps<CODE>;
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x % TG;
    // units: block, head, K or V of sequence blockIdx.y (+ gridDim.y ...)
    const uint32_t u = blockIdx.x * (128 / TG) + threadIdx.x / TG;
    const int which = (int)(u & 1u);
    const int t = (int)((u >> 1) / (uint32_t)a.Hkv), h = (int)((u >> 1) - (uint32_t)t * (uint32_t)a.Hkv);
    const uint32_t ub = blockIdx.y + blockIdx.z * gridDim.y;
    if (t >= a.touch || ub >= (uint32_t)a.B) return;
    const int b = (int)ub;

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
    const int rows = (int)(span.last - span.first);
    const int W = a.width[which];
    float *sp = a.scales[which] + ((long long)page * a.nblk + span.sub) * a.Hkv + h;
    const T *src = static_cast<const T *>(a.x[which]) +
                   ((row0 + (first - len)) * a.Hkv + h) * (long long)W;
    const int pitch = a.Hkv * W;  // elements between rows, of both sides
    uint8_t *page_base = a.pages[which] +
                         (((long long)page << a.page_shift) * a.Hkv + h) * (long long)W;
    uint8_t *dst = page_base + (long long)(first & ((1 << a.page_shift) - 1)) * pitch;
    const bool old_rows = start < len;
    float s_old = old_rows ? __ldcg(sp) : 0.f;

    // Vectors (or elements) tid, tid + TG, ...: row and column of each by
    // stepping, without a division.
    const int per_row = VEC ? W / 8 : W, unit = VEC ? 8 : 1;
    const int items = rows * per_row;
    const int dr = a.row_step[which], dc = TG - dr * per_row;  // TG / per_row
    const int sh = a.row_shift[which];  // log2(per_row), or -1
    const int r_first = sh >= 0 ? tid >> sh : tid / per_row, c_first = tid - r_first * per_row;
    struct Place {
        int c;
        long long at;
    };
    auto begin = [&]() -> Place { return {c_first, (long long)r_first * pitch + c_first * unit}; };
    auto next = [&](Place &q) {
        q.c += dc;
        q.at += (long long)dr * pitch + dc * unit;
        if (q.c >= per_row) {
            q.c -= per_row;
            q.at += pitch - per_row * unit;
        }
    };

    Vec8<T> keep[VEC ? kKeep : 1];
    uint32_t mx = 0;
    // a whole block of rows that divide the threads: no tests, one step
    const bool even = VEC && items == kKeep * TG && dc == 0;
    const long long step = (long long)dr * pitch;
    if (VEC) {
        Place q = begin();
        if (even) {
            const T *x = src + q.at;
#pragma unroll
            for (int i = 0; i < kKeep; ++i, x += step) keep[i].load(x);
        } else {
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                if (tid + i * TG < items) keep[i].load(src + q.at);
                else keep[i].clear();
                next(q);
            }
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i) mx = keep[i].max_into(mx);
        for (int it = tid + kKeep * TG; it < items; it += TG, next(q)) {
            Vec8<T> v;
            v.load(src + q.at);
            mx = v.max_into(mx);
        }
        if (sizeof(T) == 2) mx = max(mx & 0xffffu, mx >> 16);
    } else {
        Place q = begin();
        for (int it = tid; it < items; it += TG, next(q)) {
            const T x = src[q.at];
            uint32_t w = sizeof(T) == 2 ? (uint32_t)*reinterpret_cast<const uint16_t *>(&x) & 0x7fffu
                                        : *reinterpret_cast<const uint32_t *>(&x) & 0x7fffffffu;
            mx = max(mx, w);
        }
    }
    mx = group_max<TG>(mx, red);

    const float nan = __int_as_float(0x7fc00000);
    float s = mx >= Bits<T>::kInf ? nan : append_scale(Bits<T>::value(mx), CODE);
    if (old_rows) s = s_old != s_old || s != s ? nan : fmaxf(s_old, s);
    if (tid == 0 && !(old_rows && s == s_old)) *sp = s;

    // x / s: a multiplication where s is a power of two (always, unless the
    // caller's own scales are not); a NaN scale: codes 0
    const bool pow2 = (__float_as_uint(s) & 0x807fffffu) == 0u && s > 0.f && s < 1e38f;
    const float inv = pow2 ? 1.f / s : 0.f;
    auto emit = [&](auto is_pow2) {
        auto scaled = [&](float x) -> float {
            return decltype(is_pow2)::value ? x * inv : divided(x, s, Op::kMax);
        };
        Place q = begin();
        if (VEC) {
            auto put = [&](const Vec8<T> &v, uint8_t *to) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = scaled(v.at(j));
                *reinterpret_cast<uint2 *>(to) =
                    make_uint2(code4<CODE>(y[0], y[1], y[2], y[3]), code4<CODE>(y[4], y[5], y[6], y[7]));
            };
            if (even) {
                uint8_t *to = dst + q.at;
#pragma unroll
                for (int i = 0; i < kKeep; ++i, to += step) put(keep[i], to);
                return;
            }
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                if (tid + i * TG < items) put(keep[i], dst + q.at);
                next(q);
            }
            for (int it = tid + kKeep * TG; it < items; it += TG, next(q)) {
                Vec8<T> v;
                v.load(src + q.at);
                put(v, dst + q.at);
            }
        } else {
            for (int it = tid; it < items; it += TG, next(q)) dst[q.at] = Op::code(scaled(to_f32<T>(src[q.at])));
        }
    };
    if (pow2) emit(std::true_type{});
    else emit(std::false_type{});

    // earlier rows of a block whose scale has grown
    if (old_rows && !(s == s_old)) {
        uint8_t *ob = page_base + (long long)(start & ((1 << a.page_shift) - 1)) * pitch;
        const int n_old = (len - start) * W;
        const float ratio = __fdiv_rn(s_old, s);
        for (int it = tid; it < n_old; it += TG) {
            uint8_t *c = ob + (long long)(it / W) * pitch + it % W;
            float y = Op::one(*c) * ratio;
            y = fabsf(y) <= 3.402823466e38f ? y : 0.f;
            *c = Op::code(y);
        }
    }
}

template <typename T, int CODE, int TG, bool VEC>
int launch_t(const AppendArgs &a, cudaStream_t stream) {
    AppendArgs x = a;
    for (int i = 0; i < 2; ++i) {
        const int per_row = VEC ? a.width[i] / 8 : a.width[i];
        x.row_shift[i] = -1;
        for (int k = 0; k < 10; ++k)
            if (1 << k == per_row) x.row_shift[i] = k;
        x.row_step[i] = TG / per_row;
    }
    const long long units = 2LL * a.touch * a.Hkv, blocks = (units + 128 / TG - 1) / (128 / TG);
    if (units >= (1LL << 31)) {
        set_error("attn_cache_append: 2^31 or more blocks of rows in a sequence");
        return 2;
    }
    const unsigned by = a.B < 65535 ? a.B : 65535;
    append_kernel<T, CODE, TG, VEC><<<dim3((unsigned)blocks, by, (a.B + by - 1) / by), 128, 0, stream>>>(x);
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
