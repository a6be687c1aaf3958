// kernel_q8_expand.cu -- the keys and values of an 8-bit paged cache as
// contiguous rows of q's type, for the kernels that read those.
//
//     out[b][j][h][:] = code * scale        for j < Kb
//
// The product of an 8-bit code and a power-of-two scale (what the append
// writes) is exact in bf16, and in fp16 up to its range: values past +-65504
// are clamped to it.  With other scales this rounds once, to q's type.  Rows at
// or past a sequence's length are not written (no kernel reads them as
// values).  One read of the valid codes, one write of twice the bytes: bound by
// HBM, and by how many loads are in flight -- a block takes 16 rows (64: 30 us for 23), whose table
// entries and scales it reads first, and a thread has four 16-byte loads under
// way.
#include "q8.cuh"
#include "launch.h"

namespace attn {
namespace {

constexpr int kRowsPerBlock = 16;

template <typename T> __device__ __forceinline__ T to_out(float x) { return from_f32<T>(x); }
template <> __device__ __forceinline__ __half to_out<__half>(float x) {
    // a NaN stays one
    return __float2half_rn(x != x ? x : fminf(fmaxf(x, -65504.f), 65504.f));
}

struct ExpandArgs {
    Q8Cache c;
    void *out[2];
    int width[2];
    int Hkv, K;
    const int32_t *seqlens_k, *block_table;
    int max_pages, page_shift, num_pages;
};

// 16 codes times s.
template <typename T, int CODE> __device__ __forceinline__ void expand16(T *dst, const uint4 &x, float s) {
    using Op = CodeOps<CODE>;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    __align__(16) T v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t p[2];
        Op::k_pairs(w[i], p[0], p[1]);
        // the bytes of the first pair: 0 and 1, or 0 and 2
        constexpr int B1 = Op::kPerm ? 2 : 1, B2 = Op::kPerm ? 1 : 2;
        const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&p[0]));
        const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&p[1]));
        v[4 * i] = to_out<T>(f0.x * s);
        v[4 * i + B1] = to_out<T>(f0.y * s);
        v[4 * i + B2] = to_out<T>(f1.x * s);
        v[4 * i + 3] = to_out<T>(f1.y * s);
    }
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i)
        reinterpret_cast<uint4 *>(dst)[i] = reinterpret_cast<const uint4 *>(v)[i];
}

// grid: (row blocks of a sequence, K | V, sequence); VEC elements at a time
// within one head.
template <typename T, int CODE, int VEC>
__global__ void __launch_bounds__(256) expand_kernel(const __grid_constant__ ExpandArgs a) {
    using Op = CodeOps<CODE>;
    __shared__ long long page_row[kRowsPerBlock];   // row of the pool
    __shared__ long long page_blk[kRowsPerBlock];   // block of scales
    const int b = blockIdx.z, which = blockIdx.y;
    const int Kb = clamp_len(__ldg(a.seqlens_k + b), a.K);
    const int r0 = blockIdx.x * kRowsPerBlock;
    const int rows = min(kRowsPerBlock, Kb - r0);
    if (rows <= 0) return;
    const int W = a.width[which];
    if (threadIdx.x < rows) {
        const int key = r0 + threadIdx.x, at = key & ((1 << a.page_shift) - 1);
        int pg = __ldg(a.block_table + (long long)b * a.max_pages + (key >> a.page_shift));
        pg = min(max(pg, 0), a.num_pages - 1);
        page_row[threadIdx.x] = ((long long)pg << a.page_shift) + at;
        page_blk[threadIdx.x] = (long long)pg * a.c.nblk + (at >> a.c.blk_shift);
    }
    __syncthreads();
    const int pitch = a.Hkv * W, per_row = pitch / VEC;
    const uint8_t *codes = which ? a.c.v : a.c.k;
    const float *scales = which ? a.c.vs : a.c.ks;
    T *out = static_cast<T *>(a.out[which]) + ((long long)b * a.K + r0) * pitch;
    // vectors tid, tid + 256, ...: row and column by stepping
    const int dr = 256 / per_row, dc = 256 - dr * per_row;
    int r = threadIdx.x / per_row, c = threadIdx.x - r * per_row;
    constexpr int U = VEC == 16 ? 4 : 1;
    while (r < rows) {
        int rr[U], cc[U];
        uint4 x[U];
        uint8_t y[U];
        float s[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            rr[i] = r;
            cc[i] = c * VEC;
            if (r < rows) {
                const uint8_t *src = codes + page_row[r] * pitch + cc[i];
                if (VEC == 16) x[i] = __ldg(reinterpret_cast<const uint4 *>(src));
                else y[i] = __ldg(src);
                s[i] = __ldg(scales + page_blk[r] * a.Hkv + cc[i] / W);
            }
            r += dr;
            c += dc;
            if (c >= per_row) {
                c -= per_row;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (rr[i] < rows) {
                T *dst = out + (long long)rr[i] * pitch + cc[i];
                if (VEC == 16) expand16<T, CODE>(dst, x[i], s[i]);
                else *dst = to_out<T>(Op::one(y[i]) * s[i]);
            }
    }
}

template <typename T, int CODE>
int launch_t(const ExpandArgs &a, int B, cudaStream_t stream) {
    const bool vec = a.width[0] % 16 == 0 && a.width[1] % 16 == 0;
    const dim3 grid((unsigned)((a.K + kRowsPerBlock - 1) / kRowsPerBlock), 2, (unsigned)B);
    if (vec) expand_kernel<T, CODE, 16><<<grid, 256, 0, stream>>>(a);
    else expand_kernel<T, CODE, 1><<<grid, 256, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("expand kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
}

}  // namespace

// B <= 65535 sequences starting at p's; p: the paged problem (K, seqlens_k,
// block table); k_out / v_out: [B][K][Hkv][D | Dv] of dtype.
int launch_q8_expand(const AttnParams &p, const Q8Cache &c, void *k_out, void *v_out, int dtype,
                     cudaStream_t stream) {
    if (p.K == 0 || p.B == 0) return 0;
    ExpandArgs a = {};
    a.c = c;
    a.out[0] = k_out;
    a.out[1] = v_out;
    a.width[0] = p.D;
    a.width[1] = p.Dv;
    a.Hkv = p.Hkv;
    a.K = p.K;
    a.seqlens_k = p.seqlens_k;
    a.block_table = p.block_table;
    a.max_pages = p.max_pages;
    a.page_shift = p.page_shift;
    a.num_pages = p.num_pages;
    if (c.code == kCodeE4m3) {
        switch (dtype) {
            case 0: return launch_t<float, kCodeE4m3>(a, p.B, stream);
            case 1: return launch_t<__half, kCodeE4m3>(a, p.B, stream);
            default: return launch_t<__nv_bfloat16, kCodeE4m3>(a, p.B, stream);
        }
    }
    switch (dtype) {
        case 0: return launch_t<float, kCodeInt8>(a, p.B, stream);
        case 1: return launch_t<__half, kCodeInt8>(a, p.B, stream);
        default: return launch_t<__nv_bfloat16, kCodeInt8>(a, p.B, stream);
    }
}

}  // namespace attn
