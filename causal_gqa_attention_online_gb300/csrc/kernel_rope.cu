// kernel_rope.cu -- the position rotation of rows in 16 or 32 bits, into rows or
// into the pages of a cache (the arithmetic: rope.cuh).
//
// Bound: one read and one write of the rows; the single-token call is launch latency.
//
// rope_stream_kernel, for many rows in 16-byte vectors (rope_stream.cuh): with a thread's
// loads in registers, 640 threads an SM of 96 registers or 1024 of 64, rope_kernel was bound
// by their latency there (16384 tokens of 40 heads of 128 in bf16: 79 us against 61; the
// same with their values into pages, 65536 packed rows: 213 against 135).
//
// rope_kernel, for few rows and for other widths and alignments: a thread owns one item
// (two vectors of a head: VEC pairs) of a token and walks the token's heads with it, so
// that the angles are read once and kept, four heads' loads in flight at a time.  Vectors
// are 16 bytes where every width, stride and address is a multiple of them, 8 bytes for
// widths such as 56 pairs of columns of a half-rotated head (pairs have to fill whole
// vectors), else single elements.
#include "launch.h"
#include "rope_stream.cuh"

namespace attn {
namespace {

constexpr int kStreamBytes = 208 * 1024;  // of a block: one an SM

template <typename T, int VEC, bool ADJ, bool PAGED>
__global__ void __launch_bounds__(32 * kStreamWarps, 1)
    rope_stream_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ StreamShape g) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ StreamToken token[kStreamWarps][kStreamMost][32];
    __shared__ alignas(8) uint64_t full[kStreamWarps][kStreamMost];
    rope_stream<T, VEC, ADJ, PAGED>(a, g, smem, token, full, blockIdx.x, gridDim.x);
}

template <typename T, int VEC, bool ADJ, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads, VEC * sizeof(T) == 16 ? 2 : 3)
    rope_kernel(const __grid_constant__ RopeArgs a, const RopeShape g) {
    rope_rows<T, VEC, ADJ, PAGED>(a, g, blockIdx.x, blockIdx.y + blockIdx.z * gridDim.y);
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

template <typename T, int VEC, bool ADJ, bool PAGED>
int launch_stream(const RopeArgs &a, const StreamShape &g, int nsm, cudaStream_t stream) {
    auto kern = rope_stream_kernel<T, VEC, ADJ, PAGED>;
    const int smem = g.row * g.tokens * g.stages * g.warps;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes);
    if (e != cudaSuccess) {
        set_error("rotation kernel: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return 3;
    }
    const long long per = (long long)g.tokens * g.warps, work = (g.rows + per - 1) / per;
    const unsigned grid = (unsigned)(work < nsm ? work : nsm);
    kern<<<grid, 32 * g.warps, smem, stream>>>(a, g);
    return launched("rotation kernel");
}

template <typename T, int VEC> int launch_vec(const RopeArgs &a, cudaStream_t stream) {
    int dev = 0;
    const int rc = current_device(&dev);
    if (rc) return rc;
    const int nsm = sm_count(dev);
    // (Of packed rows, too, the places up to N of each sequence: rope_kernel has blocks for all
    // of them, rope_stream_kernel for the rows that are there.  63 single rows and 500 more, N
    // 500: 28 us and 7.)
    const long long work = (long long)a.B * a.N * rope_items<VEC>(a.D, a.rot) *
                           ((a.qo ? a.Hq : 0) + (a.ko ? a.Hkv : 0));
    // few: no more than the resident threads of rope_kernel take at once, four heads each
    const bool few = work < 2LL * nsm * kRopeThreads * kRopeUnroll;
    // many: enough to make up for the stages' start (40 heads of 128 in bf16, on the GPU: 1500
    // tokens 8.3 us and 6.7 with rope_kernel, 2400 tokens 8.5 and 12.1)
    const bool many = work >= 4LL * nsm * kRopeThreads * kRopeUnroll;
    if constexpr (VEC * sizeof(T) == 16) {
        StreamShape s;
        if (many && stream_shape<T, VEC>(a, kStreamBytes, kStreamWarps, nsm, s)) {
            RopeArgs x = a;
            const int rs = status_ptr(dev, &x.status);
            if (rs) return rs;
            x.wait_ns = wait_limit_ns();
            if (a.adjacent) return a.block_table ? launch_stream<T, VEC, true, true>(x, s, nsm, stream)
                                                 : launch_stream<T, VEC, true, false>(x, s, nsm, stream);
            return a.block_table ? launch_stream<T, VEC, false, true>(x, s, nsm, stream)
                                 : launch_stream<T, VEC, false, false>(x, s, nsm, stream);
        }
    }
    const RopeShape g = rope_shape<VEC>(a, few, few ? 128 : kRopeThreads);
    const long long blocks = ((long long)a.N + g.tokens - 1) / g.tokens;
    const unsigned by = a.B < 65535 ? a.B : 65535;
    const dim3 grid((unsigned)blocks, by, (a.B + by - 1) / by);
    if (a.adjacent) {
        if (a.block_table) rope_kernel<T, VEC, true, true><<<grid, g.threads, 0, stream>>>(a, g);
        else rope_kernel<T, VEC, true, false><<<grid, g.threads, 0, stream>>>(a, g);
    } else {
        if (a.block_table) rope_kernel<T, VEC, false, true><<<grid, g.threads, 0, stream>>>(a, g);
        else rope_kernel<T, VEC, false, false><<<grid, g.threads, 0, stream>>>(a, g);
    }
    return launched("rotation kernel");
}

template <typename T> int launch_type(const RopeArgs &a, cudaStream_t stream) {
    constexpr int kWide = 16 / (int)sizeof(T), kHalf = kWide / 2;
    const int vec = rope_vector(a, (int)sizeof(T), 1);
    if (vec == kWide) return launch_vec<T, kWide>(a, stream);
    if (sizeof(T) == 2 && vec == kHalf) return launch_vec<T, sizeof(T) == 2 ? kHalf : 1>(a, stream);
    return launch_vec<T, 1>(a, stream);
}

}  // namespace

// Vectors of 16 bytes, of 8 (16-bit types; four angles are 16 bytes) or single elements.
int rope_vector(const RopeArgs &a, int es, int v_unit) {
    for (int bytes = 16; bytes >= 4 * es; bytes /= 2) {
        const int vec = bytes / es;
        auto fits = [&](const void *p, long long stride) {
            return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride % vec == 0;
        };
        // pairs fill whole vectors, plain columns two of them, and heads of V v_unit
        if (a.rot % (2 * vec) || a.D % (2 * vec) || (a.v != nullptr && a.Dv % (v_unit * vec))) continue;
        if (reinterpret_cast<uintptr_t>(a.cos) % 16 || reinterpret_cast<uintptr_t>(a.sin) % 16) continue;
        // (a row of angles that does not fill 16 bytes breaks their alignment)
        if ((a.rot / 2) % 4) continue;
        if (fits(a.q, a.q_stride) && fits(a.k, a.k_stride) && fits(a.v, a.v_stride) && fits(a.qo, 0) &&
            fits(a.ko, 0) && fits(a.vo, 0))
            return vec;
    }
    return 1;
}

int launch_rope(const RopeArgs &a, int dtype, cudaStream_t stream) {
    switch (dtype) {
        case 0: return launch_type<float>(a, stream);
        case 1: return launch_type<__half>(a, stream);
        default: return launch_type<__nv_bfloat16>(a, stream);
    }
}

}  // namespace attn
