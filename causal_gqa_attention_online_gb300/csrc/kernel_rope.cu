// kernel_rope.cu -- the position rotation of rows in 16 or 32 bits, into rows or
// into the pages of a cache (the arithmetic: rope.cuh).
//
// Bound: one read and one write of the rows; the single-token call is launch
// latency.  A thread owns one item (two vectors of a head: VEC pairs) of a token and
// walks the token's heads with it, so that the angles are read once and kept, four
// heads' loads in flight at a time; V rows are copied as they are.  Tokens of few
// items share a block.  Vectors are 16 bytes where every width, stride and address is
// a multiple of them, 8 bytes for widths such as 56 pairs of columns of a half-rotated
// head (pairs have to fill whole vectors), else single elements.
#include "launch.h"
#include "rope.cuh"

namespace attn {
namespace {

template <typename T, int VEC, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a,
                                                            const RopeShape g) {
    rope_rows<T, VEC, PAGED>(a, g, blockIdx.x, blockIdx.y + blockIdx.z * gridDim.y);
}

template <typename T, int VEC> int launch_vec(const RopeArgs &a, cudaStream_t stream) {
    const RopeShape g = rope_shape<VEC>(a);
    const long long blocks = ((long long)a.N + g.tokens - 1) / g.tokens;
    const unsigned by = a.B < 65535 ? a.B : 65535;
    const dim3 grid((unsigned)blocks, by, (a.B + by - 1) / by);
    if (a.block_table) rope_kernel<T, VEC, true><<<grid, kRopeThreads, 0, stream>>>(a, g);
    else rope_kernel<T, VEC, false><<<grid, kRopeThreads, 0, stream>>>(a, g);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("rotation kernel launch: %s", cudaGetErrorString(e));
        return 3;
    }
    count_launch();
    return 0;
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
