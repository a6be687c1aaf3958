// q8_append.cuh -- what the kernels that write rows into the 8-bit paged cache
// share: magnitudes, the choice of a block's scale, codes of four values.
#pragma once

#include "q8.cuh"

namespace attn {

// |x| as an unsigned integer of the type's bits: ordered as the magnitudes are,
// infinity and NaN above every finite value.
template <typename T> struct Bits;
template <> struct Bits<float> {
    static constexpr uint32_t kInf = 0x7f800000u;
    __device__ __forceinline__ static float value(uint32_t m) { return __uint_as_float(m); }
};
template <> struct Bits<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7f80u;
    __device__ __forceinline__ static float value(uint32_t m) { return __uint_as_float(m << 16); }
};
template <> struct Bits<__half> {
    static constexpr uint32_t kInf = 0x7c00u;
    __device__ __forceinline__ static float value(uint32_t m) {
        return __half2float(__ushort_as_half((unsigned short)m));
    }
};

// Four codes of y0 .. y3, |y| <= qmax.
template <int CODE> __device__ __forceinline__ uint32_t code4(float y0, float y1, float y2, float y3) {
    if (CODE == kCodeE4m3) {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(y1), "f"(y0));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(y3), "f"(y2));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
    // adding 1.5 * 2^23 rounds to the nearest even integer and leaves it, in two's
    // complement, in the low bits
    const float k = 12582912.f;
    const uint32_t a = __float_as_uint(y0 + k), b = __float_as_uint(y1 + k);
    const uint32_t c = __float_as_uint(y2 + k), d = __float_as_uint(y3 + k);
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// x / s within +-most, 0 where it is no number.
__device__ __noinline__ static float divided(float x, float s, float most) {
    const float y = __fdiv_rn(x, s);
    return fabsf(y) <= most ? y : y > 0.f ? most : y < 0.f ? -most : 0.f;
}

// The largest `a` of the TG threads of a unit (red: a word for each of its warps).
template <int TG> __device__ __forceinline__ uint32_t group_max(uint32_t a, uint32_t *red) {
    a = __reduce_max_sync(0xffffffffu, a);
    if (TG == 32) return a;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TG / 32; ++w) a = max(a, red[w]);
    return a;
}

}  // namespace attn
