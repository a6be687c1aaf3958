// q8.cuh -- the 8-bit paged K/V cache: its descriptor and the conversions of
// its codes, shared by the append, expand and decode kernels.
//
// A page holds page_size rows [Hkv][D] of 8-bit codes and, for each block of
// page_size / nblk tokens and each head, one fp32 scale: a row's value is
// code * scale.  Codes are int8 (-127..127) or e4m3 (the NaN code is never
// written).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace attn {

enum : int { kCodeE4m3 = 0, kCodeInt8 = 1 };

struct Q8Cache {
    const uint8_t *k, *v;     // [num_pages][page_size][Hkv][D | Dv]
    const float *ks, *vs;     // [num_pages][nblk][Hkv]
    int code;
    int nblk;                 // blocks a page
    int blk_shift;            // log2(tokens a block)
};

// Codes to f16 pairs, exactly.  k0 / k1: the four bytes of a word as two pairs in
// any fixed order (kPerm: whether that is 0 2, 1 3 instead of 0 1, 2 3); even /
// odd: bytes 0 and 2, 1 and 3.  e4m3 has an instruction for adjacent bytes, so
// even / odd first bring those together.
template <int CODE> struct CodeOps;
template <> struct CodeOps<kCodeE4m3> {
    static constexpr bool kPerm = false;
    __device__ __forceinline__ static uint32_t pair(uint16_t x) {
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(x));
        return r;
    }
    __device__ __forceinline__ static void k_pairs(uint32_t x, uint32_t &k0, uint32_t &k1) {
        k0 = pair((uint16_t)x);
        k1 = pair((uint16_t)(x >> 16));
    }
    __device__ __forceinline__ static void even_odd(uint32_t x, uint32_t &even, uint32_t &odd) {
        const uint32_t y = __byte_perm(x, 0, 0x3120);
        even = pair((uint16_t)y);
        odd = pair((uint16_t)(y >> 16));
    }
    __device__ __forceinline__ static float one(uint8_t c) {
        return __half2float(__ushort_as_half((unsigned short)(pair(c) & 0xffffu)));
    }
    __device__ __forceinline__ static uint8_t code(float y) {
        return (uint8_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
    }
    static constexpr float kMax = 448.f;
};
// int8: the code with its sign bit flipped in the low byte of 0x6400 is the f16
// 1024 + (code + 128); subtracting 1152 leaves the code, exactly.
template <> struct CodeOps<kCodeInt8> {
    static constexpr bool kPerm = true;
    __device__ __forceinline__ static uint32_t debias(uint32_t t) {
        const uint32_t b = 0x64806480u;  // 1152, 1152
        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&t),
                                  *reinterpret_cast<const __half2 *>(&b));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    __device__ __forceinline__ static void even_odd(uint32_t x, uint32_t &even, uint32_t &odd) {
        even = debias((x & 0x00ff00ffu) ^ 0x64806480u);
        odd = debias(((x >> 8) & 0x00ff00ffu) ^ 0x64806480u);
    }
    __device__ __forceinline__ static void k_pairs(uint32_t x, uint32_t &k0, uint32_t &k1) { even_odd(x, k0, k1); }
    __device__ __forceinline__ static float one(uint8_t c) { return (float)(int8_t)c; }
    __device__ __forceinline__ static uint8_t code(float y) {
        return (uint8_t)(int8_t)max(-127, min(127, __float2int_rn(y)));
    }
    static constexpr float kMax = 127.f;
};

// The t-th block of tokens that n new rows behind `len` ones touch, in a cache
// whose tables hold `cap` rows a sequence: new rows [first, last) (positions in
// the sequence; none when last <= first, or past the cap, where rows have no
// place), the block's first position, its table entry and its place in the page.
struct AppendSpan {
    long long first, last, start;
    int entry, sub;
};
__host__ __device__ __forceinline__ AppendSpan append_span(int len, int n, long long cap, int t,
                                                           int page_shift, int blk_shift) {
    AppendSpan s;
    long long end = (long long)len + n;
    if (end > cap) end = cap;
    s.start = ((long long)(len >> blk_shift) + t) << blk_shift;
    s.first = s.start > len ? s.start : len;
    s.last = s.start + (1LL << blk_shift);
    if (s.last > end) s.last = end;
    s.entry = (int)(s.start >> page_shift);
    s.sub = (int)(s.start & ((1LL << page_shift) - 1)) >> blk_shift;
    return s;
}

// The keys that some row of a sequence attends to, [lo, hi) (0, 0 without any):
// the union of legal_range over its Qb rows.
__host__ __device__ __forceinline__ void unit_keys(int Qb, int Kb, int window, int mask, int &lo,
                                                   int &hi) {
    lo = hi = 0;
    if (Qb <= 0 || Kb <= 0) return;
    hi = mask == 1 && Qb < Kb ? Qb : Kb;
    // bottom-right causal: the first row with a key is max(0, Qb - Kb)
    if (mask == 0 && window > 0 && Kb - Qb - window + 1 > 0) lo = Kb - Qb - window + 1;
}

// The smallest power of two s >= 2^-100 with a <= qmax * s, for a >= 0; NaN when
// a is infinite or NaN.
__host__ __device__ __forceinline__ float append_scale(float a, int code) {
    union {
        float f;
        uint32_t u;
    } x, m;
    x.f = a;
    m.u = 0x7fc00000u;
    if (!(a <= 3.402823466e38f)) return m.f;
    // 2^ea <= a < 2^(ea + 1): with qmax 448 = 1.75 * 2^8 or 127 = 1.984375 * 2^6
    // the exponent is ea - 8 or ea - 7, resp. ea - 6 or ea - 5
    int e = (int)(x.u >> 23) - 127 - (code == kCodeE4m3 ? 8 : 6);
    if (e < -100) e = -100;
    m.u = (uint32_t)(e + 127) << 23;
    if (a > (code == kCodeE4m3 ? 448.f : 127.f) * m.f) m.u += 1u << 23;
    return m.f;
}

}  // namespace attn
