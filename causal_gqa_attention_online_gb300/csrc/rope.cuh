// rope.cuh -- the position rotation: its arguments, and the pieces that the kernels
// for 16- and 32-bit rows and for the 8-bit cache share.
//
// The first `rot` columns of a head are pairs (x1, x2) -- columns i and i + rot / 2
// ("half"), or 2 i and 2 i + 1 ("adjacent") -- turned by the angle of the row's
// position and of the pair,
//
//     y1 = x1 c - x2 s,   y2 = x2 c + x1 s,   c = cos[pos, i],  s = sin[pos, i];
//
// the other columns stay.  The transpose, which takes gradients of y to gradients of
// x, is the same with -s.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace attn {

struct RopeArgs {
    const void *q, *k, *v;      // new rows (q, v may be null)
    void *qo, *ko, *vo;         // q and, without pages, k: rows; with pages: the pools
    long long q_stride, k_stride, v_stride;  // elements between the rows of two tokens
    const float *cos, *sin;     // [max_pos][rot / 2]
    int max_pos, rot, adjacent;
    float sign;                 // 1, or -1 for the transpose
    const int32_t *positions;   // of each row, or null: the row's place in its sequence
    int B, N, Hq, Hkv, D, Dv;
    // pages (block_table != null): as AppendArgs of the 8-bit cache
    const int32_t *cu;          // packed rows: sequence b owns rows [cu[b], cu[b + 1])
    long long total;            // packed rows in all
    const int32_t *seqlens_new, *seqlens_k, *block_table;
    int max_pages, page_shift, num_pages;
    int *status;                // device status word
    unsigned long long wait_ns; // limit of a wait for a copy
};

// Sequence b's rows: the first one in the buffers, how many are real, and how many
// rows of the cache come before them.
struct RopeSeq {
    long long row0;
    int n, len;
};
__device__ __forceinline__ RopeSeq rope_seq(const RopeArgs &a, int b) {
    RopeSeq s;
    s.len = a.seqlens_k ? clamp_len(__ldg(a.seqlens_k + b), (int)((long long)a.max_pages << a.page_shift)) : 0;
    if (a.cu != nullptr) {
        s.row0 = max(0, __ldg(a.cu + b));
        s.n = clamp_len((int)min((long long)__ldg(a.cu + b + 1), a.total) - (int)s.row0, a.N);
    } else {
        s.row0 = (long long)b * a.N;
        s.n = a.seqlens_new ? clamp_len(__ldg(a.seqlens_new + b), a.N) : a.N;
    }
    return s;
}

// Position of row i of a sequence; -1 outside the table (the row becomes NaN).
__device__ __forceinline__ int rope_position(const RopeArgs &a, const RopeSeq &s, int i) {
    const long long p = a.positions ? (long long)__ldg(a.positions + s.row0 + i) : (long long)s.len + i;
    return p >= 0 && p < a.max_pos ? (int)p : -1;
}

// Row of the pools for position j of sequence b, or -1 (no page, or past the table).
__device__ __forceinline__ long long rope_cache_row(const RopeArgs &a, int b, long long j) {
    if (j >= ((long long)a.max_pages << a.page_shift)) return -1;
    const int page = __ldg(a.block_table + (long long)b * a.max_pages + (int)(j >> a.page_shift));
    if (page < 0 || page >= a.num_pages) return -1;
    return ((long long)page << a.page_shift) + (j & ((1LL << a.page_shift) - 1));
}

// The two values of a pair.  Each product and each sum is rounded by itself (no
// fused multiply-add), so that an fp32 program written with elementary operations
// gives the same bits, and with them the same 8-bit codes.
__device__ __forceinline__ void turn(float &x1, float &x2, float c, float s) {
    const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
    x2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    x1 = y1;
}

// The products of two pairs an instruction.  (The sums stay single: packed sums of packed
// products were seen to be fused with them, .rn or not.)
__device__ __forceinline__ void mul_f2(float a0, float a1, float b0, float b1, float &r0, float &r1) {
    asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
        " mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
        : "=f"(r0), "=f"(r1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// VEC elements as one access.
template <typename T, int VEC> struct RowVec {
    static constexpr int BYTES = (int)sizeof(T) * VEC;
    alignas(BYTES) T x[VEC];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (BYTES == 16) {
            *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(p);
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2 *>(x) = *reinterpret_cast<const uint2 *>(p);
        } else {
            x[0] = *p;
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (BYTES == 16) {
            *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(x);
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(x);
        } else {
            *p = x[0];
        }
    }
    // from fp32, rounded once
    __device__ __forceinline__ void set(const float *y) {
        if constexpr (sizeof(T) == 2 && VEC > 1) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                if constexpr (std::is_same_v<T, __nv_bfloat16>)
                    *reinterpret_cast<__nv_bfloat162 *>(x + i) = __floats2bfloat162_rn(y[i], y[i + 1]);
                else
                    *reinterpret_cast<__half2 *>(x + i) = __floats2half2_rn(y[i], y[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i] = from_f32<T>(y[i]);
        }
    }
};

// A head's columns as items of two vectors: item c < rot / (2 VEC) holds VEC pairs,
// the others plain columns (one element each where VEC is 1).
template <int VEC> struct RopeItem {
    int a, b;      // first column of either vector
    int trig;      // first pair, or -1: plain columns
};
template <int VEC, bool ADJ> __device__ __forceinline__ RopeItem<VEC> rope_item(int c, int rot) {
    RopeItem<VEC> it;
    const int nrot = rot / (2 * VEC);
    if (c < nrot) {
        it.trig = c * VEC;
        it.a = ADJ ? 2 * c * VEC : c * VEC;
        it.b = ADJ ? it.a + VEC : it.a + rot / 2;
    } else {
        it.trig = -1;
        it.a = rot + (c - nrot) * (VEC == 1 ? 1 : 2 * VEC);
        it.b = VEC == 1 ? it.a : it.a + VEC;
    }
    return it;
}
template <int VEC> __host__ __device__ __forceinline__ int rope_items(int D, int rot) {
    return rot / (2 * VEC) + (VEC == 1 ? D - rot : (D - rot) / (2 * VEC));
}

// cos and sin of an item's pairs (NaN where the position is not in the table).
template <int VEC> struct Trig {
    float c[VEC], s[VEC];
    __device__ __forceinline__ void set_nan() {
#pragma unroll
        for (int i = 0; i < VEC; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
    }
    // from shared memory (VEC a multiple of 4)
    __device__ __forceinline__ void load_from(const float *cs, const float *sn, float sign) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(cs + i);
            const float4 y = *reinterpret_cast<const float4 *>(sn + i);
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = sign * y.x, s[i + 1] = sign * y.y, s[i + 2] = sign * y.z, s[i + 3] = sign * y.w;
        }
    }
    __device__ __forceinline__ void load(const RopeArgs &a, int pos, int pair) {
        if (pair < 0) return;
        if (pos < 0) {
            set_nan();
            return;
        }
        const long long at = (long long)pos * (a.rot >> 1) + pair;
#pragma unroll
        for (int i = 0; i < VEC; i += VEC >= 4 ? 4 : 1) {
            if constexpr (VEC >= 4) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(a.cos + at + i));
                const float4 y = __ldg(reinterpret_cast<const float4 *>(a.sin + at + i));
                c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
                s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
            } else {
                c[i] = __ldg(a.cos + at + i);
                s[i] = __ldg(a.sin + at + i);
            }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[i] *= a.sign;
    }
};

// The item's values in fp32, turned: y[0 .. VEC) belong to its first vector.
template <typename T, int VEC, bool ADJ>
__device__ __forceinline__ void turn_item(const RopeItem<VEC> &it, const RowVec<T, VEC> &u,
                                          const RowVec<T, VEC> &w, const Trig<VEC> &t, float (&y)[2 * VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        y[i] = to_f32<T>(u.x[i]);
        y[VEC + i] = to_f32<T>(w.x[i]);
    }
    if (it.trig < 0) return;
    if constexpr (VEC == 1) {
        turn(y[0], y[1], t.c[0], t.s[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {  // pairs i, i + 1: at 2 i .. or in either vector
            float &p1 = y[ADJ ? 2 * i : i], &q1 = y[ADJ ? 2 * i + 2 : i + 1];
            float &p2 = y[ADJ ? 2 * i + 1 : VEC + i], &q2 = y[ADJ ? 2 * i + 3 : VEC + i + 1];
            float pc, qc, ps, qs, p2c, q2c, p1s, q1s;
            mul_f2(p1, q1, t.c[i], t.c[i + 1], pc, qc);
            mul_f2(p2, q2, t.s[i], t.s[i + 1], ps, qs);
            mul_f2(p2, q2, t.c[i], t.c[i + 1], p2c, q2c);
            mul_f2(p1, q1, t.s[i], t.s[i + 1], p1s, q1s);
            p1 = __fsub_rn(pc, ps);
            q1 = __fsub_rn(qc, qs);
            p2 = __fadd_rn(p2c, p1s);
            q2 = __fadd_rn(q2c, q1s);
        }
    }
}

constexpr int kRopeThreads = 256;  // the most of a block
constexpr int kRopeUnroll = 4;     // heads whose loads a thread has in flight

struct RopeShape {
    int items;    // of a head
    int lanes;    // min(items, threads)
    int heads;    // heads of a token that its threads take at a time
    int tokens;   // of a block
    int threads;  // of a block
};

// Many rows: a thread takes up to kRopeUnroll heads, so that what a token costs once (its
// place, its angles) is spread over them.  Few rows (`wide`): as many threads a token as it
// has work for.  `most`: threads of a block.
template <int VEC> RopeShape rope_shape(const RopeArgs &a, bool wide, int most) {
    RopeShape g;
    g.items = rope_items<VEC>(a.D, a.rot);
    g.lanes = g.items < most ? g.items : most;
    int heads = (a.qo ? a.Hq : 0) + (a.ko ? a.Hkv : 0);
    if (!wide) heads = (heads + kRopeUnroll - 1) / kRopeUnroll;
    g.heads = most / g.lanes;
    if (g.heads > heads) g.heads = heads > 0 ? heads : 1;
    g.tokens = wide ? 1 : most / (g.lanes * g.heads);
    if (g.tokens > a.N) g.tokens = a.N;
    g.threads = (g.lanes * g.heads * g.tokens + 31) / 32 * 32;
    return g;
}

// Heads h0, h0 + step, ... of one row: the item `it` of each.
template <typename T, int VEC, bool ADJ>
__device__ __forceinline__ void rope_heads(const T *src, T *dst, int h0, int heads, int step, int D,
                                           const RopeItem<VEC> &it, const Trig<VEC> &tr) {
    for (int h = h0; h < heads; h += step * kRopeUnroll) {
        RowVec<T, VEC> u[kRopeUnroll], w[kRopeUnroll];
        const T *from = src + h * D;
#pragma unroll
        for (int j = 0; j < kRopeUnroll; ++j) {
            if (h + j * step >= heads) break;
            u[j].load(from + j * step * D + it.a);
            w[j].load(from + j * step * D + it.b);
        }
        T *to = dst + h * D;
#pragma unroll
        for (int j = 0; j < kRopeUnroll; ++j) {
            if (h + j * step >= heads) break;
            if (it.trig >= 0) {
                float y[2 * VEC];
                turn_item<T, VEC, ADJ>(it, u[j], w[j], tr, y);
                u[j].set(y);
                w[j].set(y + VEC);
            }
            u[j].store(to + j * step * D + it.a);
            if (VEC > 1 || it.trig >= 0) w[j].store(to + j * step * D + it.b);
        }
    }
}

// Rows [bx * tokens, ...) of sequence ub, by the threads of a block.
template <typename T, int VEC, bool ADJ, bool PAGED>
__device__ __forceinline__ void rope_rows(const RopeArgs &a, const RopeShape &g, uint32_t bx, uint32_t ub) {
    const int per = g.lanes * g.heads;  // threads of a token
    const int slot = threadIdx.x / per, t = threadIdx.x - slot * per;
    const long long i64 = (long long)bx * g.tokens + slot;
    if (slot >= g.tokens || ub >= (uint32_t)a.B || i64 >= a.N) return;
    const int b = (int)ub, i = (int)i64;
    const RopeSeq sq = rope_seq(a, b);
    T *qo = static_cast<T *>(a.qo);
    const long long row = sq.row0 + i;
    if (i >= sq.n) {
        // a padded row (packed ones do not exist): +0, as attention gives
        if (a.cu == nullptr && qo != nullptr) {
            RowVec<T, VEC> z;
#pragma unroll
            for (int e = 0; e < VEC; ++e) z.x[e] = from_f32<T>(0.f);
            for (int e = t; e < a.Hq * a.D / VEC; e += per) z.store(qo + row * a.Hq * a.D + (long long)e * VEC);
        }
        return;
    }
    const int pos = rope_position(a, sq, i);
    T *ko = static_cast<T *>(a.ko), *vo = static_cast<T *>(a.vo);
    long long krow = row;
    if (PAGED) krow = rope_cache_row(a, b, (long long)sq.len + i);
    if (a.v != nullptr && krow >= 0) {  // a row of V: one run of vectors on both sides
        const T *vr = static_cast<const T *>(a.v) + row * a.v_stride;
        T *to = vo + krow * a.Hkv * a.Dv;
        const int n = a.Hkv * a.Dv / VEC;
        for (int e = t; e < n; e += per * kRopeUnroll) {
            RowVec<T, VEC> x[kRopeUnroll];
#pragma unroll
            for (int u = 0; u < kRopeUnroll; ++u)
                if (e + u * per < n) x[u].load(vr + (long long)(e + u * per) * VEC);
#pragma unroll
            for (int u = 0; u < kRopeUnroll; ++u)
                if (e + u * per < n) x[u].store(to + (long long)(e + u * per) * VEC);
        }
    }
    const int head0 = t / g.lanes;
    for (int c = t - head0 * g.lanes; c < g.items; c += g.lanes) {
        const RopeItem<VEC> it = rope_item<VEC, ADJ>(c, a.rot);
        Trig<VEC> tr;
        tr.load(a, pos, it.trig);
        if (qo != nullptr)
            rope_heads<T, VEC, ADJ>(static_cast<const T *>(a.q) + row * a.q_stride, qo + row * a.Hq * a.D, head0, a.Hq,
                               g.heads, a.D, it, tr);
        // (k's heads go on where q's end, so that no thread has one more of both)
        if (ko != nullptr && krow >= 0) {
            int h = head0;
            if (qo != nullptr) {
                h -= a.Hq % g.heads;
                if (h < 0) h += g.heads;
            }
            rope_heads<T, VEC, ADJ>(static_cast<const T *>(a.k) + row * a.k_stride, ko + krow * a.Hkv * a.D, h, a.Hkv,
                               g.heads, a.D, it, tr);
        }
    }
}

}  // namespace attn
