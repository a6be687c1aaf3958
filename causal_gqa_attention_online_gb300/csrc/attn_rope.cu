// attn_rope.cu -- the C ABI of the position rotation: rotating rows, and appending
// rotated rows to a paged cache.  Declarations and contracts: include/attn_gqa.h.
#include "attn_gqa.h"
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"

namespace attn {
namespace {

int shift_of(int n) {  // n a power of two
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

// Checks of what every entry point has: sizes, table of angles, element addresses.
int validate_rope(const RopeArgs &a, int pairs, int dtype) {
    if (a.B < 0 || a.N < 0 || a.Hq < 0 || a.Hkv < 0 || a.max_pos < 0) {
        set_error("negative size (B=%d N=%d Hq=%d Hkv=%d positions=%d)", a.B, a.N, a.Hq, a.Hkv,
                  a.max_pos);
        return ATTN_ERR_INVALID;
    }
    if (dtype < ATTN_F32 || dtype > ATTN_BF16) {
        set_error("unknown dtype %d", dtype);
        return ATTN_ERR_INVALID;
    }
    if (pairs != ATTN_ROPE_HALF && pairs != ATTN_ROPE_ADJACENT) {
        set_error("unknown pairs %d", pairs);
        return ATTN_ERR_INVALID;
    }
    if (a.D < 1 || a.D > 512 || a.Dv < 1 || a.Dv > 512) {
        set_error("head widths must be in [1, 512] (D=%d Dv=%d)", a.D, a.Dv);
        return ATTN_ERR_INVALID;
    }
    if (a.rot < 0 || a.rot > a.D || a.rot % 2) {
        set_error("the rotated columns must be an even number up to D = %d (got %d)", a.D, a.rot);
        return ATTN_ERR_INVALID;
    }
    if ((long long)a.Hq * a.D >= (1LL << 31) || (long long)a.Hkv * (a.D > a.Dv ? a.D : a.Dv) >= (1LL << 31)) {
        set_error("a token's heads have 2^31 or more elements (Hq=%d Hkv=%d D=%d Dv=%d)", a.Hq,
                  a.Hkv, a.D, a.Dv);
        return ATTN_ERR_INVALID;
    }
    if (a.q_stride < 0 || a.k_stride < 0 || a.v_stride < 0) {
        set_error("negative row stride (q %lld k %lld v %lld)", a.q_stride, a.k_stride, a.v_stride);
        return ATTN_ERR_INVALID;
    }
    if (a.rot > 0 && a.max_pos > 0 && (a.cos == nullptr || a.sin == nullptr)) {
        set_error("cos and sin must be non-null");
        return ATTN_ERR_INVALID;
    }
    const unsigned es = dtype == ATTN_F32 ? 4 : 2;
    for (const void *p : {a.q, a.k, a.v, static_cast<const void *>(a.qo), static_cast<const void *>(a.ko),
                          static_cast<const void *>(a.vo)})
        if (reinterpret_cast<uintptr_t>(p) % es) {
            set_error("tensor pointers must be aligned to their elements");
            return ATTN_ERR_INVALID;
        }
    for (const void *p : {static_cast<const void *>(a.cos), static_cast<const void *>(a.sin),
                          static_cast<const void *>(a.positions)})
        if (reinterpret_cast<uintptr_t>(p) % 4) {
            set_error("cos, sin and positions must be aligned to their elements");
            return ATTN_ERR_INVALID;
        }
    return ATTN_OK;
}

// Whether `a` of na bytes and `b` of nb share none.
bool disjoint(const void *a, long long na, const void *b, long long nb) {
    if (a == nullptr || b == nullptr || na == 0 || nb == 0) return true;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 + (uintptr_t)na <= b0 || b0 + (uintptr_t)nb <= a0;
}

// Whether rows of `width` elements, `stride` apart, share no byte with the dense rows
// (of `out_width`) at `out`.
bool apart(const void *in, long long stride, long long width, const void *out, long long out_width,
           long long rows, int es) {
    if (rows == 0 || width == 0) return true;
    return disjoint(in, ((rows - 1) * stride + width) * es, out, rows * out_width * es);
}

int overlap_error(const char *what) {
    set_error("%s overlaps an input and is not that input's own dense rows", what);
    return ATTN_ERR_INVALID;
}

int validate_pages(int page_size, int max_pages, int num_pages) {
    if (page_size < 1 || page_size > (1 << 20) || (page_size & (page_size - 1)) != 0) {
        set_error("page_size must be a power of two in [1, 2^20] (got %d)", page_size);
        return ATTN_ERR_INVALID;
    }
    if (num_pages < 1 || max_pages < 0 || (long long)num_pages * page_size >= (1LL << 31) ||
        (long long)max_pages * page_size >= (1LL << 31)) {
        set_error("bad page counts (num_pages=%d max_pages=%d page_size=%d)", num_pages,
                  max_pages, page_size);
        return ATTN_ERR_INVALID;
    }
    return ATTN_OK;
}

// What both appends check beyond the cache itself; *none: there is nothing to do.  code_size,
// nblk: bytes of an element of the pages, blocks of scales of a page (or 0).
int validate_rows(const RopeArgs &a, const float *k_scale, const float *v_scale, int code_size, int nblk,
                  int total_new, int pairs, int dtype, bool *none) {
    *none = false;
    int rc = validate_rope(a, pairs, dtype);
    if (rc) return rc;
    if (a.cu != nullptr && total_new < 0) {
        set_error("negative size (total_new=%d)", total_new);
        return ATTN_ERR_INVALID;
    }
    if (a.Hkv < 1) {
        set_error("Hkv must be positive (got %d)", a.Hkv);
        return ATTN_ERR_INVALID;
    }
    if ((a.q == nullptr) != (a.qo == nullptr) || (a.q == nullptr) != (a.Hq == 0)) {
        set_error("q and q_out come together, and Hq is 0 without them (Hq=%d)", a.Hq);
        return ATTN_ERR_INVALID;
    }
    if (a.B == 0 || a.N == 0 || (a.cu != nullptr && total_new == 0)) {
        *none = true;
        return ATTN_OK;
    }
    if (a.k == nullptr || a.v == nullptr || a.seqlens_k == nullptr || a.block_table == nullptr) {
        set_error("k, v, seqlens_k and block_table must be non-null");
        return ATTN_ERR_INVALID;
    }
    const long long rows = a.cu ? total_new : (long long)a.B * a.N;
    const int es = dtype == ATTN_F32 ? 4 : 2;
    const long long qw = (long long)a.Hq * a.D;
    if ((!(a.q == a.qo && a.q_stride == qw) && !apart(a.q, a.q_stride, qw, a.qo, qw, rows, es)) ||
        !apart(a.k, a.k_stride, (long long)a.Hkv * a.D, a.qo, qw, rows, es) ||
        !apart(a.v, a.v_stride, (long long)a.Hkv * a.Dv, a.qo, qw, rows, es))
        return overlap_error("q_out");
    const long long out = rows * qw * es, heads = (long long)a.num_pages * a.Hkv;
    const long long scales = heads * nblk * 4, row = heads * code_size << a.page_shift;
    if (!disjoint(a.qo, out, a.ko, row * a.D) || !disjoint(a.qo, out, a.vo, row * a.Dv) ||
        !disjoint(a.qo, out, k_scale, scales) || !disjoint(a.qo, out, v_scale, scales)) {
        set_error("q_out overlaps the cache");
        return ATTN_ERR_INVALID;
    }
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_rope(const void *q, const void *k, void *q_out, void *k_out, const float *cos,
              const float *sin, int B, int N, int Hq, int Hkv, int D, int rot, int max_pos,
              long long q_stride, long long k_stride, const int32_t *positions, int pairs,
              int inverse, int dtype, attn_stream_t stream) {
    clear_error();
    RopeArgs a = {};
    a.q = q;
    a.k = k;
    a.qo = q_out;
    a.ko = k_out;
    a.cos = cos;
    a.sin = sin;
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.Dv = D;
    a.rot = rot;
    a.max_pos = max_pos;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.positions = positions;
    a.adjacent = pairs == ATTN_ROPE_ADJACENT;
    a.sign = inverse ? -1.f : 1.f;
    int rc = validate_rope(a, pairs, dtype);
    if (rc) return rc;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) ||
        (Hq > 0 && (long long)B * N > 0 && q == nullptr) || (Hkv > 0 && (long long)B * N > 0 && k == nullptr)) {
        set_error("q, k and their outputs must be non-null where there are heads (Hq=%d Hkv=%d)", Hq, Hkv);
        return ATTN_ERR_INVALID;
    }
    const long long rows = (long long)B * N;
    const int es = dtype == ATTN_F32 ? 4 : 2;
    const long long qw = (long long)Hq * D, kw = (long long)Hkv * D;
    if ((!(q == q_out && q_stride == qw) && !apart(q, q_stride, qw, q_out, qw, rows, es)) ||
        !apart(k, k_stride, kw, q_out, qw, rows, es))
        return overlap_error("q_out");
    if ((!(k == k_out && k_stride == kw) && !apart(k, k_stride, kw, k_out, kw, rows, es)) ||
        !apart(q, q_stride, qw, k_out, kw, rows, es))
        return overlap_error("k_out");
    if (!apart(q_out, qw, qw, k_out, kw, rows, es)) {
        set_error("q_out and k_out overlap");
        return ATTN_ERR_INVALID;
    }
    if (rows == 0 || Hq + (long long)Hkv == 0) return ATTN_OK;
    if (Hq == 0) a.q = a.qo = nullptr;
    if (Hkv == 0) a.k = a.ko = nullptr;
    return launch_rope(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_append(const void *q, const void *k, const void *v, void *q_out, void *k_pages,
                     void *v_pages, const float *cos, const float *sin, int B, int N,
                     int total_new, int Hq, int Hkv, int D, int Dv, int rot, int max_pos,
                     long long q_stride, long long k_stride, long long v_stride,
                     const int32_t *seqlens_new, const int32_t *cu_seqlens_new,
                     const int32_t *positions, int pairs, const int32_t *seqlens_k,
                     const int32_t *block_table, int max_pages, int page_size, int num_pages,
                     int dtype, attn_stream_t stream) {
    clear_error();
    int rc = validate_pages(page_size, max_pages, num_pages);
    if (rc) return rc;
    if (k_pages == nullptr || v_pages == nullptr) {
        set_error("k_pages and v_pages must be non-null");
        return ATTN_ERR_INVALID;
    }
    if (!ptr_aligned16(k_pages) || !ptr_aligned16(v_pages)) {
        set_error("cache pointers must be 16-byte aligned");
        return ATTN_ERR_INVALID;
    }
    RopeArgs a = {q, k, v, q_out, k_pages, v_pages, q_stride, k_stride, v_stride, cos, sin, max_pos, rot,
                  pairs == ATTN_ROPE_ADJACENT, 1.f, positions, B, N, Hq, Hkv, D, Dv, cu_seqlens_new,
                  total_new, seqlens_new, seqlens_k, block_table, max_pages, shift_of(page_size),
                  num_pages};
    bool none = false;
    rc = validate_rows(a, nullptr, nullptr, dtype == ATTN_F32 ? 4 : 2, 0, total_new, pairs, dtype, &none);
    if (rc || none) return rc;
    if (a.cu != nullptr && total_new < a.N) a.N = total_new;  // (no sequence has more)
    return launch_rope(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

int attn_rope_append_q8(const void *q, const void *k, const void *v, void *q_out, void *k_pages,
                        void *v_pages, float *k_scale, float *v_scale, const float *cos,
                        const float *sin, int B, int N, int total_new, int Hq, int Hkv, int D,
                        int Dv, int rot, int max_pos, long long q_stride, long long k_stride,
                        long long v_stride, const int32_t *seqlens_new,
                        const int32_t *cu_seqlens_new, const int32_t *positions, int pairs,
                        const int32_t *seqlens_k, const int32_t *block_table, int max_pages,
                        int page_size, int num_pages, int block_size, int cache_dtype, int dtype,
                        attn_stream_t stream) {
    clear_error();
    int rc = validate_cache(k_pages, v_pages, k_scale, v_scale, Hkv, D, Dv, max_pages, page_size,
                            num_pages, block_size, cache_dtype);
    if (rc) return rc;
    RopeArgs a = {q, k, v, q_out, k_pages, v_pages, q_stride, k_stride, v_stride, cos, sin, max_pos, rot,
                  pairs == ATTN_ROPE_ADJACENT, 1.f, positions, B, N, Hq, Hkv, D, Dv, cu_seqlens_new,
                  total_new, seqlens_new, seqlens_k, block_table, max_pages, shift_of(page_size),
                  num_pages};
    bool none = false;
    rc = validate_rows(a, k_scale, v_scale, 1, page_size / block_size, total_new, pairs, dtype, &none);
    if (rc || none) return rc;
    if (a.cu != nullptr && total_new < a.N) a.N = total_new;  // (no sequence has more)
    return launch_rope_q8(a, k_scale, v_scale, page_size / block_size, shift_of(block_size),
                          cache_dtype, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
