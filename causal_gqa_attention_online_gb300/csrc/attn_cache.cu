// attn_cache.cu -- the C ABI of the 8-bit paged K/V cache: appending rows,
// attention over it, and copying, forking and compacting its pages.
// Declarations and contracts: include/attn_gqa.h.
#include <cmath>
#include <cstring>

#include "attn_gqa.h"
#include "common.cuh"
#include "launch.h"
#include "q8.cuh"

namespace attn {

int validate_cache(const void *k_pages, const void *v_pages, const float *k_scale,
                   const float *v_scale, int Hkv, int D, int Dv, int max_pages, int page_size,
                   int num_pages, int block_size, int cache_dtype) {
    if (page_size < 1 || page_size > (1 << 20) || (page_size & (page_size - 1)) != 0) {
        set_error("page_size must be a power of two in [1, 2^20] (got %d)", page_size);
        return ATTN_ERR_INVALID;
    }
    if (block_size < 1 || block_size > page_size || (block_size & (block_size - 1)) != 0) {
        set_error("block_size must be a power of two in [1, page_size = %d] (got %d)", page_size,
                  block_size);
        return ATTN_ERR_INVALID;
    }
    if (num_pages < 1 || max_pages < 0 || (long long)num_pages * page_size >= (1LL << 31) ||
        (long long)max_pages * page_size >= (1LL << 31)) {
        set_error("bad page counts (num_pages=%d max_pages=%d page_size=%d)", num_pages,
                  max_pages, page_size);
        return ATTN_ERR_INVALID;
    }
    if (cache_dtype != ATTN_CACHE_E4M3 && cache_dtype != ATTN_CACHE_INT8) {
        set_error("unknown cache dtype %d", cache_dtype);
        return ATTN_ERR_INVALID;
    }
    if (Hkv < 1 || D < 1 || D > 512 || Dv < 1 || Dv > 512) {
        set_error("head widths must be in [1, 512] and Hkv positive (Hkv=%d D=%d Dv=%d)", Hkv, D,
                  Dv);
        return ATTN_ERR_INVALID;
    }
    if ((long long)Hkv * (D > Dv ? D : Dv) >= (1LL << 31)) {
        set_error("a token's heads have 2^31 or more elements (Hkv=%d D=%d Dv=%d)", Hkv, D, Dv);
        return ATTN_ERR_INVALID;
    }
    if (k_pages == nullptr || v_pages == nullptr || k_scale == nullptr || v_scale == nullptr) {
        set_error("k_pages, v_pages, k_scale and v_scale must be non-null");
        return ATTN_ERR_INVALID;
    }
    if (!ptr_aligned16(k_pages) || !ptr_aligned16(v_pages) || !ptr_aligned16(k_scale) ||
        !ptr_aligned16(v_scale)) {
        set_error("cache pointers must be 16-byte aligned");
        return ATTN_ERR_INVALID;
    }
    return ATTN_OK;
}

namespace {

constexpr int kMaxCount = 1 << 30;  // pages of a pool and slots of a table, in the plans

int log2_of(long long n) {  // n a power of two
    int s = 0;
    while ((1LL << s) < n) ++s;
    return s;
}

int append_common(const void *k, const void *v, void *k_pages, void *v_pages, float *k_scale,
                  float *v_scale, int B, int N, long long total, int Hkv, int D, int Dv,
                  const int32_t *seqlens_new, const int32_t *cu_new, const int32_t *seqlens_k,
                  const int32_t *block_table, int max_pages, int page_size, int num_pages,
                  int block_size, int cache_dtype, int dtype, cudaStream_t stream) {
    if (B < 0 || N < 0) {
        set_error("negative size (B=%d N=%d)", B, N);
        return ATTN_ERR_INVALID;
    }
    if (dtype < ATTN_F32 || dtype > ATTN_BF16) {
        set_error("unknown dtype %d", dtype);
        return ATTN_ERR_INVALID;
    }
    int rc = validate_cache(k_pages, v_pages, k_scale, v_scale, Hkv, D, Dv, max_pages, page_size,
                            num_pages, block_size, cache_dtype);
    if (rc) return rc;
    if (B == 0 || N == 0 || max_pages == 0 || (cu_new != nullptr && total == 0)) return ATTN_OK;
    if (k == nullptr || v == nullptr || seqlens_k == nullptr || block_table == nullptr) {
        set_error("k, v, seqlens_k and block_table must be non-null");
        return ATTN_ERR_INVALID;
    }
    if (!ptr_aligned16(k) || !ptr_aligned16(v)) {
        set_error("tensor pointers must be 16-byte aligned");
        return ATTN_ERR_INVALID;
    }
    return launch_cache_append(k, v, k_pages, v_pages, k_scale, v_scale, B, N, Hkv, D, Dv,
                               seqlens_new, cu_new, total, seqlens_k, block_table, max_pages,
                               log2_of(page_size), num_pages, page_size / block_size,
                               log2_of(block_size), cache_dtype, dtype, stream);
}

// Bytes of expanded keys and values that one group of sequences may take (a
// longer sequence than this is a group of its own).  Larger groups fill the
// prefill's grid better: four sequences of up to 8192 keys (134 MB) take one
// launch of 256 units instead of two of 128, half of them over a short tail.
constexpr long long kExpandBytes = 512LL << 20;

// Attention over contiguous 16- or 32-bit copies of the keys and values, for
// problems the 8-bit kernels do not take: groups of sequences one after the
// other, in one workspace.
int run_expanded(const AttnParams &p, const Q8Cache &c, int dtype, int algo, cudaStream_t stream) {
    int dev = 0;
    int rc = current_device(&dev);
    if (rc) return rc;
    cudaMemPool_t pool = nullptr;
    rc = pool_for(dev, &pool);
    if (rc) return rc;
    const long long es = dtype == ATTN_F32 ? 4 : 2;
    const long long kb = (long long)p.K * p.Hkv * p.D * es, vb = (long long)p.K * p.Hkv * p.Dv * es;
    long long group = kExpandBytes / (kb + vb > 0 ? kb + vb : 1);
    if (group < 1) group = 1;
    // every group's rows of q and o start on a 16-byte boundary
    const bool odd = (p.Q * (long long)p.Hq * p.D * es) % 16 || (p.Q * (long long)p.Hq * p.Dv * es) % 16;
    const long long unit = odd ? 8 : 1;
    group = (group + unit - 1) / unit * unit;
    // (the grids of the expansion and of the CUDA-core kernel)
    const long long most = 65535 / p.Hkv / unit * unit;
    if (group > most) group = most > 0 ? most : unit;
    if (group > p.B) group = p.B;
    // the values start on a 256-byte boundary
    const long long v_at = (group * kb + 255) / 256 * 256;
    void *ws = nullptr;
    const size_t bytes = (size_t)(v_at + group * vb);
    cudaError_t e = cudaMallocFromPoolAsync(&ws, bytes > 0 ? bytes : 256, pool, stream);
    if (e != cudaSuccess) {
        set_error("workspace cudaMallocFromPoolAsync(%zu): %s", bytes, cudaGetErrorString(e));
        return ATTN_ERR_CUDA;
    }
    char *kx = static_cast<char *>(ws), *vx = kx + v_at;
    for (long long b0 = 0; b0 < p.B && rc == 0; b0 += group) {
        AttnParams g = p;
        g.B = (int)(p.B - b0 < group ? p.B - b0 : group);
        g.q = static_cast<const char *>(p.q) + b0 * p.Q * p.Hq * p.D * es;
        g.o = static_cast<char *>(p.o) + b0 * p.Q * p.Hq * p.Dv * es;
        g.lse = p.lse ? p.lse + b0 * p.Q * p.Hq : nullptr;
        g.seqlens_q = p.seqlens_q ? p.seqlens_q + b0 : nullptr;
        g.seqlens_k = p.seqlens_k + b0;
        g.block_table = p.block_table + b0 * p.max_pages;
        rc = launch_q8_expand(g, c, kx, vx, dtype, stream);
        if (rc) break;
        g.k = kx;
        g.v = vx;
        g.block_table = nullptr;
        g.Tq = (long long)g.B * g.Q;
        g.Tk = (long long)g.B * g.K;
        rc = run_forward(g, dtype, algo, stream);
    }
    e = cudaFreeAsync(ws, stream);
    if (e != cudaSuccess && rc == 0) {
        set_error("workspace cudaFreeAsync: %s", cudaGetErrorString(e));
        rc = ATTN_ERR_CUDA;
    }
    return rc;
}

int validate_pools(const void *const *src, void *const *dst, const long long *bytes, int n,
                   const char *what) {
    if (n < 0 || (n > 0 && (src == nullptr || dst == nullptr || bytes == nullptr))) {
        set_error("%s: npools (%d) must not be negative, and its arrays non-null", what, n);
        return ATTN_ERR_INVALID;
    }
    for (int i = 0; i < n; ++i) {
        if (bytes[i] < 1) {
            set_error("%s: pool %d has pages of %lld bytes", what, i, bytes[i]);
            return ATTN_ERR_INVALID;
        }
        if (src[i] == nullptr || dst[i] == nullptr) {
            set_error("%s: pool %d is null", what, i);
            return ATTN_ERR_INVALID;
        }
    }
    return ATTN_OK;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_cache_append(const void *k, const void *v, void *k_pages, void *v_pages, float *k_scale,
                      float *v_scale, int B, int N, int Hkv, int D, int Dv,
                      const int32_t *seqlens_new, const int32_t *seqlens_k,
                      const int32_t *block_table, int max_pages, int page_size, int num_pages,
                      int block_size, int cache_dtype, int dtype, attn_stream_t stream) {
    clear_error();
    return append_common(k, v, k_pages, v_pages, k_scale, v_scale, B, N, (long long)B * N, Hkv, D,
                         Dv, seqlens_new, nullptr, seqlens_k, block_table, max_pages, page_size,
                         num_pages, block_size, cache_dtype, dtype,
                         reinterpret_cast<cudaStream_t>(stream));
}

int attn_cache_append_varlen(const void *k, const void *v, void *k_pages, void *v_pages,
                             float *k_scale, float *v_scale, int B, int total_new, int max_new,
                             int Hkv, int D, int Dv, const int32_t *cu_seqlens_new,
                             const int32_t *seqlens_k, const int32_t *block_table, int max_pages,
                             int page_size, int num_pages, int block_size, int cache_dtype,
                             int dtype, attn_stream_t stream) {
    clear_error();
    if (total_new < 0) {
        set_error("negative size (total_new=%d)", total_new);
        return ATTN_ERR_INVALID;
    }
    if (B > 0 && cu_seqlens_new == nullptr) {
        set_error("cu_seqlens_new must be non-null");
        return ATTN_ERR_INVALID;
    }
    return append_common(k, v, k_pages, v_pages, k_scale, v_scale, B, max_new, total_new, Hkv, D,
                         Dv, nullptr, cu_seqlens_new, seqlens_k, block_table, max_pages, page_size,
                         num_pages, block_size, cache_dtype, dtype,
                         reinterpret_cast<cudaStream_t>(stream));
}

int attn_fwd_paged_q8(const void *q, const void *k_pages, const void *v_pages,
                      const float *k_scale, const float *v_scale, void *o, float *lse, int B,
                      int Hq, int Hkv, int Q, int D, int Dv, const int32_t *block_table,
                      int max_pages, int page_size, int num_pages, int block_size,
                      int cache_dtype, const int32_t *seqlens_q, const int32_t *seqlens_k,
                      int window, float scale, int mask, int dtype, int algo,
                      attn_stream_t stream) {
    clear_error();
    int rc = validate_cache(k_pages, v_pages, k_scale, v_scale, Hkv, D, Dv, max_pages, page_size,
                            num_pages, block_size, cache_dtype);
    if (rc) return rc;
    const int K = max_pages * page_size;  // key capacity of a sequence
    rc = validate(q, k_pages, v_pages, o, lse, B, Hq, Hkv, Q, K, D, Dv, dtype, algo);
    if (rc) return rc;
    if (mask < ATTN_MASK_CAUSAL || mask > ATTN_MASK_NONE) {
        set_error("unknown mask %d", mask);
        return ATTN_ERR_INVALID;
    }
    if (mask == ATTN_MASK_NONE && window > 0) {
        set_error("a window needs a causal mask (window=%d with ATTN_MASK_NONE)", window);
        return ATTN_ERR_INVALID;
    }
    if (!std::isfinite(scale)) {
        set_error("the scale must be finite (got %g)", (double)scale);
        return ATTN_ERR_INVALID;
    }
    if ((long long)B * Q * Hq == 0) return ATTN_OK;
    if ((max_pages > 0 && block_table == nullptr) || seqlens_k == nullptr) {
        set_error("paged K/V needs block_table and seqlens_k");
        return ATTN_ERR_INVALID;
    }
    AttnParams p;
    memset(&p, 0, sizeof(p));
    p.q = q;
    p.k = k_pages;
    p.v = v_pages;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.Q = Q;
    p.K = K;
    p.Tq = (long long)B * Q;
    p.Tk = (long long)num_pages * page_size;
    p.D = D;
    p.Dv = Dv;
    p.seqlens_q = seqlens_q;
    p.seqlens_k = seqlens_k;
    p.window = (window <= 0 || window >= K) ? 0 : window;
    p.mask = mask;
    p.block_table = block_table;
    p.page_size = page_size;
    p.page_shift = log2_of(page_size);
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.nsplit = 1;
    p.split_len = K > 0 ? K : 1;
    p.wait_ns = wait_limit_ns();
    Q8Cache c;
    c.k = static_cast<const uint8_t *>(k_pages);
    c.v = static_cast<const uint8_t *>(v_pages);
    c.ks = k_scale;
    c.vs = v_scale;
    c.code = cache_dtype;
    c.nblk = page_size / block_size;
    c.blk_shift = log2_of(block_size);
    // few rows read the codes; ATTN_ALGO_DECODE is that kernel, the others' names
    // choose among the kernels that read the expanded rows
    const bool decode = q8_decode_supported(p, dtype);
    if (algo == ATTN_ALGO_DECODE && !decode) {
        set_error("the 8-bit decode kernel takes bf16/fp16, Q * Hq / Hkv <= 1024, D and Dv multiples of "
                  "16 up to 256 and pages of 8 rows or more");
        return ATTN_ERR_UNSUPPORTED;
    }
    int dev = 0;
    rc = current_device(&dev);
    if (rc == 0) rc = status_ptr(dev, &p.status);
    if (rc) return rc;
    const int nsm = sm_count(dev);
    if (algo == ATTN_ALGO_DECODE || (algo == ATTN_ALGO_AUTO && decode && q8_decode_wins(p, nsm))) {
        return with_workspace(q8_decode_workspace(p, nsm), reinterpret_cast<cudaStream_t>(stream),
                              [&](void *ws) {
            return launch_q8_decode(p, c, dtype, nsm, ws, reinterpret_cast<cudaStream_t>(stream));
        });
    }
    return run_expanded(p, c, dtype, algo, reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_copy(const void *const *src_pools, void *const *dst_pools,
                    const long long *page_bytes, int npools, int src_pages, int dst_pages,
                    const int32_t *src, const int32_t *dst, int n, attn_stream_t stream) {
    clear_error();
    int rc = validate_pools(src_pools, dst_pools, page_bytes, npools, "attn_pages_copy");
    if (rc) return rc;
    if (n < 0 || src_pages < 0 || dst_pages < 0) {
        set_error("attn_pages_copy: negative size (n=%d src_pages=%d dst_pages=%d)", n, src_pages,
                  dst_pages);
        return ATTN_ERR_INVALID;
    }
    if (n == 0 || npools == 0) return ATTN_OK;
    if (src == nullptr || dst == nullptr) {
        set_error("attn_pages_copy: src and dst must be non-null");
        return ATTN_ERR_INVALID;
    }
    return launch_pages_copy(src_pools, dst_pools, page_bytes, npools, src_pages, dst_pages, src,
                             dst, n, reinterpret_cast<cudaStream_t>(stream));
}

int attn_pages_fork(void *const *pools, const long long *page_bytes, int npools,
                    const int32_t *block_table, const int32_t *seqlens, const int32_t *refcount,
                    int S, int max_pages, int num_pages, int page_size, const int32_t *parents,
                    const int32_t *new_tokens, int N, int32_t *block_table_out,
                    int32_t *seqlens_out, int32_t *refcount_out, int32_t *status,
                    attn_stream_t stream) {
    clear_error();
    int rc = validate_pools(const_cast<const void *const *>(pools), pools, page_bytes, npools,
                            "attn_pages_fork");
    if (rc) return rc;
    if (page_size < 1 || page_size > (1 << 20) || (page_size & (page_size - 1)) != 0) {
        set_error("page_size must be a power of two in [1, 2^20] (got %d)", page_size);
        return ATTN_ERR_INVALID;
    }
    // (slots and pages are stepped through in 32 bits)
    if (S < 0 || N < 0 || max_pages < 0 || num_pages < 1 || N > kMaxCount || num_pages > kMaxCount ||
        (long long)max_pages * page_size >= (1LL << 31)) {
        set_error("attn_pages_fork: bad sizes (S=%d N=%d max_pages=%d num_pages=%d page_size=%d)",
                  S, N, max_pages, num_pages, page_size);
        return ATTN_ERR_INVALID;
    }
    if (refcount == nullptr || refcount_out == nullptr || status == nullptr ||
        (S > 0 && (seqlens == nullptr || (max_pages > 0 && block_table == nullptr))) ||
        (N > 0 && (parents == nullptr || seqlens_out == nullptr ||
                   (max_pages > 0 && block_table_out == nullptr)))) {
        set_error("attn_pages_fork: null pointer");
        return ATTN_ERR_INVALID;
    }
    if (refcount == refcount_out || (block_table != nullptr && block_table == block_table_out) ||
        (seqlens != nullptr && seqlens == seqlens_out)) {
        set_error("attn_pages_fork: the outputs are a new version and may not alias the inputs");
        return ATTN_ERR_INVALID;
    }
    return with_workspace(pages_fork_workspace(page_bytes, npools, N, max_pages, num_pages),
                          reinterpret_cast<cudaStream_t>(stream), [&](void *ws) {
        return launch_pages_fork(pools, page_bytes, npools, block_table, seqlens, refcount, S,
                                 max_pages, num_pages, log2_of(page_size), parents, new_tokens, N,
                                 block_table_out, seqlens_out, refcount_out, status, ws,
                                 reinterpret_cast<cudaStream_t>(stream));
    });
}

int attn_pages_compact(void *const *pools, const long long *page_bytes, int npools,
                       const int32_t *block_table, const int32_t *refcount, int S, int max_pages,
                       int num_pages, int32_t *block_table_out, int32_t *refcount_out,
                       int32_t *remap, int32_t *n_live, attn_stream_t stream) {
    clear_error();
    int rc = validate_pools(const_cast<const void *const *>(pools), pools, page_bytes, npools,
                            "attn_pages_compact");
    if (rc) return rc;
    if (S < 0 || max_pages < 0 || num_pages < 1 || num_pages > kMaxCount) {
        set_error("attn_pages_compact: bad sizes (S=%d max_pages=%d num_pages=%d)", S, max_pages,
                  num_pages);
        return ATTN_ERR_INVALID;
    }
    if (refcount == nullptr || refcount_out == nullptr || remap == nullptr || n_live == nullptr ||
        ((long long)S * max_pages > 0 && (block_table == nullptr || block_table_out == nullptr))) {
        set_error("attn_pages_compact: null pointer");
        return ATTN_ERR_INVALID;
    }
    if (refcount == refcount_out) {
        set_error("attn_pages_compact: refcount_out may not alias refcount");
        return ATTN_ERR_INVALID;
    }
    return with_workspace(pages_compact_workspace(page_bytes, npools, S, max_pages, num_pages),
                          reinterpret_cast<cudaStream_t>(stream), [&](void *ws) {
        return launch_pages_compact(pools, page_bytes, npools, block_table, refcount, S, max_pages,
                                    num_pages, block_table_out, refcount_out, remap, n_live, ws,
                                    reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
