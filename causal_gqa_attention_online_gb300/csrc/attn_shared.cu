// attn_shared.cu -- the C ABI of attention over paged keys that sequences share.
// Declaration and contract: include/attn_gqa.h.
#include <cmath>
#include <cstring>

#include "attn_gqa.h"
#include "common.cuh"
#include "launch.h"

using namespace attn;

extern "C" int attn_fwd_paged_shared(const void *q, const void *k_pages, const void *v_pages,
                                     void *o, float *lse, int B, int Hq, int Hkv, int Q, int D,
                                     int Dv, const int32_t *block_table, int max_pages,
                                     int page_size, int num_pages, const int32_t *seqlens_q,
                                     const int32_t *seqlens_k, const int32_t *cu_groups,
                                     const int32_t *shared_lens, int num_groups, float scale,
                                     int dtype, int algo, attn_stream_t stream) {
    clear_error();
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
    const int K = max_pages * page_size;  // key capacity of a sequence
    int rc = validate(q, k_pages, v_pages, o, lse, B, Hq, Hkv, Q, K, D, Dv, dtype, algo);
    if (rc) return rc;
    if (num_groups < 0 || num_groups >= (1 << 30)) {
        set_error("bad number of groups (%d)", num_groups);
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
    if (num_groups > 0 && (cu_groups == nullptr || shared_lens == nullptr)) {
        set_error("groups need cu_groups and shared_lens");
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
    p.block_table = block_table;
    p.page_size = page_size;
    while ((1 << p.page_shift) < page_size) ++p.page_shift;
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.nsplit = 1;
    p.split_len = K > 0 ? K : 1;
    p.wait_ns = wait_limit_ns();
    const bool tc = shared_tc_supported(p, dtype);
    if (algo == ATTN_ALGO_TCGEN05 && !tc) {
        set_error("the shared-prefix kernel takes bf16/fp16, D and Dv multiples of 16 in [64, 128], "
                  "Hq / Hkv <= 128, pages of 8 rows or more, and fewer than 2^30 rows and keys");
        return ATTN_ERR_UNSUPPORTED;
    }
    // the other kernels read every sequence's own table; without groups nothing is shared
    if (algo != ATTN_ALGO_TCGEN05 && (algo != ATTN_ALGO_AUTO || !tc || num_groups == 0))
        return run_forward(p, dtype, algo, reinterpret_cast<cudaStream_t>(stream));
    int dev = 0;
    rc = current_device(&dev);
    if (rc == 0) rc = status_ptr(dev, &p.status);
    if (rc) return rc;
    const int nsm = sm_count(dev);
    return with_workspace(shared_tc_workspace(p, num_groups, nsm),
                          reinterpret_cast<cudaStream_t>(stream), [&](void *ws) {
        return launch_shared_tc(p, cu_groups, shared_lens, num_groups, dtype, nsm, ws,
                                reinterpret_cast<cudaStream_t>(stream));
    });
}
