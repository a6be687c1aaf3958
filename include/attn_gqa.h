/*
 * attn_gqa.h -- C ABI of the GB300 (sm_103a) causal grouped-query attention
 * forward library (libattn_gqa.so).
 *
 * Operation.  Every entry point computes, for each sequence b, query head h and
 * valid query row q, the softmax attention
 *
 *     O[q,h,:] = sum_k p_k V[k,kh,:],   p_k = exp(s_k - LSE[q,h]),
 *     s_k      = scale * <Q[q,h,:], K[k,kh,:]>,
 *     LSE[q,h] = log sum_{k legal} exp(s_k)            (natural log)
 *
 * over the legal keys of the row, with kh = h / (Hq / Hkv):
 *
 *     0 <= k < Kb,   k <= q + Kb - Qb,
 *     and, when window > 0,   k >= q + Kb - Qb - window + 1.
 *
 * Sources: "Attention execution mapping: 现状、缺口与有界实验"
 * (LuisaCompute), section 1 (bottom-right causal GQA, kh = h / (Hq/Hkv),
 * legal keys k <= q + K - Q, one online-softmax program for prefill and
 * decode with row max / row sum / accumulator carried across KV blocks) and
 * section 5 (split-KV needs a legal merge of the (max, sum, acc) state);
 * "快速後端" (Laya fast backends), numerical verification (sliding window,
 * int32 per-sequence lengths, empty sequences, finite padded output).
 * The window reading (the w most recent keys including the diagonal one),
 * the empty-row convention and the natural-log LSE are this library's
 * readings where the pages are silent.
 *
 * Rows with no legal key (Kb = 0, leading rows when Qb > Kb, or a window
 * that excludes every key) return O = +0.0 and LSE = -inf.  Padded query rows
 * q >= Qb of the padded layout are written as O = +0.0 and LSE = -inf.
 *
 * Memory and ownership.  All tensor and length pointers are DEVICE pointers
 * owned by the caller; the library never frees or retains them.  Tensors are
 * dense and contiguous (row-major in the order given), 16-byte aligned.
 * Key / value rows past a sequence's length are never used as values: they
 * may hold anything, NaN included.
 *
 * Asynchrony.  Every call validates its host-side arguments, enqueues its
 * kernels on `stream` and returns; nothing synchronises.  Split-KV calls take
 * their temporary workspace from a library-owned stream-ordered pool
 * (cudaMallocAsync / cudaFreeAsync on `stream`).
 *
 * Errors.  Calls return ATTN_OK or a status below; no exception crosses the
 * ABI.  attn_last_error() gives a message for the calling thread's last
 * failure.  Device-side contract violations found by the kernels (a bounded
 * wait that ran out) are recorded in a device status word read by
 * attn_device_status().
 */
#ifndef ATTN_GQA_H
#define ATTN_GQA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *attn_stream_t;

/* Element types of q, k, v and o.  lse is always float32. */
enum attn_dtype { ATTN_F32 = 0, ATTN_F16 = 1, ATTN_BF16 = 2 };

/* Status codes. */
enum attn_status {
    ATTN_OK = 0,
    ATTN_ERR_INVALID = 1,     /* null pointer, negative size, Hq % Hkv != 0 ... */
    ATTN_ERR_UNSUPPORTED = 2, /* dtype / head-width / algorithm combination */
    ATTN_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed */
    ATTN_ERR_TIMEOUT = 4      /* a kernel's bounded wait ran out (device status) */
};

/* Kernel selection for the *_algo entry points. */
enum attn_algo {
    ATTN_ALGO_AUTO = 0,     /* choose by dtype, head widths and query length */
    ATTN_ALGO_GENERIC = 1,  /* CUDA-core online softmax: any dtype, D, Dv <= 512 */
    ATTN_ALGO_TCGEN05 = 2,  /* tcgen05/TMEM prefill: bf16/fp16, D, Dv multiples of 16 in
                               [64, 512], not paged above 128; in the backward, the
                               tcgen05 dQ and dK/dV kernels (D, Dv in [64, 128]) */
    ATTN_ALGO_DECODE = 3,   /* split-KV tensor-core decode: bf16/fp16, Q*G <= 16 */
    ATTN_ALGO_MMA = 4       /* warp-level mma.sync tensor cores, bf16/fp16: the forward for
                               D, Dv multiples of 8 up to 512 (chosen by AUTO where the
                               tcgen05 and decode kernels do not apply), the backward for
                               D, Dv multiples of 8 up to 128 */
};

/* Which keys a query row may attend to (attn_fwd_ex, attn_fwd_varlen_ex). */
enum attn_mask {
    ATTN_MASK_CAUSAL = 0,          /* bottom-right causal: key k <= q + Kb - Qb (attn_fwd's) */
    ATTN_MASK_CAUSAL_TOP_LEFT = 1, /* top-left causal: key k <= q */
    ATTN_MASK_NONE = 2             /* every key k < Kb (no window allowed) */
};

/* Element types of an 8-bit paged cache's codes (attn_cache_append). */
enum attn_cache_dtype { ATTN_CACHE_E4M3 = 0, ATTN_CACHE_INT8 = 1 };

/*
 * attn_fwd -- padded layout.
 *   q   [B, Q, Hq, D]    o   [B, Q, Hq, Dv]    lse [B, Q, Hq] (float32, may be NULL)
 *   k   [B, K, Hkv, D]   v   [B, K, Hkv, Dv]
 *   Q, K        padded capacities (query rows / key rows per sequence).
 *   seqlens_q   int32 [B] valid query rows per sequence, or NULL for all Q.
 *   seqlens_k   int32 [B] valid key rows per sequence, or NULL for all K.
 *               Values outside [0, Q] / [0, K] are clamped into range.
 *   window      > 0: keep the `window` most recent keys (diagonal included);
 *               <= 0: no window.
 *   scale       multiplies Q.K (pass 1/sqrt(D) for the usual scaling).
 *   dtype       attn_dtype of q, k, v and o.
 * Returns ATTN_OK, ATTN_ERR_INVALID (bad pointer or size, Hq % Hkv != 0,
 * D or Dv outside [1, 512]), ATTN_ERR_UNSUPPORTED or ATTN_ERR_CUDA.
 * B = 0, Q = 0 or Hq = 0 work is a successful no-op.
 */
ATTN_API int attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
             int Hkv, int Q, int K, int D, int Dv, const int32_t *seqlens_q,
             const int32_t *seqlens_k, int window, float scale, int dtype,
             attn_stream_t stream);

/*
 * attn_fwd_varlen -- packed layout.
 *   q [Tq, Hq, D]  k [Tk, Hkv, D]  v [Tk, Hkv, Dv]  o [Tq, Hq, Dv]  lse [Tq, Hq] (may be NULL)
 *   total_q, total_k   rows of the packed buffers (Tq, Tk): bounds every read
 *               and write; cu_seqlens_q[B] <= total_q, cu_seqlens_k[B] <= total_k.
 *   cu_seqlens_q, cu_seqlens_k   int32 [B+1], cu[0] = 0, non-decreasing:
 *               sequence b owns query rows [cu_q[b], cu_q[b+1]) and key rows
 *               [cu_k[b], cu_k[b+1]); an empty sequence owns none.
 *   max_Q, max_K   upper bounds of the per-sequence lengths (sizes the grid;
 *               a sequence longer than them is cut to its first max_Q query
 *               rows / max_K key rows).
 * Other arguments and return codes as attn_fwd.  Rows outside every
 * sequence are not written.
 */
ATTN_API int attn_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                    int Hq, int Hkv, int total_q, int total_k, int max_Q, int max_K, int D, int Dv,
                    const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int window,
                    float scale, int dtype, attn_stream_t stream);

/* The same two operations with an explicit kernel choice (attn_algo).  A
 * choice that cannot run the given shape returns ATTN_ERR_UNSUPPORTED. */
ATTN_API int attn_fwd_algo(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                  int Hq, int Hkv, int Q, int K, int D, int Dv, const int32_t *seqlens_q,
                  const int32_t *seqlens_k, int window, float scale, int dtype, int algo,
                  attn_stream_t stream);
ATTN_API int attn_fwd_varlen_algo(const void *q, const void *k, const void *v, void *o, float *lse,
                         int B, int Hq, int Hkv, int total_q, int total_k, int max_Q, int max_K,
                         int D, int Dv,
                         const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int window,
                         float scale, int dtype, int algo, attn_stream_t stream);

/*
 * attn_fwd_ex / attn_fwd_varlen_ex -- the two operations with an explicit
 * mask (attn_mask) and kernel choice (attn_algo).  The pages define the
 * bottom-right causal mask only; the top-left causal mask and no mask are
 * extensions of this library: the same online-softmax recurrence over a
 * different set of legal keys (a window applies to the causal masks only:
 * ATTN_MASK_NONE with window > 0 is ATTN_ERR_INVALID).
 */
ATTN_API int attn_fwd_ex(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                         int Hq, int Hkv, int Q, int K, int D, int Dv, const int32_t *seqlens_q,
                         const int32_t *seqlens_k, int window, float scale, int mask, int dtype,
                         int algo, attn_stream_t stream);
ATTN_API int attn_fwd_varlen_ex(const void *q, const void *k, const void *v, void *o, float *lse,
                                int B, int Hq, int Hkv, int total_q, int total_k, int max_Q,
                                int max_K, int D, int Dv, const int32_t *cu_seqlens_q,
                                const int32_t *cu_seqlens_k, int window, float scale, int mask,
                                int dtype, int algo, attn_stream_t stream);

/*
 * attn_lse_combine -- the legal merge of split-KV partial states (the
 * "(max, sum, acc)" merge of the LuisaCompute page, section 5), written as a
 * merge of normalised partials:
 *   o_parts   float32 [nsplit, rows, Dv]   each partial normalised by its own sum
 *   lse_parts float32 [nsplit, rows]       natural-log LSE of each partial;
 *                                          -inf marks a partial with no key
 *   o         [rows, Dv] in `dtype`;  lse [rows] float32 (may be NULL)
 *   L = log sum_s exp(lse_s);   o = sum_s exp(lse_s - L) o_s.
 * A row whose partials are all -inf gives o = +0 and lse = -inf.
 */
ATTN_API int attn_lse_combine(const float *o_parts, const float *lse_parts, void *o, float *lse,
                     int nsplit, long long rows, int Dv, int dtype, attn_stream_t stream);

/*
 * attn_lse_combine_ex -- attn_lse_combine with the partials in any storage
 * dtype: parts_dtype ATTN_F32 is attn_lse_combine; ATTN_F16 / ATTN_BF16 take
 * o_parts [nsplit, rows, Dv] in that dtype (as attn_fwd wrote them, each
 * normalised by its own sum) and need dtype == parts_dtype.  This merges the
 * outputs of one sequence's key shards computed on several GPUs and exchanged
 * as they are (the sharded decode of the Python package).  Accumulation is in
 * fp32; return codes as attn_lse_combine.
 */
ATTN_API int attn_lse_combine_ex(const void *o_parts, const float *lse_parts, void *o, float *lse,
                                 int nsplit, long long rows, int Dv, int parts_dtype, int dtype,
                                 attn_stream_t stream);

/*
 * attn_fwd_paged -- attn_fwd with the keys and values in pages: a serving
 * layout (the pages have no counterpart; the attention itself is unchanged).
 *   q [B, Q, Hq, D], o [B, Q, Hq, Dv], lse [B, Q, Hq] as in attn_fwd.
 *   k_pages [num_pages, page_size, Hkv, D], v_pages [num_pages, page_size, Hkv, Dv]:
 *               pools of pages of page_size key rows (a power of two).
 *   block_table int32 [B, max_pages] on the device: key j of sequence b is row
 *               j % page_size of page block_table[b][j / page_size].  Entries
 *               outside [0, num_pages) are clamped into it.
 *   seqlens_k   int32 [B] on the device (required), at most max_pages * page_size.
 *   mask, algo  as in attn_fwd_ex.  The tcgen05 prefill takes page sizes that
 *               are multiples of 128; the decode and fp32 kernels take any.
 * Return codes as attn_fwd.
 */
ATTN_API int attn_fwd_paged(const void *q, const void *k_pages, const void *v_pages, void *o,
                            float *lse, int B, int Hq, int Hkv, int Q, int D, int Dv,
                            const int32_t *block_table, int max_pages, int page_size,
                            int num_pages, const int32_t *seqlens_q, const int32_t *seqlens_k,
                            int window, float scale, int mask, int dtype, int algo,
                            attn_stream_t stream);

/*
 * attn_fwd_masked -- attn_fwd_ex with an arbitrary boolean mask on top of the
 * mask mode and the window: key k is legal for query row q of sequence b and
 * query head h only if it is legal under `mask` / `window` and bit k % 32 of
 * word k / 32 of mask row ((b * mask_heads + hm) * Q + q) is set, where hm = h
 * when mask_heads == Hq and hm = 0 when mask_heads == 1 (one mask shared by
 * every head).  ATTN_MASK_NONE with this mask gives a purely arbitrary mask.
 * "Attention execution mapping" (LuisaCompute), section 7, names arbitrary
 * masks as a semantic extension beyond the pages' bottom-right rule; the rest
 * of the definition (the online softmax over the legal keys, +0 / -inf for a
 * row without one) is unchanged.
 *   mask_bits   uint32 [B, mask_heads, Q, mask_words] on the device, 16-byte
 *               aligned; bits of keys at or past a sequence's length are ignored
 *   mask_words  words per row: a multiple of 4, at least 4 * ceil(K / 128)
 *   mask_heads  1 or Hq
 * Padded layout only; other arguments as attn_fwd_ex.  The tcgen05 prefill
 * (ATTN_ALGO_AUTO's choice for bf16/fp16 widths 64..128) skips 128-key tiles in
 * which no row of a work unit has an allowed key, without loading them; the
 * CUDA-core kernel (ATTN_ALGO_GENERIC, and AUTO otherwise) tests every key.
 * ATTN_ALGO_DECODE and ATTN_ALGO_MMA return ATTN_ERR_UNSUPPORTED.  Extra
 * workspace from the library's pool: ceil(K / 128) bytes per query block and
 * head group.  Return codes as attn_fwd.
 */
ATTN_API int attn_fwd_masked(const void *q, const void *k, const void *v, void *o, float *lse,
                             int B, int Hq, int Hkv, int Q, int K, int D, int Dv,
                             const int32_t *seqlens_q, const int32_t *seqlens_k,
                             const uint32_t *mask_bits, int mask_words, int mask_heads, int window,
                             float scale, int mask, int dtype, int algo, attn_stream_t stream);

/*
 * attn_fwd_decode_noalloc -- attn_fwd's split-KV decode for callers that may
 * not allocate device memory while attention runs: for example a serving
 * process whose device memory is owned by another runtime's allocator or held
 * under a hard cap, or a latency-critical decode loop where an allocation (or
 * a synchronisation it may bring) is not allowed.  The pages have no
 * counterpart to this entry point; it is a deployment aid of this library.
 *
 * Same arguments, layout and result as attn_fwd, restricted to the shapes the
 * decode kernel takes (bf16/fp16, D and Dv in {64, 128} or both 256, Q * Hq / Hkv <= 16).
 * The split-KV partials live in a fixed 32 MiB __device__ array that every
 * GPU using the library keeps until the process exits; the call makes no
 * allocation of any kind.  A problem whose partials would not fit returns
 * ATTN_ERR_UNSUPPORTED with a message giving the bytes needed.  The first
 * call on a device looks up the array's device address (make that call before
 * any stream capture).  All calls share the array: calls that overlap on the
 * GPU (other streams or host threads on the same device) race on it and must
 * be serialised by the caller.  Nothing in the array needs to start at zero.
 */
ATTN_API int attn_fwd_decode_noalloc(const void *q, const void *k, const void *v, void *o,
                                     float *lse, int B, int Hq, int Hkv, int Q, int K, int D,
                                     int Dv, const int32_t *seqlens_q, const int32_t *seqlens_k,
                                     int window, float scale, int dtype, attn_stream_t stream);

/*
 * attn_fwd_staged -- attn_fwd on tensors that live in host memory.  A
 * serving aid of this library (the pages have no counterpart): the batch is
 * cut into `chunks` groups of sequences (<= 0: 4; at most B and 32), and for
 * each group the host->device copy of its inputs, its attention launch (on
 * `stream`, exactly as attn_fwd) and the device->host copy of its outputs are
 * ordered by events across three streams, so the copies of one group overlap
 * the attention of another.
 *   hq, hk, hv, ho, hlse   host tensors, padded layout as in attn_fwd (hlse
 *                          may be NULL); page-locked memory is needed for the
 *                          copies to overlap anything
 *   q, k, v, o, lse        caller-owned device buffers of the same shapes,
 *                          used as staging (lse may be NULL only with hlse)
 *   seqlens_q, seqlens_k   as in attn_fwd (device int32 [B] or NULL), and
 *   seqlens_q_host, seqlens_k_host  the same values in host memory (NULL
 *                          exactly when the device array is NULL): only rows
 *                          [0, Qb) of q and [0, Kb) of k and v are copied in;
 *                          every row of o and lse is copied out
 *   bytes_in, bytes_out    (may be NULL) receive the bytes copied each way
 * Asynchronous like attn_fwd: `stream` is ordered after the last copy out.
 * Calls on one device are serialised inside the library (they share its two
 * copy streams).  Return codes as attn_fwd.
 */
ATTN_API int attn_fwd_staged(const void *hq, const void *hk, const void *hv, void *ho, float *hlse,
                             void *q, void *k, void *v, void *o, float *lse, int B, int Hq,
                             int Hkv, int Q, int K, int D, int Dv, const int32_t *seqlens_q,
                             const int32_t *seqlens_k, const int32_t *seqlens_q_host,
                             const int32_t *seqlens_k_host, int window, float scale, int dtype,
                             int chunks, unsigned long long *bytes_in,
                             unsigned long long *bytes_out, attn_stream_t stream);

/*
 * attn_bwd -- gradients of attn_fwd_ex (padded layout) for a loss whose
 * gradient with respect to o is dout.  "Accelerating PyTorch on AMD GPUs
 * with FlyDSL", section on FMHA through AOTriton, describes such a backward
 * as separate dQ and dK/dV kernels reusing the forward's building blocks,
 * without its arithmetic; the arithmetic here is the derivative of the
 * forward definition (O = softmax(scale Q K^T + mask) V per row, with the
 * row's log-sum-exp kept).  With P = exp(scale q.k - LSE) over the row's legal
 * keys and Dq = sum(dO * O) over the row:
 *     dS = P (dO . v - Dq)
 *     dq = scale sum_k dS k
 *     dk = scale sum over rows of dS q
 *     dv = sum over rows of P dO
 * where a KV head's dk and dv sum over every query head of its group.
 *   q, k, v       the forward's inputs, shapes as in attn_fwd
 *   o, lse        the forward's outputs for those inputs (lse required);
 *                 P is recomputed from lse, nothing else is stored
 *   dout          [B, Q, Hq, Dv], same dtype as q
 *   dq, dk, dv    outputs shaped like q, k, v (same dtype), written in full:
 *                 rows past seqlens_q, keys past seqlens_k, rows without a
 *                 legal key and keys no row attends to get zeros
 *   seqlens_q, seqlens_k, window, scale, mask   as in attn_fwd_ex
 *   algo          ATTN_ALGO_AUTO (ATTN_ALGO_TCGEN05 where it applies, else
 *                 ATTN_ALGO_MMA, else the CUDA-core kernels), ATTN_ALGO_GENERIC,
 *                 ATTN_ALGO_MMA (mma.sync dK/dV and dQ; bf16/fp16, widths
 *                 multiples of 8 up to 128) or ATTN_ALGO_TCGEN05 (tcgen05
 *                 dQ and dK/dV kernels -- the dK/dV one when Hq / Hkv
 *                 divides 128, else mma.sync; bf16/fp16, widths multiples of
 *                 16 in [64, 128], padded or packed layout)
 * Head widths up to 256 (wider ones return ATTN_ERR_UNSUPPORTED).
 * All pointers are device memory, 16-byte aligned.  A workspace of
 * 4 * B * Q * Hq bytes comes from the library's stream-ordered pool.  The
 * result is deterministic (no atomics: dk/dv and dq are written by separate
 * kernels, each element by one thread).  Returns ATTN_OK, ATTN_ERR_INVALID,
 * ATTN_ERR_UNSUPPORTED (ATTN_ALGO_MMA on a shape it does not take) or
 * ATTN_ERR_CUDA; asynchronous on `stream`.
 */
ATTN_API int attn_bwd(const void *q, const void *k, const void *v, const void *o,
                      const float *lse, const void *dout, void *dq, void *dk, void *dv, int B,
                      int Hq, int Hkv, int Q, int K, int D, int Dv, const int32_t *seqlens_q,
                      const int32_t *seqlens_k, int window, float scale, int mask, int dtype,
                      int algo, attn_stream_t stream);

/* attn_bwd on the packed layout of attn_fwd_varlen_ex: q, o, dout, dq
 * [total_q, Hq, *], k, v, dk, dv [total_k, Hkv, *], sequences given by
 * cu_seqlens_q / cu_seqlens_k (int32 [B + 1]).  Rows of dq, dk and dv
 * outside every sequence are not written. */
ATTN_API int attn_bwd_varlen(const void *q, const void *k, const void *v, const void *o,
                             const float *lse, const void *dout, void *dq, void *dk, void *dv,
                             int B, int Hq, int Hkv, int total_q, int total_k, int max_Q,
                             int max_K, int D, int Dv, const int32_t *cu_seqlens_q,
                             const int32_t *cu_seqlens_k, int window, float scale, int mask,
                             int dtype, int algo, attn_stream_t stream);

/*
 * The 8-bit paged cache.  A serving layout of this library (the pages have no
 * counterpart): the pools of attn_fwd_paged with one byte an element,
 *   k_pages  [num_pages, page_size, Hkv, D]   v_pages [num_pages, page_size, Hkv, Dv]
 *   k_scale, v_scale  float32 [num_pages, page_size / block_size, Hkv]
 * where an element of row r of a page stands for code * scale[page, r / block_size,
 * head]: one scale for each block of block_size tokens (a power of two up to
 * page_size) and head.  cache_dtype ATTN_CACHE_INT8 holds -127..127,
 * ATTN_CACHE_E4M3 the e4m3 values up to +-448 (the NaN code is never written).  Block tables and lengths as in attn_fwd_paged.
 *
 * attn_cache_append -- writes N new rows of each sequence behind the seqlens_k
 * rows it has (seqlens_k is not changed: the caller adds the new rows to it).
 *   k [B, N, Hkv, D], v [B, N, Hkv, Dv]   the new rows, in `dtype` (attn_dtype)
 *   seqlens_new  int32 [B] on the device, new rows of each sequence (clamped to
 *                [0, N]), or NULL for N of each
 *   block_table  int32 [B, max_pages]: every page that gets rows must be there
 *                already and belong to one sequence only (attn_pages_fork sees
 *                to both).  Rows whose entry is outside [0, num_pages), or past
 *                the table, are dropped.
 * A block's scale is the smallest power of two s >= 2^-100 with |x| <= qmax * s
 * (qmax 127 or 448) for its rows, and codes are round-to-nearest-even(x / s).  In
 * a block that has rows already the scale is max(old, needed), and where it
 * grows the block's earlier codes are rounded again under it (e4m3: exactly, down
 * to its subnormals; int8: the roundings sum to at most one step).  Rows and
 * scales of blocks behind the new rows are left as they were.  A block that
 * receives an infinity or a NaN gets the scale NaN and codes 0, and rows that
 * attend to it are what attn_fwd gives for NaN keys and values; it stays so
 * until its page is used afresh.
 * attn_cache_append_varlen takes the new rows packed: k [total_new, Hkv, D],
 * sequence b's rows [cu_seqlens_new[b], cu_seqlens_new[b + 1]), max_new an upper
 * bound of their number.
 * Widths in [1, 512].  Returns ATTN_OK, ATTN_ERR_INVALID, ATTN_ERR_UNSUPPORTED
 * (2^31 or more blocks of rows in a sequence) or ATTN_ERR_CUDA; asynchronous on `stream`.
 */
ATTN_API int attn_cache_append(const void *k, const void *v, void *k_pages, void *v_pages,
                               float *k_scale, float *v_scale, int B, int N, int Hkv, int D,
                               int Dv, const int32_t *seqlens_new, const int32_t *seqlens_k,
                               const int32_t *block_table, int max_pages, int page_size,
                               int num_pages, int block_size, int cache_dtype, int dtype,
                               attn_stream_t stream);
ATTN_API int attn_cache_append_varlen(const void *k, const void *v, void *k_pages, void *v_pages,
                                      float *k_scale, float *v_scale, int B, int total_new,
                                      int max_new, int Hkv, int D, int Dv,
                                      const int32_t *cu_seqlens_new, const int32_t *seqlens_k,
                                      const int32_t *block_table, int max_pages, int page_size,
                                      int num_pages, int block_size, int cache_dtype, int dtype,
                                      attn_stream_t stream);

/*
 * attn_fwd_paged_q8 -- attn_fwd_paged over an 8-bit paged cache: the attention of
 * the values code * scale.  q [B, Q, Hq, D], o [B, Q, Hq, Dv], lse as in
 * attn_fwd_paged; seqlens_k counts the rows to attend to, the new ones among
 * them (append first, then attend); `scale` is finite.  Codes and scales past a sequence's length
 * are never used as values.
 * Kernels (`algo`): ATTN_ALGO_AUTO reads the codes themselves (ATTN_ALGO_DECODE:
 * bf16/fp16, Q * Hq / Hkv <= 1024, D and Dv multiples of 16 up to 256, pages of 8
 * rows or more) where Q * Hq / Hkv <= 64 (32 with D or Dv above 128) or where few
 * sequences and heads leave the other kernels too little to do at once.  Scales
 * then multiply scores and probabilities in fp32 and no key or value is rounded; a
 * key's weight (probability times value scale) is rounded to fp16 in a unit that keeps
 * 11 bits down to 2^-22 of the largest weight among the keys that the row attends to,
 * and steps of 2^-32 of it below; probabilities under 2^-126 of the row's largest count
 * as 0.  Small problems take one launch without a workspace, others a second one that
 * merges the partials of sequences cut between blocks.  Other problems, and the other values of algo
 * (as in attn_fwd_ex), run on a copy of the keys and values in q's type, made
 * group by group of sequences in a workspace from the library's pool (512 MB, or
 * one sequence; eight where a sequence's rows of q or o are no multiple of 16 bytes).
 * The copy is exact with the powers of two that attn_cache_append writes, but for
 * fp16: there values past +-65504 become +-65504 and values below 2^-14 are rounded
 * to steps of 2^-24, which the kernel that reads the codes does not do.  Other scales
 * round once.  Kernels, groups and workspaces go by max_pages, not by lengths, which
 * the host does not know: a table no wider than the longest sequence is the fastest.
 * A sequence's key that a row
 * attends to and whose scale or code is NaN makes that row what attn_fwd gives for
 * a NaN key or value (the kernel that reads the codes: NaN, for a value's code in its
 * column, and no other row changes; the others may, as in attn_fwd, give NaN to rows of
 * the same tile that do not attend to a NaN value as well).
 * Return codes as attn_fwd.
 */
ATTN_API int attn_fwd_paged_q8(const void *q, const void *k_pages, const void *v_pages,
                               const float *k_scale, const float *v_scale, void *o, float *lse,
                               int B, int Hq, int Hkv, int Q, int D, int Dv,
                               const int32_t *block_table, int max_pages, int page_size,
                               int num_pages, int block_size, int cache_dtype,
                               const int32_t *seqlens_q, const int32_t *seqlens_k, int window,
                               float scale, int mask, int dtype, int algo, attn_stream_t stream);

/*
 * Pages of a cache.  A pool is any array whose first axis counts pages: the K or
 * V pages of a layer, or their scales.  `pools` is a HOST array of npools device
 * pointers, page_bytes the bytes of one page of each (any number, also more than
 * one launch takes).  All pools share the block tables.  Tables have at most 2^30
 * slots, pools 2^30 pages.
 *
 * attn_pages_copy -- copies page src[i] of src_pools[p] to page dst[i] of
 * dst_pools[p] for i < n and every p.  src and dst are device int32; pairs with a
 * number outside [0, src_pages) or [0, dst_pages) are skipped.  The dst pages must
 * be distinct and, in the same pool, none of them a src page.
 */
ATTN_API int attn_pages_copy(const void *const *src_pools, void *const *dst_pools,
                             const long long *page_bytes, int npools, int src_pages,
                             int dst_pages, const int32_t *src, const int32_t *dst, int n,
                             attn_stream_t stream);

/*
 * attn_pages_fork -- the next version of a block table: slot i of the new table
 * goes on from slot parents[i] of the old one (beams and branches share a parent,
 * -1 is an empty slot, and an old slot that nobody names is freed), with pages
 * for new_tokens[i] more tokens (NULL: none) behind its seqlens tokens.
 *   block_table int32 [S, max_pages], entries without a page negative;
 *   seqlens int32 [S]; refcount int32 [num_pages]: references to each page by the
 *   table's entries, and by anyone else who holds it (a page of count 0 is free)
 *   parents, new_tokens  int32 [N]
 *   block_table_out [N, max_pages], seqlens_out [N] (tokens, new ones not counted),
 *   refcount_out [num_pages]: the new version; may not alias the old
 *   status int32 [4]: pages that were missing, slots whose tokens do not fit
 *   max_pages, pages newly taken, pages copied
 * Pages full of tokens are shared.  The entries that the slot's next rows go to
 * (from the partly filled page on) are its own: the parent's page goes to the
 * first slot that wants it, unless an entry uses it as a full page or someone
 * outside the table holds it; the others take free pages (those of count 0 in
 * `refcount`), lowest first in the order of slots and entries, and the tokens of a
 * partly filled page are copied into them in every pool.  When pages are missing
 * or a slot is too wide (status[0] or status[1] not 0) nothing is copied,
 * refcount_out equals refcount and the new table is empty: the old version still
 * stands.  Tables that break the rules above give wrong pages, never a bad
 * address.  Runs on `stream` without synchronising; workspace from the library's
 * pool.  The result is deterministic.
 */
ATTN_API int attn_pages_fork(void *const *pools, const long long *page_bytes, int npools,
                             const int32_t *block_table, const int32_t *seqlens,
                             const int32_t *refcount, int S, int max_pages, int num_pages,
                             int page_size, const int32_t *parents, const int32_t *new_tokens,
                             int N, int32_t *block_table_out, int32_t *seqlens_out,
                             int32_t *refcount_out, int32_t *status, attn_stream_t stream);

/*
 * attn_pages_compact -- moves the live pages (refcount > 0) to the front of every
 * pool: with n of them, those at or behind n go to the free pages before n, both
 * in ascending order; the others stay.
 *   block_table_out [S, max_pages] (may alias block_table), refcount_out
 *   [num_pages]: renumbered; remap int32 [num_pages]: the new number of each live
 *   page, -1 for free ones; n_live int32 [1].
 * Entries of pages that are not live become -1.  Runs on `stream` without
 * synchronising; workspace from the library's pool.
 */
ATTN_API int attn_pages_compact(void *const *pools, const long long *page_bytes, int npools,
                                const int32_t *block_table, const int32_t *refcount, int S,
                                int max_pages, int num_pages, int32_t *block_table_out,
                                int32_t *refcount_out, int32_t *remap, int32_t *n_live,
                                attn_stream_t stream);

/*
 * The position rotation.  A serving and training companion of the attention (the
 * pages have no counterpart).  The first `rot` columns (even, 0 .. D) of a head
 * are pairs (x1, x2) -- columns i and i + rot / 2 with ATTN_ROPE_HALF, 2 i and
 * 2 i + 1 with ATTN_ROPE_ADJACENT -- and become
 *     y1 = x1 c - x2 s,   y2 = x2 c + x1 s,   c = cos[pos, i],  s = sin[pos, i]
 * for tables cos, sin of float32 [max_pos, rot / 2] on the device; the other
 * columns are copied.  Products and sums are rounded one by one in fp32 and the
 * result once to the type.  A row whose position is outside [0, max_pos) has NaN in
 * its rotated columns.
 *
 * attn_rope -- q [B, N, Hq, D] and k [B, N, Hkv, D] to q_out, k_out of those
 * shapes.  positions: int32 [B, N] on the device, or NULL for row i of each
 * sequence at position i.  inverse != 0 turns the other way: given gradients of
 * q_out and k_out it gives those of q and k (the rotation's transpose).  Either of
 * q and k may be NULL, with 0 heads.
 *   q_stride, k_stride   elements from one token's row of heads to the next (row
 *                        (b, i) is b * N + i rows in): Hq * D when dense, more for
 *                        views of a fused projection
 * Outputs are dense; each may be its own input where that is dense too (in place),
 * and overlaps no other one.  Tensors need the alignment of their elements only;
 * 16-byte aligned ones with widths and strides to match are the fastest.
 *
 * attn_rope_append -- the rows of a serving step: q is rotated into q_out, k is
 * rotated and, like v as it is, written into the pages of attn_fwd_paged behind
 * the seqlens_k rows each sequence has (seqlens_k is not changed: the caller adds
 * the new rows to it).  Row i of sequence b goes to its row seqlens_k[b] + i, and
 * that is its position too unless `positions` says otherwise.
 *   q [B, N, Hq, D], k [B, N, Hkv, D], v [B, N, Hkv, Dv]   rows, strides as above
 *                (q and q_out may be NULL together, with Hq 0; q_out may be q itself
 *                where that is dense, and overlaps neither other rows nor the cache)
 *   seqlens_new  int32 [B], new rows of each sequence (clamped to [0, N]), or NULL
 *                for N of each; q_out gets +0 in the other rows
 *   cu_seqlens_new   NULL, or int32 [B + 1]: the rows are packed [total_new, ..],
 *                sequence b's are [cu[b], cu[b + 1]), at most N of them (a bound
 *                near the longest is the fastest); rows of q_out outside every
 *                sequence are left as they were
 *   positions    int32, one for each row of the buffers, or NULL
 *   rot 0 (cos and sin may be NULL then) appends without a rotation
 *   k_pages [num_pages, page_size, Hkv, D], v_pages [.., Dv] in `dtype`,
 *   block_table int32 [B, max_pages], as in attn_fwd_paged.  Every page that gets
 *                rows must be there already and belong to one sequence only
 *                (attn_pages_fork sees to both).  Rows whose entry is outside [0,
 *                num_pages), or past the table, are dropped; nothing else of a page
 *                is written.
 * attn_rope_append_q8 -- the same into the 8-bit cache: scales, codes and earlier
 * rows of a block as attn_cache_append writes them, for the rotated keys in fp32
 * (not rounded to `dtype` first).
 * Widths in [1, 512].  Return ATTN_OK, ATTN_ERR_INVALID, ATTN_ERR_UNSUPPORTED (2^31
 * or more blocks of rows in a sequence) or ATTN_ERR_CUDA; one launch (the 8-bit append
 * of many queries: two), no workspace; asynchronous on `stream`.
 */
enum attn_rope_pairs { ATTN_ROPE_HALF = 0, ATTN_ROPE_ADJACENT = 1 };
ATTN_API int attn_rope(const void *q, const void *k, void *q_out, void *k_out, const float *cos,
                       const float *sin, int B, int N, int Hq, int Hkv, int D, int rot,
                       int max_pos, long long q_stride, long long k_stride,
                       const int32_t *positions, int pairs, int inverse, int dtype,
                       attn_stream_t stream);
ATTN_API int attn_rope_append(const void *q, const void *k, const void *v, void *q_out,
                              void *k_pages, void *v_pages, const float *cos, const float *sin,
                              int B, int N, int total_new, int Hq, int Hkv, int D, int Dv, int rot,
                              int max_pos, long long q_stride, long long k_stride,
                              long long v_stride, const int32_t *seqlens_new,
                              const int32_t *cu_seqlens_new, const int32_t *positions, int pairs,
                              const int32_t *seqlens_k, const int32_t *block_table, int max_pages,
                              int page_size, int num_pages, int dtype, attn_stream_t stream);
ATTN_API int attn_rope_append_q8(const void *q, const void *k, const void *v, void *q_out,
                                 void *k_pages, void *v_pages, float *k_scale, float *v_scale,
                                 const float *cos, const float *sin, int B, int N, int total_new,
                                 int Hq, int Hkv, int D, int Dv, int rot, int max_pos,
                                 long long q_stride, long long k_stride, long long v_stride,
                                 const int32_t *seqlens_new, const int32_t *cu_seqlens_new,
                                 const int32_t *positions, int pairs, const int32_t *seqlens_k,
                                 const int32_t *block_table, int max_pages, int page_size,
                                 int num_pages, int block_size, int cache_dtype, int dtype,
                                 attn_stream_t stream);

/*
 * attn_fwd_paged_shared -- attn_fwd_paged (bottom-right causal mask, no window) for a
 * batch whose sequences begin alike, such as beams and samples of one prompt or
 * requests behind one system prompt: the keys that a group shares are read once
 * for the rows of all its members, and the results joined with those of the keys
 * that each sequence has alone.
 *   q [B, Q, Hq, D], pages, block_table [B, max_pages], seqlens_q, seqlens_k, o,
 *   lse as in attn_fwd_paged (seqlens_k counts all keys of a sequence)
 *   cu_groups    int32 [num_groups + 1] on the device, ascending: group n is the
 *                sequences [cu_groups[n], cu_groups[n + 1]) of the batch; the others
 *                share nothing (with num_groups 0 it and shared_lens may be NULL)
 *   shared_lens  int32 [num_groups] on the device: the first shared_lens[n] keys of
 *                the members are the same -- their table entries name the same pages,
 *                or pages of equal contents (a partly filled page copied for each, as
 *                attn_pages_fork does).  They are read through the table of the first
 *                member, and never past its length; members may be shorter than that.
 *   scale        finite
 * Kernels (`algo`): ATTN_ALGO_AUTO and ATTN_ALGO_TCGEN05 take bf16/fp16, D and Dv
 * multiples of 16 in [64, 128], Hq / Hkv <= 128, pages of 8 rows or more and fewer
 * than 2^30 rows (B * Q * Hq) and keys (max_pages * page_size), with at least one group
 * for AUTO.  AUTO runs other
 * problems, and the other values of algo run all of theirs, on the kernels of
 * attn_fwd_paged, which read each sequence's own table for every key.  AUTO does not
 * weigh the two: where few keys are shared (up to 8192 by four sequences of one
 * token, up to 320 by 64), attn_fwd_paged itself is the faster call.  The tcgen05
 * kernel rounds probabilities to q's type before the product with V, as attn_fwd
 * does; partial results are joined in fp32 in a fixed order, so that results do not
 * depend on timing.  A NaN or infinite value of a key that some row of the batch's
 * tile attends to may, as in attn_fwd, give NaN to rows of the tile that do not;
 * scores that are NaN give NaN.  The keys that a sequence has alone go through the same
 * kernel, or, for Q * Hq / Hkv <= 16 and widths of 64 and 128, through the decode's.
 * Workspace from the library's pool: about 8 * (Dv + 2) * (2 * B * Q * Hq + 256 * SMs)
 * bytes; with the decode's kernel 4 * (Dv + 2) bytes for each of these rows once, and
 * for each row and part of its own keys (up to 64 where B * Hkv is small, one where it
 * is 4 * SMs).  Groups that overlap or descend give
 * wrong results, never a bad address.  Return codes as attn_fwd.
 */
ATTN_API int attn_fwd_paged_shared(const void *q, const void *k_pages, const void *v_pages,
                                   void *o, float *lse, int B, int Hq, int Hkv, int Q, int D,
                                   int Dv, const int32_t *block_table, int max_pages,
                                   int page_size, int num_pages, const int32_t *seqlens_q,
                                   const int32_t *seqlens_k, const int32_t *cu_groups,
                                   const int32_t *shared_lens, int num_groups, float scale,
                                   int dtype, int algo, attn_stream_t stream);

/* Message for the calling thread's most recent failed call ("" if none). */
ATTN_API const char *attn_last_error(void);

/* Reads and clears the device status word of the current device
 * (synchronises the device).  Returns ATTN_OK, ATTN_ERR_TIMEOUT, or
 * ATTN_ERR_CUDA if the read itself failed; *detail (may be NULL) receives the
 * kernel-specific detail code. */
ATTN_API int attn_device_status(int *detail);

/*
 * Sets the time limit of the mbarrier waits inside the tcgen05 kernels
 * (prefill, backward, shared beginnings) and of the rotations of many rows
 * for launches made after the call, in nanoseconds, for
 * every thread and device of the process; 0 restores the default of 2 s.
 * Returns the previous limit.  A wait that runs out records ATTN_ERR_TIMEOUT
 * and a detail code in the device status word (attn_device_status), and the
 * launch unwinds: its blocks wait (up to 2 s, whatever this limit) for their
 * own copies and tensor-core operations in flight, free their tensor memory
 * and return, leaving the outputs incomplete and the context usable.  A
 * diagnostic aid: a limit shorter than the kernel's run makes a correct launch
 * time out on purpose, which is how the timeout path is tested.  The pages
 * have no counterpart ("Attention execution mapping" records a submission
 * stall, section 21.9, which is why the waits are bounded at all).
 */
ATTN_API unsigned long long attn_set_wait_limit(unsigned long long ns);

/* Number of kernels this library has launched in the process so far (all
 * devices, all threads).  A measurement aid: the difference around a region
 * counts the library's launches inside it. */
ATTN_API unsigned long long attn_kernel_launches(void);

/* Library version, e.g. "0.1.0". */
ATTN_API const char *attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GQA_H */
