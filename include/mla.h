/*
 * mla.h -- C ABI of libmla: absorbed (MQA-mode) Multi-head Latent Attention decode
 * over a paged latent KV cache, for NVIDIA B200 (sm_100a).
 *
 * The method is the one of the itwiki article "멀티 헤드 잠재 어텐션"
 * (Multi-head latent attention):
 *   - section 구조 (structure): the cache holds the joint latent c^KV_t = W^DKV h_t
 *     (d_c wide); keys and values are W^UK c and W^UV c with W^UK, W^UV of shape
 *     [n_h*d_h, d_c].
 *   - section 행렬 흡수 (matrix absorption): the score q^T W^UK c is computed as
 *     (W^UK^T q)^T c, so each head's query is moved into the latent space and all
 *     heads score the same cached c^KV; W^UV is applied after the weighted sum.
 *   - section 분리 RoPE (decoupled RoPE): a per-head RoPE query q^R and one shared
 *     RoPE key k^R_t are concatenated to the content parts; the cache stores
 *     [c^KV_t ; k^R_t], d_c + d_R values per token; scores are divided by
 *     sqrt(d_h + d_R) and softmaxed over the tokens j <= t.
 *   - section 구현 (implementation): half-split RoPE, angle pos * base^(-2k/d_R).
 * The lecture page "MHA · GQA · MQA · MLA", section "Why Projection Absorption
 * Helps", gives the same identity q^T W_UK c_t = (W_UK^T q)^T c_t.
 *
 * One decode step of one layer is four calls, in this order on one stream:
 *   mla_cache_append  -- write the new tokens' [c^KV ; RoPE(k^R)] rows into the cache
 *   mla_absorb_q      -- q_abs = [W^UK_h^T q^C ; RoPE(q^R)]  per token and head
 *   mla_decode        -- split-KV attention over the cache + log-sum-exp combine
 *   mla_out_proj      -- o = W^UV_h o_lat per token and head
 *
 * Conventions shared by every call
 *   Memory     The caller owns every buffer; all pointers are device pointers of one
 *              device (the current device) unless a comment says otherwise.  The
 *              library allocates no device memory.  Its only device storage is static:
 *              one error word per device (see mla_get_last_device_error) and the scratch
 *              array of mla_decode_fixed_scratch.
 *   Streams    Calls only enqueue work on `stream` (NULL = the legacy default stream)
 *              and return; results are ready in stream order.  mla_absorb_q, mla_decode
 *              and mla_out_proj launch their kernels as programmatic dependents of the
 *              kernel ahead of them on the stream (CUDA programmatic dependent launch):
 *              their blocks may start while that kernel drains, and they wait for it on
 *              the device before reading any activation, cache or table or writing any
 *              output.
 *   Weights    w_uk and w_uv are treated as constants of the layer: mla_absorb_q and
 *              mla_out_proj start reading them before that wait.  Write the weights
 *              before the first call that uses them and make that write complete
 *              (synchronize the stream or device, or wait on an event recorded after
 *              it); do not produce them in the kernel that immediately precedes the call.
 *   Layouts    Row-major, contiguous, as each argument states.
 *   Errors     Arguments are checked on the host before anything is launched; a bad
 *              argument returns an error and launches nothing.  A launch failure
 *              returns MLA_ERR_CUDA.  Conditions only the device can see (a block id
 *              outside the pool, a sequence length outside its table) make the kernel
 *              skip the offending access and set the device error word, which
 *              mla_get_last_device_error reports.  Nothing throws across the ABI.
 *   Softmax    The scale is 1/sqrt(d_h + d_R) (분리 RoPE section, output equation).
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so the header needs no CUDA include. */
typedef struct CUstream_st *mla_stream_t;

typedef enum {
    MLA_OK = 0,
    MLA_ERR_INVALID_ARG = 1,         /* null pointer, negative size, misaligned pointer */
    MLA_ERR_UNSUPPORTED = 2,         /* dims / dtype combination not built into the library */
    MLA_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < mla_decode_workspace_size(...) */
    MLA_ERR_BAD_BLOCK_TABLE = 4,     /* device saw a block id outside [0, num_blocks) */
    MLA_ERR_BAD_SEQ_LEN = 5,         /* device saw a length < s_q or > max_blocks*page */
    MLA_ERR_DEVICE_TIMEOUT = 6,      /* a bounded device-side wait gave up */
    MLA_ERR_CUDA = 7,                /* a CUDA runtime call failed */
    MLA_ERR_BAD_TREE = 8,            /* device saw drafted nodes, parents or kept nodes that are no tree's */
    MLA_ERR_OUT_OF_PAGES = 9,        /* device found fewer free pages than a call to grow wants */
    MLA_ERR_BAD_SEQ_INDEX = 10       /* device saw a sequence index outside the table, or one twice */
} mla_status_t;

typedef enum {
    MLA_DTYPE_F32 = 0,
    MLA_DTYPE_BF16 = 1,
    MLA_DTYPE_FP8_E4M3 = 2 /* cache only: e4m3 content + per-token fp32 scale + bf16 RoPE key */
} mla_dtype_t;

/* flags */
#define MLA_FLAG_SIMT_DECODE 1u /* run mla_decode on the CUDA-core kernel even where the
                                   tensor-core kernel applies (cross-checks) */
#define MLA_FLAG_SIMT_PROJ 2u   /* same for mla_absorb_q and mla_out_proj */
/* FP8 cache only: compute the content part of the scores on the FP8 tensor core
 * (tcgen05 kind::f8f6f4) from the cached e4m3 codes as they are, instead of dequantising every
 * page to bf16 first.  The absorbed query is split per head into two e4m3 parts,
 * q_lat ~ alpha_h (hi + lo) with alpha_h = max|q_lat| / 448, hi = e4m3(q_lat / alpha_h),
 * lo = e4m3(q_lat / alpha_h - hi) (about 7 significant bits, near bf16's 8), and the RoPE part
 * runs in bf16 on (q_R / alpha_h) . (k_R / s_j), so each score is
 *     s_j = alpha_h s_j [ (hi + lo) . c8_j + (q_R / alpha_h) . (k_R,j / s_j) ] / sqrt(d_h + d_R).
 * The value product P . V keeps bf16 V (dequantised on chip).  QuantMLA review, Motivation
 * & Problem Statement (an FP8 content cache next to a high-precision RoPE-key cache). */
#define MLA_FLAG_FP8_MMA 8u
#define MLA_FLAG_TEST_GIVE_UP 4u /* test of the failure path of the tensor-core decodes: in
                                    every cluster with two or more pages, after the copies of
                                    the first page have started, one bounded wait (20 us) on a
                                    barrier that nothing completes gives up.  The cluster then
                                    does what any timed-out wait does: it flags both of its CTAs,
                                    records MLA_ERR_DEVICE_TIMEOUT in the device error word,
                                    waits (2 s bound) for the copies and MMAs it has started, and
                                    exits.  The call's outputs are invalid; nothing faults. */

typedef struct {
    int n_h;            /* heads */
    int d_h;            /* head dim of the content query q^C and of the output o */
    int d_c;            /* latent width of c^KV */
    int d_r;            /* RoPE width d_R (even) */
    int page_size;      /* tokens per cache block (64) */
    float rope_base;    /* RoPE base (1e4) */
    mla_dtype_t act_dtype; /* q_c, q_r, q_abs, c_kv/k_r append inputs, w_uk, w_uv: F32 or BF16 */
    mla_dtype_t kv_dtype;  /* cache: F32, BF16 or FP8_E4M3 */
    unsigned flags;
} mla_dims_t;

/* ----------------------------------------------------------------------------------------
 * mla_absorb_q -- the query side of the absorbed form (행렬 흡수 section; 분리 RoPE section
 * for q^R).  For every token t < T and head h:
 *     q_abs[t, h, 0:d_c]         = W^UK_h^T q_c[t, h, :]      (W^UK_h = rows h*d_h .. of w_uk)
 *     q_abs[t, h, d_c:d_c+d_r]   = RoPE(q_r[t, h, :], pos[t])
 *   q_c   [T, n_h, d_h]   act dtype
 *   q_r   [T, n_h, d_r]   act dtype, before rotation
 *   pos   [T]             int32 position of each token (>= 0)
 *   w_uk  [n_h*d_h, d_c]  act dtype (the nn.Linear(d_c, n_h*d_h) weight)
 *   q_abs [T, n_h, d_c+d_r] act dtype, written
 * Accumulation is fp32.  The rotation angle pos * base^(-2k/d_r) is formed in fp64 and reduced
 * modulo 2 pi in fp64; cos and sin of the reduced angle are fp32.  T == 0 is a no-op.
 * ---------------------------------------------------------------------------------------- */
mla_status_t mla_absorb_q(const mla_dims_t *dims, int T, const void *q_c, const void *q_r,
                          const int32_t *pos, const void *w_uk, void *q_abs,
                          mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * mla_cache_append -- write new tokens into the paged latent cache (분리 RoPE section: the
 * cache holds c^KV_t and k^R_t = RoPE(W^KR h_t), d_c + d_R values per token).
 * Token t goes to sequence s = seq_idx[t] at position p = pos[t]:
 *     block = block_table[s * max_blocks_per_seq + p / page_size],  slot = p % page_size.
 *   c_kv [T, d_c] act dtype;  k_r [T, d_r] act dtype, before rotation.
 *   BF16 / F32 cache: kv_pool [num_blocks, page_size, d_c + d_r] of that dtype, row =
 *       [c_kv ; RoPE(k_r, p)].  kr_pool and kv_scale must be NULL.
 *   FP8_E4M3 cache: kv_pool [num_blocks, page_size, d_c] uint8 e4m3 codes,
 *       kr_pool [num_blocks, page_size, d_r] bf16 RoPE(k_r, p),
 *       kv_scale [num_blocks, page_size] fp32.  Per token s = amax|c_kv|/448 computed in
 *       fp32 (at least FLT_MIN; 1 when amax = 0); codes = e4m3(c_kv / s), nearest-even,
 *       saturating.
 * A token whose block id or table index is out of range is skipped and sets
 * MLA_ERR_BAD_BLOCK_TABLE on the device.  Never reads the pool.
 * ---------------------------------------------------------------------------------------- */
mla_status_t mla_cache_append(const mla_dims_t *dims, int T, const void *c_kv, const void *k_r,
                              const int32_t *seq_idx, const int32_t *pos,
                              const int32_t *block_table, int num_seqs, int max_blocks_per_seq,
                              int num_blocks, void *kv_pool, void *kr_pool, float *kv_scale,
                              mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * mla_append_absorb -- mla_cache_append followed by mla_absorb_q, in one call.  The two
 * write different buffers (the cache; q_abs) and neither reads the other's output, so where
 * the tensor-core absorption applies (n_h any, d_h = 128, d_c = 512, d_r = 64, bf16
 * activations, bf16 or FP8 cache, no MLA_FLAG_SIMT_PROJ, 16-byte aligned q_c, q_r, w_uk,
 * q_abs) both run in ONE launch, the cache writes overlapping the absorption's weight fetch;
 * elsewhere the two are launched one after the other.  The results are bit for bit those of
 * the two calls.
 *   Arguments: those of mla_cache_append (T_new new tokens, pos_new their positions), then
 *   those of mla_absorb_q (T query tokens, pos their positions).
 * Errors: those of either call, checked before anything is launched.
 * ---------------------------------------------------------------------------------------- */
mla_status_t mla_append_absorb(const mla_dims_t *dims, int T_new, const void *c_kv, const void *k_r,
                               const int32_t *seq_idx, const int32_t *pos_new,
                               const int32_t *block_table, int num_seqs, int max_blocks_per_seq,
                               int num_blocks, void *kv_pool, void *kr_pool, float *kv_scale, int T,
                               const void *q_c, const void *q_r, const int32_t *pos, const void *w_uk,
                               void *q_abs, mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * mla_decode_workspace_size -- bytes of device workspace mla_decode needs for B sequences of
 * s_q queries each and sequence lengths up to max_seq_len, on the current device.  Returns 0
 * for invalid arguments or when the current device cannot be queried.
 * ---------------------------------------------------------------------------------------- */
size_t mla_decode_workspace_size(const mla_dims_t *dims, int B, int s_q, int max_seq_len);

/* ----------------------------------------------------------------------------------------
 * mla_decode -- absorbed attention over the paged cache (분리 RoPE section output equation
 * in the latent form of the 행렬 흡수 section).  Query i < s_q of sequence b (row
 * t = b*s_q + i) sits at position P = seq_lens[b] - s_q + i and, for every head h,
 *     s_j     = (q_abs[t,h,0:d_c] . c_j + q_abs[t,h,d_c:] . kR_j) / sqrt(d_h + d_r),  j <= P
 *     o_lat   = sum_j softmax(s)_j c_j,       lse = ln sum_j exp(s_j)
 * where (c_j ; kR_j) is cache row j of sequence b (FP8: c_j = e4m3(code) * scale_j).
 * Precision: bf16 operands, fp32 accumulation and softmax.  With an FP8 cache the kernel
 * dequantises each page on chip to bf16(e4m3(code) * scale_j), one rounding per value, the
 * same a bf16 cache applies when it is written.
 * The tokens are split into segments processed in parallel; the partial results are merged
 * exactly by a log-sum-exp combine kernel.
 *   q_abs       [B*s_q, n_h, d_c+d_r] act dtype (from mla_absorb_q)
 *   kv_pool, kr_pool, kv_scale: the cache, as in mla_cache_append (read only)
 *   block_table [B, max_blocks_per_seq] int32
 *   seq_lens    [B] int32 device array; each in [s_q, max_seq_len]
 *   max_seq_len host-side upper bound of seq_lens (<= max_blocks_per_seq * page_size)
 *   workspace   device scratch of workspace_bytes >= mla_decode_workspace_size(...);
 *               its content on entry does not matter.
 *   o_lat       [B*s_q, n_h, d_c] fp32, written
 *   lse         [B*s_q, n_h] fp32 natural-log normaliser, written (may be NULL)
 * Deterministic: the result depends only on the logical cache content, not on which
 * physical blocks hold it.
 * ---------------------------------------------------------------------------------------- */
mla_status_t mla_decode(const mla_dims_t *dims, int B, int s_q, const void *q_abs,
                        const void *kv_pool, const void *kr_pool, const float *kv_scale,
                        const int32_t *block_table, int max_blocks_per_seq, int num_blocks,
                        const int32_t *seq_lens, int max_seq_len, void *workspace,
                        size_t workspace_bytes, float *o_lat, float *lse, mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * mla_decode_fixed_scratch -- mla_decode without a caller workspace.  This call is a
 * library convenience: the pages describe no counterpart to it.  It computes exactly what
 * mla_decode computes, with the same arguments minus workspace / workspace_bytes.
 *
 * Who it is for: callers that cannot allocate device memory at decode time.  Examples are
 * services with a fixed device-memory budget that is reserved up front (a decode-time
 * allocation may fail once that budget is taken), and code on a latency-critical path where
 * cudaFree / cudaMalloc are not acceptable because they may synchronise the device.
 * Instead of a workspace argument, the call uses a scratch array of
 * MLA_DECODE_FIXED_SCRATCH_BYTES that lives in the library's own static device storage.
 * It allocates nothing itself.
 *
 *   Set-up     The first call on a device looks up that device's scratch address (the CUDA
 *              runtime may load the library's device code at that moment).  Make the first
 *              call on each device before any stream capture begins.  Later calls only read
 *              a cached pointer.
 *   Limit      If mla_decode_workspace_size(dims, B, s_q, max_seq_len) exceeds
 *              MLA_DECODE_FIXED_SCRATCH_BYTES, the call returns MLA_ERR_WORKSPACE_TOO_SMALL
 *              and launches nothing.  Use mla_decode with your own workspace instead.
 *   Sharing    Every call on a device uses the same scratch array.  Calls whose executions
 *              overlap on the device (on different streams without ordering between them)
 *              race on it and produce wrong results.  Serialize them, for example on one
 *              stream.  The scratch needs no clearing: every value the kernels read from it
 *              is written earlier in the same call.
 *   Errors     As for mla_decode; MLA_ERR_CUDA also when the scratch address cannot be
 *              obtained.
 * ---------------------------------------------------------------------------------------- */
#define MLA_DECODE_FIXED_SCRATCH_BYTES (32u << 20) /* 32 MiB per device */
mla_status_t mla_decode_fixed_scratch(const mla_dims_t *dims, int B, int s_q, const void *q_abs,
                                      const void *kv_pool, const void *kr_pool,
                                      const float *kv_scale, const int32_t *block_table,
                                      int max_blocks_per_seq, int num_blocks,
                                      const int32_t *seq_lens, int max_seq_len, float *o_lat,
                                      float *lse, mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * mla_out_proj -- value up-projection after the aggregation (행렬 흡수 section):
 *     o[t, h, :] = W^UV_h o_lat[t, h, :]      (d_h <- d_c; W^UV_h = rows h*d_h .. of w_uv)
 *   o_lat [T, n_h, d_c] fp32;  w_uv [n_h*d_h, d_c] act dtype;
 *   o     [T, n_h, d_h] of out_dtype (F32 or BF16), written.  fp32 accumulation.
 * ---------------------------------------------------------------------------------------- */
mla_status_t mla_out_proj(const mla_dims_t *dims, int T, const float *o_lat, const void *w_uv,
                          void *o, mla_dtype_t out_dtype, mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * mla_decode_project -- mla_decode followed by mla_out_proj in one call: the attention of
 * mla_decode, then o = W^UV_h o_lat (행렬 흡수 section: the value up-projection applied after
 * the aggregation).  Where the tensor-core kernels apply (n_h = 128, d_h = 128, d_c = 512,
 * d_r = 64, page 64, bf16 activations, bf16 or FP8 cache, no MLA_FLAG_SIMT_* flag), the merge
 * of the split partials and the projection run as ONE kernel, which never reads o_lat back;
 * elsewhere the call runs mla_decode and mla_out_proj one after the other.  Either way o,
 * o_lat and lse are bit for bit those of mla_decode followed by mla_out_proj.
 *   Arguments as for mla_decode, plus
 *   w_uv       [n_h*d_h, d_c] act dtype (as for mla_out_proj; written before the call)
 *   o          [B*s_q, n_h, d_h] of out_dtype (F32 or BF16), written
 *   o_lat      [B*s_q, n_h, d_c] fp32, written; 16-byte aligned
 *   lse        as for mla_decode (may be NULL)
 *   workspace  as for mla_decode (mla_decode_workspace_size)
 * Errors: those of mla_decode and mla_out_proj; MLA_ERR_INVALID_ARG also for a null w_uv or
 * o, or an o_lat that is not 16-byte aligned.
 * ---------------------------------------------------------------------------------------- */
mla_status_t mla_decode_project(const mla_dims_t *dims, int B, int s_q, const void *q_abs,
                                const void *kv_pool, const void *kr_pool, const float *kv_scale,
                                const int32_t *block_table, int max_blocks_per_seq, int num_blocks,
                                const int32_t *seq_lens, int max_seq_len, void *workspace,
                                size_t workspace_bytes, const void *w_uv, void *o,
                                mla_dtype_t out_dtype, float *o_lat, float *lse,
                                mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * mla_prefill -- causal attention over whole prompts in MHA ("naive") mode: the keys and
 * values are reconstructed per head from the latent (구조 section), k_{j,h} = [W^UK_h c_j ;
 * RoPE(k^R_j, j)] and v_{j,h} = W^UV_h c_j, and for every prompt token t and head h
 *     o[t,h,:] = sum_{j <= t} softmax_j( [q^C ; RoPE(q^R, t)]_{t,h} . k_{j,h} / sqrt(d_h + d_r) ) v_{j,h}
 * (분리 RoPE section output equation).  The 한계 section and the mode remarks of the 행렬 흡수
 * section: with as many queries as keys, reconstructing K and V once costs less than the
 * 576-wide latent scores of the absorbed form, which pays off in decode only.
 * Positions are token indices within each prompt (0 .. L_b - 1).  The call does not write the
 * cache: append the prompt with mla_cache_append for the decode steps that follow.
 * Supported shape: d_h = 128, d_c = 512, d_r = 64, even n_h, bf16 activations and weights
 * (MLA_ERR_UNSUPPORTED otherwise).  Precision: bf16 operands (K and V rounded to bf16 once,
 * P to bf16), fp32 accumulation and softmax.
 *   B            number of prompts
 *   cu_seqlens   [B+1] int32 device array: prompt b is tokens cu_seqlens[b] .. cu_seqlens[b+1]-1
 *                of the packed inputs; cu_seqlens[0] = 0, cu_seqlens[B] = total_tokens
 *   total_tokens T, the packed token count
 *   max_seq_len  host-side upper bound of the prompt lengths
 *   q_c [T, n_h, d_h], q_r [T, n_h, d_r] (before RoPE), c_kv [T, d_c], k_r [T, d_r] (before
 *                RoPE): bf16, row-major; q_c, q_r, c_kv 16-byte aligned
 *   w_uk, w_uv   [n_h*d_h, d_c] bf16, 16-byte aligned (written before the call)
 *   workspace    device scratch of workspace_bytes >= mla_prefill_workspace_size(dims, T),
 *                256-byte aligned; its content on entry does not matter
 *   o            [T, n_h, d_h] bf16, 16-byte aligned, written
 *   lse          [T, n_h] fp32 natural-log normaliser, written (may be NULL)
 * Errors: MLA_ERR_INVALID_ARG for bad sizes, null or misaligned pointers; a prompt table that
 * is not as stated (or a prompt longer than max_seq_len) is reported by the device as
 * MLA_ERR_BAD_SEQ_LEN through mla_get_last_device_error, with no access outside the buffers.
 * ---------------------------------------------------------------------------------------- */
size_t mla_prefill_workspace_size(const mla_dims_t *dims, int total_tokens);
mla_status_t mla_prefill(const mla_dims_t *dims, int B, const int32_t *cu_seqlens, int total_tokens,
                         int max_seq_len, const void *q_c, const void *q_r, const void *c_kv,
                         const void *k_r, const void *w_uk, const void *w_uv, void *workspace,
                         size_t workspace_bytes, void *o, float *lse, mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * Sequence split across GPUs (long contexts): exact merge of decode results.
 *
 * MLA article, section 한계 (limitations): every head reads the whole latent cache, so tensor
 * parallelism over heads cannot shard it.  The context can be split instead: each rank holds
 * a contiguous range of every sequence's pages, runs mla_decode (s_q = 1) over its own pages
 * only, and the ranks' results merge exactly.  For query row r and head h, with rank i's
 * (o_lat_i, lse_i) from mla_decode:
 *     M = max_i lse_i,  w_i = e^{lse_i - M},
 *     o_lat = sum_i w_i o_lat_i / sum_i w_i,   lse = M + ln sum_i w_i.
 * One step per rank before the cross-rank sum and one after it:
 *   1. lse_max = all-reduce(max) of lse over the ranks       (the caller's collective)
 *   2. mla_lse_merge_prepare: acc = [w o_lat ; w]            (this rank)
 *   3. acc = all-reduce(sum) of acc over the ranks            (the caller's collective)
 *   4. mla_lse_merge_finish: o_lat = acc_o / acc_w, lse = M + ln acc_w
 * Arguments (device pointers, fp32, row-major):
 *   o_lat   [rows, n_h, d_c]  this rank's mla_decode output (prepare) / the merged one (finish)
 *   lse     [rows, n_h]       this rank's lse (prepare, natural log; -inf: no token) / merged
 *                             (finish; may be NULL)
 *   lse_max [rows, n_h]       the maximum of lse over the ranks
 *   acc     [rows * n_h * (d_c + 1)]  w o_lat for every (row, head), then the rows*n_h weights
 *                             w; the caller owns it and sums it over the ranks between the calls
 * A row and head that no rank saw (every lse -inf) merge to o_lat = 0, lse = -inf.  Errors:
 * MLA_ERR_INVALID_ARG for a negative or oversized count or a null pointer (rows = 0 is a no-op).
 * ---------------------------------------------------------------------------------------- */
mla_status_t mla_lse_merge_prepare(int rows, int n_h, int d_c, const float *o_lat, const float *lse,
                                   const float *lse_max, float *acc, mla_stream_t stream);
mla_status_t mla_lse_merge_finish(int rows, int n_h, int d_c, const float *acc, const float *lse_max,
                                  float *o_lat, float *lse, mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * Drafted trees (speculative decoding).
 *
 * A drafter proposes for every sequence a tree of tokens that would follow its committed ones,
 * the target model scores all of them in one step, and the longest path that it agrees with is
 * kept.  MLA article, section 분리 RoPE: a token's cache row is [c^KV ; RoPE(k^R)] and its score
 * set is its own past.  For a drafted node that past is every committed token and, of the
 * drafted ones, its ancestors and itself.
 *
 * A batch's trees are packed like prompts: sequence b's nodes are rows cu_nodes[b] ..
 * cu_nodes[b+1] - 1 of every per-node array, parents before children, n_b = their number (0: none).
 * cu_nodes is a device array [B+1], cu_nodes[0] = 0, non-decreasing.  cu_nodes[B] may be less than
 * total_nodes: the rows behind it belong to no sequence (a captured step's padding) and every call
 * leaves their outputs as they were, except that mla_tree_prepare marks them (below).
 * seq_lens[b] counts the committed tokens and the drafted nodes, as mla_decode's counts the current
 * tokens.  With ctx_b = seq_lens[b] - n_b, node k of sequence b
 *     sits in cache slot   ctx_b + k                 (nodes of equal depth need slots of their own)
 *     has RoPE position    ctx_b + depth(k)          (0 for a child of the last committed token)
 *     sees token j         if j < ctx_b, or if bit (j - ctx_b) of its mask row is set.
 * One step: mla_tree_prepare once; per layer mla_tree_append, mla_absorb_q (pos from
 * mla_tree_prepare), mla_decode_tree, mla_out_proj; after verification mla_cache_keep.
 * A sequence with more nodes than the arguments allow, or whose rows are not rows of the batch, sets
 * MLA_ERR_BAD_TREE on the device; its outputs mean nothing then, and nor do the batch's (each call takes the
 * other sequences or leaves them out).  At most MLA_MAX_TREE_NODES nodes a sequence.
 * ---------------------------------------------------------------------------------------- */
#define MLA_MAX_TREE_NODES 1024

/* mla_tree_prepare -- masks, slots and positions of a batch's trees from their parents.
 *   cu_nodes   [B+1] int32;  parent [total_nodes] int32: the parent's number within the sequence
 *              (less than the node's own), -1 for a child of the last committed token
 *   seq_lens   [B] int32, committed tokens and nodes
 *   mask_words 32-bit words of a mask row, >= max_b ceil(n_b / 32), <= MLA_MAX_TREE_NODES / 32
 *   mask       [total_nodes, mask_words], written: bit k % 32 of word k / 32 is set for every ancestor
 *              k of the node and for the node itself
 *   pos, slot, seq_idx [total_nodes] int32, written: RoPE position, cache slot, sequence.  Rows behind
 *              cu_nodes[B], and those of a sequence with seq_lens[b] < n_b (MLA_ERR_BAD_SEQ_LEN), get
 *              seq_idx -1, which mla_tree_append skips; the former get mask, pos and slot 0.
 * A parent outside [-1, k) sets MLA_ERR_BAD_TREE; the node is taken as a child of the last committed
 * token.  The rows of a sequence that is no tree of the batch get seq_idx -1, pos and slot 0.  B = 0 with total_nodes = 0 is a no-op. */
mla_status_t mla_tree_prepare(int B, const int32_t *cu_nodes, int total_nodes, const int32_t *parent,
                              const int32_t *seq_lens, int mask_words, uint32_t *mask, int32_t *pos,
                              int32_t *slot, int32_t *seq_idx, mla_stream_t stream);

/* mla_tree_append -- mla_cache_append for drafted nodes: token t's row is rotated at pos[t] and written
 * to slot[t] of sequence seq_idx[t].  A token with seq_idx -1 is skipped.  Other arguments, cache
 * formats and errors as for mla_cache_append (slot in the place of pos where the table is indexed).
 * A slot is written by one token of a call. */
mla_status_t mla_tree_append(const mla_dims_t *dims, int T, const void *c_kv, const void *k_r,
                             const int32_t *seq_idx, const int32_t *slot, const int32_t *pos,
                             const int32_t *block_table, int num_seqs, int max_blocks_per_seq,
                             int num_blocks, void *kv_pool, void *kr_pool, float *kv_scale,
                             mla_stream_t stream);

/* mla_decode_tree -- absorbed attention of every drafted node over the cache: for node row t of
 * sequence b and head h, over the tokens j that it sees,
 *     s_j = (q_abs[t,h,0:d_c] . c_j + q_abs[t,h,d_c:] . kR_j) / sqrt(d_h + d_r),
 *     o_lat = sum_j softmax(s)_j c_j,       lse = ln sum_j exp(s_j).
 * A node that sees no token (no committed one and an empty mask row) gets o_lat = 0, lse = -inf.
 * The mask is taken as it is: any set of drafted tokens, not only ancestors.
 * What a masked token's row holds does not matter, infinities and NaN included.  Nor does what a drafted row holds
 * reach a node that gives it a score of -inf: a token of weight 0 is no part of the sums.  Committed rows are taken
 * to be finite.  Where one is not, its scores are what the formula says (so lse is, and
 * a score of +inf or NaN makes its row NaN); of a token whose score is -inf the tensor-core kernel over a bf16 cache
 * makes the columns of o NaN in which the row is not finite, the others leave it out.
 *   cu_nodes    [B+1], total_nodes, max_nodes: a host-side upper bound of the n_b
 *   q_abs       [total_nodes, n_h, d_c+d_r] act dtype (from mla_absorb_q)
 *   cache, block_table, seq_lens, max_seq_len: as for mla_decode; seq_lens[b] in [n_b, max_seq_len]
 *               (otherwise MLA_ERR_BAD_SEQ_LEN on the device, the sequence's rows 0 and -inf)
 *   mask        [total_nodes, mask_words], mask_words >= ceil(max_nodes / 32)
 *   workspace   device scratch of workspace_bytes >= mla_decode_tree_workspace_size(dims, B,
 *               total_nodes, max_seq_len), 256-byte aligned; its content on entry does not matter
 *   o_lat       [total_nodes, n_h, d_c] of out_dtype (F32 or BF16), written
 *   lse         [total_nodes, n_h] fp32, written (may be NULL)
 * The tensor-core kernel runs for d_c = 512, d_r = 64, 64-token pages, bf16 activations, a bf16 or FP8
 * cache, any number of heads and no MLA_FLAG_SIMT_DECODE (q_abs, pools and o_lat 16-byte aligned, or
 * MLA_ERR_INVALID_ARG); other shapes with d_c + d_r <= 1452 run on the CUDA cores (MLA_ERR_UNSUPPORTED beyond).
 * Precision: operands as they are (FP8: the codes exactly, the scales in fp32), fp32 accumulation and
 * softmax.  On the tensor cores P is rounded to bf16 for the value product, as in mla_decode; over an FP8
 * cache P times the token's scale to fp16 instead (11 bits; fewer for a token below 2^-16 of the row's
 * largest, or of 2^-80 if that is larger, to 2^-27 of it), and a query's content elements below 2^-9 of their
 * row's largest, or of 2^-61 if that is larger, are taken to 2^-17 of it.  A query row with infinities or NaN gets NaN.
 * MLA_FLAG_FP8_MMA does not concern this call.  MLA_FLAG_TEST_GIVE_UP does what it does in the tensor-core
 * decode, in every pair of SMs with two or more steps of 256 tokens.
 * Deterministic: the result depends only on the logical cache content. */
size_t mla_decode_tree_workspace_size(const mla_dims_t *dims, int B, int total_nodes, int max_seq_len);
mla_status_t mla_decode_tree(const mla_dims_t *dims, int B, const int32_t *cu_nodes, int total_nodes,
                             int max_nodes, const void *q_abs, const void *kv_pool, const void *kr_pool,
                             const float *kv_scale, const int32_t *block_table, int max_blocks_per_seq,
                             int num_blocks, const int32_t *seq_lens, int max_seq_len,
                             const uint32_t *mask, int mask_words, void *workspace,
                             size_t workspace_bytes, void *o_lat, mla_dtype_t out_dtype, float *lse,
                             mla_stream_t stream);

/* One layer's cache buffers, as mla_cache_append takes them. */
typedef struct {
    void *kv_pool;
    void *kr_pool;   /* FP8 cache only, otherwise NULL */
    float *kv_scale; /* FP8 cache only, otherwise NULL */
} mla_pool_t;

/* mla_cache_keep -- after verification: the accepted path's rows move up behind the committed ones, in
 * every layer.  The row of node keep[b, i] of sequence b goes to slot ctx_b + i, i < num_keep[b]; rows
 * are moved as they are (a path's i-th node was rotated at ctx_b + i already).
 *   pools       [num_pools] host array, the layers' caches behind one block table
 *   keep        [B, max_keep] int32 on the device, each row's first num_keep[b] strictly ascending
 *   num_keep    [B] int32, in [0, min(max_keep, n_b)]
 *   new_lens    [B] int32, written: ctx_b + num_keep[b] (may be NULL; not seq_lens itself, which the
 *               layers' blocks read while it is written)
 * B = 0 or num_pools = 0 is a no-op: nothing is written, new_lens neither.
 * A sequence whose kept nodes are not as stated (MLA_ERR_BAD_TREE), or whose length or pages are bad,
 * is left as it is, its new length seq_lens[b].  Pages of the drafted rows are the sequence's own
 * (mla_pages_grow sees to that): a page that two sequences of the call share is not written in order. */
mla_status_t mla_cache_keep(const mla_dims_t *dims, int num_pools, const mla_pool_t *pools, int B,
                            const int32_t *cu_nodes, int total_nodes, const int32_t *block_table,
                            int max_blocks_per_seq, int num_blocks, const int32_t *seq_lens,
                            const int32_t *keep, const int32_t *num_keep, int max_keep,
                            int32_t *new_lens, mla_stream_t stream);

/* ----------------------------------------------------------------------------------------
 * Pages of the cache.
 *
 * A page (cache block) may be held by several sequences: samples of one prompt, beams, a common
 * prefix.  These calls keep, on the device and in stream order (no host round trip, so a captured step
 * can hold them),
 *     block_table [num_seqs, max_blocks]  int32, -1: no page
 *     refs        [num_blocks] int32      how many table entries hold the page; 0: free
 *     seq_lens    [num_seqs] int32        tokens
 * for all layers at once: the layers' pools share the table.  Every result is determined by the
 * arguments: free pages are taken lowest id first, in the order of the call's entries.
 * A sequence's rows are written only behind its length, and mla_pages_grow makes the page they start
 * in the sequence's own; so full pages are shared for good, and a part-filled one until a holder grows.
 * Lists (parent, child, seqs, new_lens) are device arrays [n].  A list entry that is out of range, or
 * a sequence named twice where one is asked for, sets MLA_ERR_BAD_SEQ_INDEX (MLA_ERR_BAD_SEQ_LEN for a
 * length that is negative or does not fit the table); what the call then does is said with each.
 *   workspace  device scratch of workspace_bytes >= mla_pages_workspace_size(table, n) (n: the longest
 *              list it serves, 0 for mla_pages_compact alone), 256-byte aligned, content on entry of no
 *              matter.  Calls that may run at the same time take a workspace each.
 * ---------------------------------------------------------------------------------------- */
typedef struct {
    int page_size;
    int num_seqs;    /* rows of block_table */
    int max_blocks;  /* entries of a row */
    int num_blocks;  /* pages of the pool */
    int32_t *block_table;
    int32_t *refs;
    int32_t *seq_lens;
} mla_page_table_t;

size_t mla_pages_workspace_size(const mla_page_table_t *table, int n);

/* mla_pages_fork -- sequence child[i] becomes a copy of parent[i] as it was before the call: its table
 * row, whose pages gain a holder, and its length.  What child[i] held before is given back.  A sequence
 * may be parent of many and child of one, of itself too (a beam search's reordering).  A bad entry is
 * skipped; where one child is named twice, both entries are.  A page of the parent's that is none of the pool's
 * sets MLA_ERR_BAD_BLOCK_TABLE, and the child's entry is -1. */
mla_status_t mla_pages_fork(const mla_page_table_t *table, int n, const int32_t *parent,
                            const int32_t *child, void *workspace, size_t workspace_bytes,
                            mla_stream_t stream);

/* mla_pages_grow -- sequence seqs[i] (NULL: sequence i) grows to new_lens[i] tokens: pages for them are
 * taken, and its last page, where that is part-filled and held by others too, is replaced by a page of
 * its own, whose content moves[k] = (from, to) asks mla_cache_copy_pages for.  Of the sequences of one
 * call that share such a page the last keeps it if nobody else holds it.  An entry with new_lens[i] <=
 * its length is left as it is.  Entries beyond the length that already hold a page keep it if the page is the
 * sequence's alone (where a length was lowered with pages left behind it and another sequence holds one of those too,
 * mla_pages_trim comes first); otherwise the entry is bad (MLA_ERR_BAD_BLOCK_TABLE), as is one whose part-filled page
 * nobody holds.
 *   moves      [n, 2] int32, num_moves [1] int32 on the device, written
 * All or nothing: a bad entry, or too few free pages (MLA_ERR_OUT_OF_PAGES), leaves the table as it
 * was, with num_moves 0. */
mla_status_t mla_pages_grow(const mla_page_table_t *table, int n, const int32_t *seqs,
                            const int32_t *new_lens, int32_t *moves, int32_t *num_moves,
                            void *workspace, size_t workspace_bytes, mla_stream_t stream);

/* mla_pages_trim -- sequence seqs[i] (NULL: sequence i) is cut to new_lens[i] tokens (0: it ends): its
 * pages behind them lose a holder, pages reserved beyond its length among them; a longer new_lens[i]
 * leaves the length.  A sequence may be named more than once: the shortest counts.  Bad entries are
 * skipped. */
mla_status_t mla_pages_trim(const mla_page_table_t *table, int n, const int32_t *seqs,
                            const int32_t *new_lens, mla_stream_t stream);

/* mla_pages_compact -- the pages in use take the lowest ids: with u pages in use, the k-th one behind
 * the first u ids moves to the k-th free id among them, table and counts follow, and moves[k] = (from,
 * to) asks mla_cache_copy_pages for its content.  Pages u .. num_blocks - 1 are free afterwards.
 *   moves      [num_blocks / 2, 2] int32, num_moves [1] int32 on the device, written
 * A table entry that names a page nobody holds is left and sets MLA_ERR_BAD_BLOCK_TABLE. */
mla_status_t mla_pages_compact(const mla_page_table_t *table, int32_t *moves, int32_t *num_moves,
                               void *workspace, size_t workspace_bytes, mla_stream_t stream);

/* mla_cache_copy_pages -- page moves[k].from is copied to page moves[k].to in every layer.
 *   moves      [max_moves, 2] int32 on the device; num_moves [1] int32 on the device, how many of them
 *              (NULL: max_moves); more than max_moves are not read
 * No page is the target of two moves, nor target of one and source of another.  A move that names a page
 * outside the pool is skipped and sets MLA_ERR_BAD_BLOCK_TABLE. */
mla_status_t mla_cache_copy_pages(const mla_dims_t *dims, int num_pools, const mla_pool_t *pools,
                                  int num_blocks, const int32_t *moves, const int32_t *num_moves,
                                  int max_moves, mla_stream_t stream);

/* Reads and clears the device error word of the current device.  Synchronises the device.
 * Returns MLA_OK, MLA_ERR_BAD_BLOCK_TABLE, MLA_ERR_BAD_SEQ_LEN, MLA_ERR_DEVICE_TIMEOUT,
 * MLA_ERR_BAD_TREE, MLA_ERR_OUT_OF_PAGES or MLA_ERR_BAD_SEQ_INDEX (the first condition seen since
 * the last call), or MLA_ERR_CUDA. */
mla_status_t mla_get_last_device_error(void);

/* Static, human-readable name of a status code. */
const char *mla_status_string(mla_status_t status);

/* Library ABI version (major * 100 + minor). */
int mla_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MLA_H_ */
