// Shared by the drafted-tree and page kernels: argument blocks, the checks of a batch's packed trees,
// and the parts of a pool's rows.
#pragma once

#include <limits.h>

#include "mla_internal.cuh"

namespace mla {

constexpr int kMaxTreeNodes = 1024;  // drafted nodes of one sequence

// Arguments of mla_decode_tree as the kernels take them.
struct TreeArgs {
    int B, T, max_nodes, n_h, d_c, d_r, page;
    float scale_log2;  // log2(e) / sqrt(d_h + d_r)
    const void *q_abs, *kv_pool, *kr_pool;
    const float *kv_scale;
    const int32_t *cu, *bt, *seq_lens;
    int max_blocks, num_blocks, max_seq_len;
    const uint32_t *mask;
    int mask_words;
    void *o;
    int out_bf16;
    float *lse;
    unsigned *err;
    int test_give_up;  // MLA_FLAG_TEST_GIVE_UP
};

// Partial results of one token segment: o [segment][T * n_h][d_c], m and l [segment][T * n_h].
struct TreePartials {
    float *o, *m, *l;
};

struct TreeSpan {
    int t0, n;  // the sequence's first node row, and how many
};

// Sequence b's rows of the packed trees; false if they are not rows of the batch or too many.
__device__ __forceinline__ bool tree_span(const int32_t *cu, int b, int B, int T, int max_nodes, TreeSpan *sp) {
    const int t0 = cu[b], t1 = cu[b + 1];
    const bool ok = t0 >= 0 && t1 >= t0 && t1 <= T && t1 - t0 <= max_nodes && (b > 0 || t0 == 0);
    sp->t0 = ok ? t0 : 0;
    sp->n = ok ? t1 - t0 : 0;
    return ok;
}

// Committed tokens of a sequence of L tokens and n nodes, -1 where L is less than n (any int: no difference that
// passes the type's range comes out as a length).
__device__ __forceinline__ int committed(int L, int n) { return L < n ? -1 : L - n; }

// The sequence that drafted row t: kTreeNone behind the last sequence, kTreeBad where cu is not a
// non-decreasing list of rows or the sequence has more than max_nodes.
constexpr int kTreeNone = -1, kTreeBad = -2;
__device__ __forceinline__ int tree_of_node(const int32_t *cu, int B, int T, int max_nodes, int t, TreeSpan *sp) {
    if (t >= cu[B]) return cu[B] < 0 ? kTreeBad : kTreeNone;
    int lo = 0, hi = B;  // the last b with cu[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    if (!tree_span(cu, lo, B, T, max_nodes, sp) || t < sp->t0 || t >= sp->t0 + sp->n) return kTreeBad;
    return lo;
}

// A pool's buffers as byte rows: [c ; k_R] rows, or codes, RoPE keys and scales of an FP8 cache.
constexpr int kPoolParts = 3, kPoolsPerLaunch = 64;
struct PoolRef {
    char *part[kPoolParts];
};
struct PoolSet {
    int row_bytes[kPoolParts];  // of a token's row or a page; 0: the cache type has no such part
    PoolRef pool[kPoolsPerLaunch];
};
// Fills *set for rows of `tokens` tokens (1, or a page); returns the widest of 16, 4 and 1 bytes that
// divides every row and base address of the first two parts (the scales are moved as they are, 4 bytes each).
inline int make_pool_set(const mla_dims_t &d, int tokens, const mla_pool_t *pools, int n, PoolSet *set) {
    const bool fp8 = d.kv_dtype == MLA_DTYPE_FP8_E4M3;
    const int es = d.kv_dtype == MLA_DTYPE_F32 ? 4 : 2;
    set->row_bytes[0] = tokens * (fp8 ? d.d_c : (d.d_c + d.d_r) * es);
    set->row_bytes[1] = tokens * (fp8 ? d.d_r * 2 : 0);
    set->row_bytes[2] = tokens * (fp8 ? 4 : 0);
    uintptr_t all = (uintptr_t)set->row_bytes[0] | (uintptr_t)set->row_bytes[1];
    for (int i = 0; i < n; ++i) {
        set->pool[i].part[0] = reinterpret_cast<char *>(pools[i].kv_pool);
        set->pool[i].part[1] = reinterpret_cast<char *>(pools[i].kr_pool);
        set->pool[i].part[2] = reinterpret_cast<char *>(pools[i].kv_scale);
        for (int k = 0; k < (fp8 ? 2 : 1); ++k) all |= reinterpret_cast<uintptr_t>(set->pool[i].part[k]);
    }
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
}

// A launch as a programmatic dependent of the kernel before it on the stream: the kernel starts with
// griddepcontrol.wait, so that only its set-up overlaps that kernel.
template <typename... P, typename... A>
inline cudaError_t launch_dependent_cluster(void (*kern)(P...), dim3 grid, dim3 cluster, int threads, size_t smem,
                                            cudaStream_t st, A... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster.x;
    attr[1].val.clusterDim.y = cluster.y;
    attr[1].val.clusterDim.z = cluster.z;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    return launch_dependent_cluster(kern, grid, dim3(1), threads, smem, st, args...);
}
// At the start of such a kernel: dependents of its own may be set up, and what came before is complete.
__device__ __forceinline__ void dependent_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- launchers ---------------------------------------------------------------------------------
bool tree_simt_supported(const mla_dims_t &d);  // d_c + d_r up to 1452: shared memory
size_t tree_simt_workspace_bytes(const mla_dims_t &d, int T, int max_seq_len);
cudaError_t launch_tree_simt(const mla_dims_t &d, const TreeArgs &a, void *ws, cudaStream_t st);
// Tensor cores: d_c = 512, d_r = 64, 64-token pages, bf16 activations.
bool tree_tc_supported(const mla_dims_t &d);
size_t tree_tc_workspace_bytes(const mla_dims_t &d, int B, int T);
cudaError_t launch_tree_tc(const mla_dims_t &d, const TreeArgs &a, void *ws, cudaStream_t st);
cudaError_t launch_tree_prepare(int B, const int32_t *cu, int T, const int32_t *parent, const int32_t *seq_lens,
                                int words, uint32_t *mask, int32_t *pos, int32_t *slot, int32_t *seq_idx,
                                cudaStream_t st);
cudaError_t launch_tree_append(const mla_dims_t &d, int T, const void *c_kv, const void *k_r, const int32_t *seq_idx,
                               const int32_t *slot, const int32_t *pos, const int32_t *bt, int num_seqs,
                               int max_blocks, int num_blocks, void *kv_pool, void *kr_pool, float *kv_scale,
                               cudaStream_t st);
cudaError_t launch_cache_keep(const mla_dims_t &d, int num_pools, const mla_pool_t *pools, int B, const int32_t *cu,
                              int T, const int32_t *bt, int max_blocks, int num_blocks, const int32_t *seq_lens,
                              const int32_t *keep, const int32_t *num_keep, int max_keep, int32_t *new_lens,
                              cudaStream_t st);

// The paged cache's bookkeeping (pages.cu).
struct PageTable {
    int page, num_seqs, max_blocks, num_blocks;
    int32_t *bt, *refs, *seq_lens;
    unsigned *err;
};
size_t pages_workspace_bytes(const PageTable &p, int n);
cudaError_t launch_pages_fork(const PageTable &p, int n, const int32_t *parent, const int32_t *child, void *ws,
                              cudaStream_t st);
cudaError_t launch_pages_grow(const PageTable &p, int n, const int32_t *seqs, const int32_t *new_lens, int32_t *moves,
                              int32_t *num_moves, void *ws, cudaStream_t st);
cudaError_t launch_pages_trim(const PageTable &p, int n, const int32_t *seqs, const int32_t *new_lens,
                              cudaStream_t st);
cudaError_t launch_pages_compact(const PageTable &p, int32_t *moves, int32_t *num_moves, void *ws, cudaStream_t st);
cudaError_t launch_copy_pages(const mla_dims_t &d, int num_pools, const mla_pool_t *pools, int num_blocks,
                              const int32_t *moves, const int32_t *num_moves, int max_moves, cudaStream_t st);

}  // namespace mla
