// Drafted trees over the paged latent cache: the tree's bookkeeping (mla_tree_prepare), the accepted
// path's rows (mla_cache_keep), and the CUDA-core form of mla_decode_tree for every shape.
//
// A batch's trees are packed: sequence b drafted the nodes cu_nodes[b] .. cu_nodes[b+1] - 1, node k
// of them at cache slot ctx_b + k, where ctx_b = seq_lens[b] - n_b counts the committed tokens.
// MLA article (itwiki "멀티 헤드 잠재 어텐션"), section 분리 RoPE, output equation in the absorbed
// form of section 행렬 흡수, with the causal set j <= t replaced by the node's own: all committed
// tokens, and the drafted ones whose mask bit is set,
//   s_j = (q_lat . c_j + q^R . k^R_j) / sqrt(d_h + d_R),   o_lat = sum_j softmax(s)_j c_j.
#include <float.h>
#include <math.h>

#include "mla_internal.cuh"
#include "sm100.cuh"
#include "tree.cuh"

namespace mla {
namespace {

// ---- mla_tree_prepare ------------------------------------------------------------------------
// Block per sequence, thread per node: a node walks up its parents (in shared memory), counting its
// depth and collecting its ancestors' bits.  Parents come before their children, so the walk meets
// the mask's words from the last to the first and each is written once.  The last block clears the
// rows behind the last sequence, so that mla_tree_append skips them.
constexpr int kPrepThreads = 128;

__global__ void __launch_bounds__(kPrepThreads)
tree_prepare_kernel(int B, const int32_t *cu, int T, const int32_t *parent,
                    const int32_t *seq_lens, int words, uint32_t *mask,
                    int32_t *pos, int32_t *slot, int32_t *seq_idx,
                    unsigned *err) {
    dependent_start();
    __shared__ int16_t up[kMaxTreeNodes];
    const int b = blockIdx.x;
    if (b == B) {
        for (int t = max(cu[B], 0) + threadIdx.x; t < T; t += kPrepThreads) {
            pos[t] = slot[t] = 0;
            seq_idx[t] = -1;
            for (int w = 0; w < words; ++w) mask[(size_t)t * words + w] = 0u;
        }
        return;
    }
    TreeSpan sp;
    if (!tree_span(cu, b, B, T, 32 * words, &sp)) {
        if (threadIdx.x == 0) record_error(err, kErrBadTree);
        // what an earlier step left in these rows must not send mla_tree_append anywhere
        for (int t = (b == 0 ? 0 : max(cu[b], 0)) + threadIdx.x; t < min(cu[b + 1], T); t += kPrepThreads) {
            pos[t] = slot[t] = 0;
            seq_idx[t] = -1;
        }
        return;
    }
    const int ctx = committed(seq_lens[b], sp.n);
    if (ctx < 0 && threadIdx.x == 0) record_error(err, kErrBadSeqLen);
    bool bad = false;
    for (int k = threadIdx.x; k < sp.n; k += kPrepThreads) {
        int p = parent[sp.t0 + k];
        if (p < -1 || p >= k) {
            bad = true;
            p = -1;
        }
        up[k] = (int16_t)p;
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) record_error(err, kErrBadTree);
    for (int k = threadIdx.x; k < sp.n; k += kPrepThreads) {
        const int t = sp.t0 + k;
        uint32_t *row = mask + (size_t)t * words;
        int w = k >> 5, depth = 0;
        for (int z = words - 1; z > w; --z) row[z] = 0u;
        uint32_t bits = 1u << (k & 31);
        for (int p = up[k]; p >= 0; p = up[p]) {
            ++depth;
            if ((p >> 5) != w) {
                row[w] = bits;
                bits = 0u;
                while (--w > (p >> 5)) row[w] = 0u;
            }
            bits |= 1u << (p & 31);
        }
        row[w] = bits;
        while (--w >= 0) row[w] = 0u;
        pos[t] = max(ctx, 0) + depth;
        slot[t] = max(ctx, 0) + k;
        seq_idx[t] = ctx < 0 ? -1 : b;
    }
}

// ---- mla_cache_keep --------------------------------------------------------------------------
// Block per (sequence, pool).  A thread owns one V-byte column of the rows and moves it for all kept
// nodes, kBatch rows read before any of them is written.  keep is ascending, so the row a later node
// is read from (slot ctx + keep[j] >= ctx + j) lies behind every row written before (ctx + i, i < j)
// and the moves need no copy of the rows.
constexpr int kKeepThreads = 96;
constexpr int kBatch = 8;

struct KeepArgs {
    int B, page, max_blocks, num_blocks, max_keep, T;
    const int32_t *bt, *seq_lens, *cu, *keep, *num_keep;
    int32_t *new_lens;
    unsigned *err;
};

template <typename V>
__device__ __forceinline__ void keep_part(char *part, int cols, const int64_t *rows, int nk) {
    V *base = reinterpret_cast<V *>(part);
    for (int c = threadIdx.x; c < cols; c += kKeepThreads) {
        for (int i0 = 0; i0 < nk; i0 += kBatch) {
            V v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i0 + i < nk && rows[2 * (i0 + i)] >= 0) v[i] = base[rows[2 * (i0 + i)] * cols + c];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i0 + i < nk && rows[2 * (i0 + i)] >= 0) base[rows[2 * (i0 + i) + 1] * cols + c] = v[i];
        }
    }
}

template <typename V>
__global__ void __launch_bounds__(kKeepThreads)
cache_keep_kernel(const __grid_constant__ KeepArgs a, const __grid_constant__ PoolSet pools) {
    dependent_start();
    extern __shared__ int64_t rows[];  // per kept node: source and destination row of the pool, -1: nothing to move
    const int b = blockIdx.x;
    TreeSpan sp;
    const bool tree_ok = tree_span(a.cu, b, a.B, a.T, INT_MAX, &sp);
    const int L = a.seq_lens[b], nk = a.num_keep[b];
    const int ctx = committed(L, sp.n);
    bool bad = !tree_ok || nk < 0 || nk > a.max_keep || nk > sp.n;
    const bool bad_len = tree_ok && (ctx < 0 || L > a.max_blocks * a.page);
    bool bad_block = false;
    if (!bad && !bad_len) {
        const int32_t *keep = a.keep + (size_t)b * a.max_keep;
        for (int i = threadIdx.x; i < nk; i += kKeepThreads) {
            const int k = keep[i];
            int64_t s = -1, d = -1;
            if (k < 0 || k >= sp.n || (i > 0 && keep[i - 1] >= k)) {
                bad = true;
            } else if (k != i) {
                const int32_t *bt = a.bt + (size_t)b * a.max_blocks;
                const int sb = bt[(ctx + k) / a.page], db = bt[(ctx + i) / a.page];
                if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
                    bad_block = true;
                } else {
                    s = (int64_t)sb * a.page + (ctx + k) % a.page;
                    d = (int64_t)db * a.page + (ctx + i) % a.page;
                }
            }
            rows[2 * i] = s;
            rows[2 * i + 1] = d;
        }
    }
    bad = __syncthreads_or(bad);
    bad_block = __syncthreads_or(bad_block);
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        if (bad || bad_len || bad_block) record_error(a.err, bad ? kErrBadTree : bad_len ? kErrBadSeqLen : kErrBadBlock);
        if (a.new_lens) a.new_lens[b] = (bad || bad_len || bad_block) ? L : ctx + nk;
    }
    if (bad || bad_len || bad_block) return;
    const PoolRef &p = pools.pool[blockIdx.y];
    keep_part<V>(p.part[0], pools.row_bytes[0] / (int)sizeof(V), rows, nk);
    if (pools.row_bytes[1]) {
        keep_part<V>(p.part[1], pools.row_bytes[1] / (int)sizeof(V), rows, nk);
        keep_part<uint32_t>(p.part[2], 1, rows, nk);
    }
}

// ---- mla_decode_tree, CUDA cores ---------------------------------------------------------------
// Any dims and cache type, and the cross-check of the tensor-core kernel.  A block takes one node, 8
// of its heads (a warp each) and one segment of its tokens; the online softmax runs in log2 units.
// A masked token's value is never multiplied: its weight is skipped, not zero, so that what a
// sibling's row holds cannot reach this node.  NC: columns of o a lane holds; the smallest of 4, 16 and 32
// that covers d_c (with 32 for all, the toy layer's 4 columns cost a loop of 32: 28 us a call, now 13).
constexpr int kHeads = 8, kTile = 32;

template <int KV>  // 0 = f32 pool, 1 = bf16 pool, 2 = fp8 content pool + bf16 RoPE pool
__device__ __forceinline__ float load_cache(const TreeArgs &a, size_t slot, int k) {
    const int d_c = a.d_c, d_r = a.d_r;
    if (KV == 0) return reinterpret_cast<const float *>(a.kv_pool)[slot * (d_c + d_r) + k];
    if (KV == 1) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.kv_pool)[slot * (d_c + d_r) + k]);
    if (k < d_c) {
        const uint8_t code = reinterpret_cast<const uint8_t *>(a.kv_pool)[slot * d_c + k];
        return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3))) * a.kv_scale[slot];
    }
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.kr_pool)[slot * d_r + (k - d_c)]);
}

template <typename Ta, int KV, int NC, bool JOIN>
__global__ void __launch_bounds__(kHeads * 32)
tree_simt_kernel(const __grid_constant__ TreeArgs a, int seg_len, int n_split, TreePartials part) {
    dependent_start();
    extern __shared__ float smem[];
    const int row = a.d_c + a.d_r, kv_stride = row + 1;  // padding: lanes read different rows
    float *q_s = smem, *kv_s = smem + kHeads * row;
    const int t = blockIdx.x, split = blockIdx.y, h0 = blockIdx.z * kHeads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = h0 + warp;
    TreeSpan sp;
    const int b = tree_of_node(a.cu, a.B, a.T, a.max_nodes, t, &sp);
    const bool first = threadIdx.x == 0 && split == 0 && blockIdx.z == 0;
    if (b < 0) {
        if (b == kTreeBad && first) record_error(a.err, kErrBadTree);
        return;  // a row behind the last sequence, or of no sequence: left as it is
    }
    const int L = a.seq_lens[b], ctx = committed(L, sp.n);
    const bool bad = ctx < 0 || L > a.max_seq_len || L > a.max_blocks * a.page;
    if (bad && first) record_error(a.err, kErrBadSeqLen);
    const int j_begin = split * seg_len, j_end = bad ? 0 : j_begin + min(L - j_begin, seg_len);
    const size_t pr = ((size_t)split * a.T + t) * a.n_h + h;  // this warp's partial row
    const uint32_t *mask = a.mask + (size_t)t * a.mask_words;

    for (int k = lane; k < row; k += 32)
        q_s[warp * row + k] = h < a.n_h ? to_f32(reinterpret_cast<const Ta *>(a.q_abs)[((size_t)t * a.n_h + h) * row + k]) : 0.f;
    float o[NC];
#pragma unroll
    for (int q = 0; q < NC; ++q) o[q] = 0.f;
    float m = -INFINITY, l = 0.f;
    for (int j0 = j_begin; j0 < j_end; j0 += kTile) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTile / kHeads; ++i) {  // a warp's four tokens
            const int jj = warp + i * kHeads, j = j0 + jj;
            int blk = -1;
            if (j < j_end) {
                blk = a.bt[(size_t)b * a.max_blocks + j / a.page];
                if ((blk < 0 || blk >= a.num_blocks) && lane == 0) record_error(a.err, kErrBadBlock);
            }
            const bool have = blk >= 0 && blk < a.num_blocks;
            const size_t slot = (size_t)blk * a.page + j % a.page;
            for (int k = lane; k < row; k += 32) kv_s[jj * kv_stride + k] = have ? load_cache<KV>(a, slot, k) : 0.f;
        }
        __syncthreads();
        if (h >= a.n_h) continue;
        const int j = j0 + lane, d = j - ctx;
        const bool see = j < j_end && (d < 0 || ((mask[d >> 5] >> (d & 31)) & 1u));
        const float *qh = q_s + warp * row, *kvj = kv_s + lane * kv_stride;
        float s = 0.f;
        for (int k = 0; k < row; ++k) s = fmaf(qh[k], kvj[k], s);
        const float s2 = see ? s * a.scale_log2 : -INFINITY;
        float mt = s2;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
        const float m_new = fmaxf(m, mt), base = m_new == -INFINITY ? 0.f : m_new;
        const float corr = exp2f(m - base), p = see ? exp2f(s2 - base) : 0.f;
        float ps = p;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
        l = l * corr + ps;
        m = m_new;
#pragma unroll
        for (int q = 0; q < NC; ++q) o[q] *= corr;
        for (int jj = 0; jj < kTile; ++jj) {
            const float pj = __shfl_sync(0xffffffffu, p, jj);
            if (pj == 0.f) continue;
            const float *kvr = kv_s + jj * kv_stride;
#pragma unroll
            for (int q = 0; q < NC; ++q)
                if (lane + 32 * q < a.d_c) o[q] = fmaf(pj, kvr[lane + 32 * q], o[q]);
        }
    }
    if (l != l) m = l;  // scores of NaN move no maximum, and the join drops what has none
    if (!JOIN) {
        if (h >= a.n_h) return;
#pragma unroll
        for (int q = 0; q < NC; ++q)
            if (lane + 32 * q < a.d_c) part.o[pr * a.d_c + lane + 32 * q] = o[q];
        if (lane == 0) {
            part.m[pr] = m;
            part.l[pr] = l;
        }
        return;
    }
    // The segments' blocks are a cluster: each leaves (o, m, l) in the place of its queries, and joins its
    // share of the columns over all of them.
#pragma unroll
    for (int q = 0; q < NC; ++q)
        if (lane + 32 * q < a.d_c) q_s[warp * row + lane + 32 * q] = o[q];
    if (lane == 0) {
        q_s[warp * row + a.d_c] = m;
        q_s[warp * row + a.d_c + 1] = l;
    }
    sm100::cluster_sync();
    if (h < a.n_h) {
        const uint32_t mine = sm100::smem_u32(q_s + warp * row);
        float w = 0.f, mk = -INFINITY, lk = 0.f;  // lane k: segment k
        if (lane < n_split) {
            const uint32_t at = sm100::mapa(mine, lane) + 4 * a.d_c;
            mk = sm100::ld_cluster_f32(at);
            lk = sm100::ld_cluster_f32(at + 4);
        }
        float M = mk;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float base = M == -INFINITY ? 0.f : M;
        w = exp2f(mk - base);
        float total = w == 0.f ? 0.f : w * lk;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
        const float inv = total == 0.f ? 0.f : 1.f / total;
        const size_t r = (size_t)t * a.n_h + h;
        const int share = (a.d_c + n_split - 1) / n_split, c1 = min(a.d_c, share * (split + 1));
        for (int c0 = share * split; c0 < c1; c0 += 32) {
            float acc = 0.f;
            for (int k = 0; k < n_split; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                if (wk != 0.f && c0 + lane < c1)
                    acc = fmaf(wk, sm100::ld_cluster_f32(sm100::mapa(mine, k) + 4 * (c0 + lane)), acc);
            }
            if (c0 + lane < c1) {
                if (a.out_bf16) reinterpret_cast<__nv_bfloat16 *>(a.o)[r * a.d_c + c0 + lane] = __float2bfloat16_rn(acc * inv);
                else reinterpret_cast<float *>(a.o)[r * a.d_c + c0 + lane] = acc * inv;
            }
        }
        if (a.lse && split == 0 && lane == 0) a.lse[r] = total == 0.f ? -INFINITY : (base + log2f(total)) * 0.69314718055994531f;
    }
    sm100::cluster_sync();  // no block leaves while another reads its sums
}

// More segments than a cluster has blocks: joins a row's partials, o = sum_s 2^(m_s - M) o_s /
// sum_s 2^(m_s - M) l_s.  A segment without a visible token (m = -inf) has weight 0 and is not read.
constexpr int kJoinThreads = 128;
template <typename To>
__global__ void __launch_bounds__(kJoinThreads)
tree_join_kernel(const __grid_constant__ TreeArgs a, int n_split, TreePartials part) {
    dependent_start();
    const int t = blockIdx.x, h = blockIdx.y;
    TreeSpan sp;
    if (tree_of_node(a.cu, a.B, a.T, a.max_nodes, t, &sp) < 0) return;
    const size_t r = (size_t)t * a.n_h + h, step = (size_t)a.T * a.n_h;
    float M = -INFINITY;
    for (int s = 0; s < n_split; ++s) M = fmaxf(M, part.m[s * step + r]);
    const float base = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    for (int s = 0; s < n_split; ++s) l += exp2f(part.m[s * step + r] - base) * part.l[s * step + r];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int c = threadIdx.x; c < a.d_c; c += kJoinThreads) {
        float acc = 0.f;
        for (int s = 0; s < n_split; ++s) {
            const float w = exp2f(part.m[s * step + r] - base);
            if (w != 0.f) acc = fmaf(w, part.o[(s * step + r) * a.d_c + c], acc);
        }
        reinterpret_cast<To *>(a.o)[r * a.d_c + c] = from_f32<To>(acc * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[r] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.69314718055994531f;
}

int sm_count() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

// Segments of the token axis: enough blocks for four on every SM, a tile of tokens at least.  Up to
// kClusterSegs of them are a cluster that joins them itself (one launch: 17 us a call of the toy layer became
// 13); more only where even so many leave half of the SMs without a block.
constexpr int kClusterSegs = 8;
struct TreeSimtPlan {
    int n_split, seg_len;
    bool join;  // in the cluster
};
TreeSimtPlan tree_simt_plan(const mla_dims_t &d, int T, int max_seq_len) {
    const int sms = sm_count();
    const int64_t blocks = (int64_t)T * ((d.n_h + kHeads - 1) / kHeads), target = 4 * sms;
    const int tiles = (max_seq_len - 1) / kTile + 1;
    int64_t n = blocks > 0 ? (target + blocks - 1) / blocks : 1;
    if (n > tiles) n = tiles;
    if (n > kClusterSegs && blocks * kClusterSegs * 2 >= sms) n = kClusterSegs;
    const int seg = (int)((tiles + n - 1) / n) * kTile;
    const int n_split = (max_seq_len - 1) / seg + 1;
    return {n_split, seg, n_split <= kClusterSegs};
}

}  // namespace

// Shared memory of a block: its queries and a tile's rows.
static size_t tree_simt_smem(const mla_dims_t &d) {
    const size_t row = (size_t)d.d_c + d.d_r;
    return sizeof(float) * (kHeads * row + kTile * (row + 1));
}
bool tree_simt_supported(const mla_dims_t &d) { return tree_simt_smem(d) <= 232448; }

size_t tree_simt_workspace_bytes(const mla_dims_t &d, int T, int max_seq_len) {
    const TreeSimtPlan pl = tree_simt_plan(d, T, max_seq_len);
    if (pl.join) return 0;
    const size_t rows = (size_t)pl.n_split * T * d.n_h;
    return align_up(rows * d.d_c * sizeof(float), 256) + 2 * align_up(rows * sizeof(float), 256);
}

cudaError_t launch_tree_simt(const mla_dims_t &d, const TreeArgs &a, void *ws, cudaStream_t st) {
    const TreeSimtPlan pl = tree_simt_plan(d, a.T, a.max_seq_len);
    const size_t rows = (size_t)pl.n_split * a.T * d.n_h;
    TreePartials part = {};
    if (!pl.join) {
        char *w = reinterpret_cast<char *>(ws);
        part.o = reinterpret_cast<float *>(w);
        w += align_up(rows * d.d_c * sizeof(float), 256);
        part.m = reinterpret_cast<float *>(w);
        part.l = reinterpret_cast<float *>(w + align_up(rows * sizeof(float), 256));
    }
    const size_t smem = tree_simt_smem(d);
    const dim3 grid(a.T, pl.n_split, (d.n_h + kHeads - 1) / kHeads);
    cudaError_t e = cudaSuccess;
    auto run = [&](auto kern) {
        if (smem > 48 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
            e = launch_dependent_cluster(kern, grid, dim3(1, pl.join ? pl.n_split : 1, 1), kHeads * 32, smem, st, a,
                                         pl.seg_len, pl.n_split, part);
    };
#define MLA_TREE_SIMT2(TA, KV, JOIN)                                          \
    do {                                                                      \
        if (d.d_c <= 128) run(tree_simt_kernel<TA, KV, 4, JOIN>);             \
        else if (d.d_c <= 512) run(tree_simt_kernel<TA, KV, 16, JOIN>);       \
        else run(tree_simt_kernel<TA, KV, 32, JOIN>);                         \
    } while (0)
#define MLA_TREE_SIMT(TA, KV)                                                 \
    do {                                                                      \
        if (pl.join) MLA_TREE_SIMT2(TA, KV, true);                            \
        else MLA_TREE_SIMT2(TA, KV, false);                                   \
    } while (0)
    const bool ab = d.act_dtype == MLA_DTYPE_BF16;
    if (d.kv_dtype == MLA_DTYPE_F32) {
        if (ab) MLA_TREE_SIMT(__nv_bfloat16, 0); else MLA_TREE_SIMT(float, 0);
    } else if (d.kv_dtype == MLA_DTYPE_BF16) {
        if (ab) MLA_TREE_SIMT(__nv_bfloat16, 1); else MLA_TREE_SIMT(float, 1);
    } else {
        if (ab) MLA_TREE_SIMT(__nv_bfloat16, 2); else MLA_TREE_SIMT(float, 2);
    }
#undef MLA_TREE_SIMT
#undef MLA_TREE_SIMT2
    if (e != cudaSuccess || pl.join) return e;
    const dim3 jg(a.T, d.n_h);
    return launch_dependent(a.out_bf16 ? tree_join_kernel<__nv_bfloat16> : tree_join_kernel<float>, jg, kJoinThreads, 0,
                            st, a, pl.n_split, part);
}

cudaError_t launch_tree_prepare(int B, const int32_t *cu, int T, const int32_t *parent, const int32_t *seq_lens,
                                int words, uint32_t *mask, int32_t *pos, int32_t *slot, int32_t *seq_idx,
                                cudaStream_t st) {
    return launch_dependent(tree_prepare_kernel, dim3(B + 1), kPrepThreads, 0, st, B, cu, T, parent, seq_lens, words,
                            mask, pos, slot, seq_idx, device_error_word());
}

cudaError_t launch_cache_keep(const mla_dims_t &d, int num_pools, const mla_pool_t *pools, int B, const int32_t *cu,
                              int T, const int32_t *bt, int max_blocks, int num_blocks, const int32_t *seq_lens,
                              const int32_t *keep, const int32_t *num_keep, int max_keep, int32_t *new_lens,
                              cudaStream_t st) {
    KeepArgs a{B, d.page_size, max_blocks, num_blocks, max_keep, T, bt, seq_lens, cu, keep, num_keep, new_lens,
               device_error_word()};
    const size_t smem = (size_t)2 * sizeof(int64_t) * max_keep;
    for (int p0 = 0; p0 < num_pools; p0 += kPoolsPerLaunch) {
        PoolSet set;
        const int n = num_pools - p0 < kPoolsPerLaunch ? num_pools - p0 : kPoolsPerLaunch;
        const int v = make_pool_set(d, 1, pools + p0, n, &set);
        if (p0 > 0) a.new_lens = nullptr;
        const dim3 grid(B, n);
        const cudaError_t e = launch_dependent(v == 16  ? cache_keep_kernel<uint4>
                                               : v == 4 ? cache_keep_kernel<uint32_t>
                                                        : cache_keep_kernel<uint8_t>,
                                               grid, kKeepThreads, smem, st, a, set);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mla
