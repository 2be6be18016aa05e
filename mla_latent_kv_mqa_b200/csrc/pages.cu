// Pages of the latent cache, kept on the device: which sequence holds which (the block table), how
// many sequences hold each (the reference counts), and the copies that sharing and moving ask for.
//
// The tables are small and every answer depends on all of them (the lowest free page, the k-th page in
// use), so the deciding kernels are one block each; what grows with the cache's bytes (the copies) runs
// on the whole GPU.  All results are integers that depend on the arguments alone: counts are added with
// atomics, whose order does not show, and pages are taken in the order of their ids.
//
// Measured (one B200, warm, whole calls): forking and growing beams with 447 MB of copies 82 us, compacting
// with 1.08 GB moved 197 us: 5.4 TB/s, 0.83 of a plain copy's rate, with ~10 us of deciding ahead of the
// copies; with little to copy the host's calls take most of the time (39-43 us for fork, grow and copies, or trim,
// compact and copies, with the three copies that fill the tables before them).
#include "mla_internal.cuh"
#include "tree.cuh"

namespace mla {
namespace {

__device__ __forceinline__ int pages_of(int len, int page) { return len / page + (len % page != 0); }

// ---- mla_pages_fork --------------------------------------------------------------------------
// All parents' rows are read (into the workspace) before any child's row is written, so a sequence may
// be parent and child at once (a beam search's reordering).
constexpr int kForkThreads = 128;

__global__ void __launch_bounds__(kForkThreads)
fork_read_kernel(const __grid_constant__ PageTable p, int n, const int32_t *parent,
                 const int32_t *child, int32_t *lens, int32_t *rows) {
    dependent_start();
    const int i = blockIdx.x, s = parent[i], c = child[i];
    bool bad = s < 0 || s >= p.num_seqs || c < 0 || c >= p.num_seqs;
    for (int k = threadIdx.x; k < n; k += kForkThreads) bad |= k != i && child[k] == c;  // a child once
    bad = __syncthreads_or(bad);
    const int len = bad ? 0 : p.seq_lens[s];
    const bool bad_len = len < 0 || pages_of(len, p.page) > p.max_blocks;
    if (threadIdx.x == 0) {
        if (bad) record_error(p.err, kErrBadSeqIndex);
        else if (bad_len) record_error(p.err, kErrBadSeqLen);
        lens[i] = bad || bad_len ? -1 : len;
    }
    if (bad || bad_len) return;
    const int np = pages_of(len, p.page);
    for (int k = threadIdx.x; k < np; k += kForkThreads) {
        int v = p.bt[(size_t)s * p.max_blocks + k];
        if (v < 0 || v >= p.num_blocks) {
            record_error(p.err, kErrBadBlock);
            v = -1;
        } else {
            atomicAdd(&p.refs[v], 1);
        }
        rows[(size_t)i * p.max_blocks + k] = v;
    }
}

__global__ void __launch_bounds__(kForkThreads)
fork_write_kernel(const __grid_constant__ PageTable p, const int32_t *child,
                  const int32_t *lens, const int32_t *rows) {
    dependent_start();
    const int i = blockIdx.x, len = lens[i];
    if (len < 0) return;
    const int c = child[i], np = pages_of(len, p.page);
    for (int k = threadIdx.x; k < p.max_blocks; k += kForkThreads) {
        int32_t *e = &p.bt[(size_t)c * p.max_blocks + k];
        const int old = *e;
        if (old >= 0 && old < p.num_blocks) atomicSub(&p.refs[old], 1);
        *e = k < np ? rows[(size_t)i * p.max_blocks + k] : -1;
    }
    if (threadIdx.x == 0) p.seq_lens[c] = len;
}

// ---- mla_pages_trim --------------------------------------------------------------------------
__global__ void __launch_bounds__(kForkThreads)
trim_kernel(const __grid_constant__ PageTable p, const int32_t *seqs,
            const int32_t *new_lens) {
    dependent_start();
    const int i = blockIdx.x, s = seqs ? seqs[i] : i, len = new_lens[i];
    if (s < 0 || s >= p.num_seqs || len < 0) {
        if (threadIdx.x == 0) record_error(p.err, len < 0 ? kErrBadSeqLen : kErrBadSeqIndex);
        return;
    }
    for (int k = pages_of(len, p.page) + threadIdx.x; k < p.max_blocks; k += kForkThreads) {
        int32_t *e = &p.bt[(size_t)s * p.max_blocks + k];
        if (*e == -1) continue;
        const int old = atomicExch(e, -1);  // whoever takes the entry gives the page back, once
        if (old >= 0 && old < p.num_blocks) atomicSub(&p.refs[old], 1);
    }
    if (threadIdx.x == 0) atomicMin(&p.seq_lens[s], len);
}

// ---- one block's scans -------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
struct ScanScratch {
    int warp[32];
};
// Exclusive scan of x over the block; *total gets the sum.  Ends with a barrier.
__device__ __forceinline__ int block_exclusive(int x, ScanScratch *s, int *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) s->warp[w] = v;
    __syncthreads();
    if (w == 0) {
        int t = s->warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        s->warp[lane] = t;
    }
    __syncthreads();
    const int before = w > 0 ? s->warp[w - 1] : 0;
    *total = s->warp[31];
    __syncthreads();
    return before + v - x;
}

// ---- mla_pages_grow --------------------------------------------------------------------------
// One block.  1: every entry's wants: pages its table row has none of, and a copy of its last page
// where that is not full and another sequence holds it too.  Of the sequences that share such a page
// and grow in this call each takes a copy, except the last of them if nobody else holds the page (what
// growing them one after the other comes to); so the sharers are counted per page first.  2: the lowest
// free pages, as many as are wanted; fewer refuse the whole call.  3: the pages to the entries, in order.
struct GrowWs {
    int32_t *owner;   // [num_seqs] which entry named the sequence
    int32_t *count;   // [num_blocks] entries of this call that share a last page
    int32_t *last;    // [num_blocks] the last of them
    int32_t *want;    // [n] pages wanted; bit 30: the first of them is a copy
    int32_t *free_;   // [num_blocks] the free pages taken
};
constexpr int kWantCopy = 1 << 30, kFewPages = 8, kSearch = 8;

__global__ void __launch_bounds__(kPlanThreads)
grow_kernel(const __grid_constant__ PageTable p, int n, const int32_t *seqs,
            const int32_t *new_lens, int32_t *moves, int32_t *num_moves,
            const __grid_constant__ GrowWs ws) {
    dependent_start();
    __shared__ ScanScratch scan;
    __shared__ int err_code;
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) err_code = 0;
    __syncthreads();
    auto seq = [&](int i) { return seqs ? seqs[i] : i; };
    auto entry = [&](int s, int k) { return &p.bt[(size_t)s * p.max_blocks + k]; };
    // checks; a sequence named twice
    for (int i = tid; i < n; i += kPlanThreads) {
        const int s = seq(i);
        if (s < 0 || s >= p.num_seqs) err_code = kErrBadSeqIndex;
        else if (seqs) ws.owner[s] = i;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads) {
        const int s = seq(i);
        if (s < 0 || s >= p.num_seqs) continue;
        if (seqs && ws.owner[s] != i) err_code = kErrBadSeqIndex;
        const int cur = p.seq_lens[s], len = new_lens[i];
        if (cur < 0 || len < 0 || pages_of(len, p.page) > p.max_blocks) err_code = kErrBadSeqLen;
        else if (len > cur && cur % p.page) {
            const int v = *entry(s, cur / p.page);
            if (v < 0 || v >= p.num_blocks || p.refs[v] < 1) err_code = kErrBadBlock;
            else {
                ws.count[v] = 0;
                ws.last[v] = -1;
            }
        }
    }
    __syncthreads();
    if (err_code) {
        if (tid == 0) {
            record_error(p.err, (unsigned)err_code);
            *num_moves = 0;
        }
        return;
    }
    for (int i = tid; i < n; i += kPlanThreads) {
        const int s = seq(i), cur = p.seq_lens[s];
        if (new_lens[i] > cur && cur % p.page) {
            const int v = *entry(s, cur / p.page);
            atomicAdd(&ws.count[v], 1);
            atomicMax(&ws.last[v], i);
        }
    }
    __syncthreads();
    // 1: wants, a thread per entry (its loads run beside the others'); a warp where an entry grows by many pages
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int s = 0, cur = 0, len = 0, want = 0;
        if (i < n) {
            s = seq(i);
            cur = p.seq_lens[s];
            len = new_lens[i];
        }
        const int lo = pages_of(cur, p.page), hi = len > cur ? pages_of(len, p.page) : lo;
        const bool few = hi - lo <= kFewPages;
        auto wants = [&](int at, int k) {  // a page; one that is there has to be the sequence's alone, its rows are written next
            const int v = *entry(at, k);
            if (v >= 0 && (v >= p.num_blocks || p.refs[v] != 1)) err_code = kErrBadBlock;
            return (int)(v < 0);
        };
        if (few)
            for (int k = lo; k < hi; ++k) want += wants(s, k);
        for (unsigned many = __ballot_sync(0xffffffffu, !few); many; many &= many - 1) {
            const int who = __ffs(many) - 1;
            const int ws_ = __shfl_sync(0xffffffffu, s, who), wlo = __shfl_sync(0xffffffffu, lo, who), whi = __shfl_sync(0xffffffffu, hi, who);
            int w = 0;
            for (int k = wlo + lane; k < whi; k += 32) w += wants(ws_, k);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
            if (lane == who) want = w;
        }
        if (i < n) {
            if (len > cur && cur % p.page) {
                const int v = *entry(s, cur / p.page);
                if (ws.count[v] < p.refs[v] || ws.last[v] != i) want = (want + 1) | kWantCopy;
            }
            ws.want[i] = want;
        }
    }
    __syncthreads();
    if (err_code) {
        if (tid == 0) {
            record_error(p.err, (unsigned)err_code);
            *num_moves = 0;
        }
        return;
    }
    int total = 0, copies = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {  // the entries' first pages and first copies
        const int i = i0 + tid, w = i < n ? ws.want[i] : 0;
        int sum;
        block_exclusive(w & ~kWantCopy, &scan, &sum);
        total += sum;
        block_exclusive((w & kWantCopy) != 0, &scan, &sum);
        copies += sum;
    }
    // 2: the lowest free pages, kSearch consecutive ids a thread at a time
    int found = 0;
    for (int v0 = 0; v0 < p.num_blocks && found < total; v0 += kPlanThreads * kSearch) {
        const int v1 = v0 + tid * kSearch;
        unsigned mine = 0;
#pragma unroll
        for (int k = 0; k < kSearch; ++k) mine |= (unsigned)(v1 + k < p.num_blocks && p.refs[v1 + k] == 0) << k;
        int sum;
        int at = found + block_exclusive(__popc(mine), &scan, &sum);
        for (; mine && at < total; mine &= mine - 1) ws.free_[at++] = v1 + __ffs(mine) - 1;
        found += sum;
    }
    if (found < total) {
        if (tid == 0) {
            record_error(p.err, kErrOutOfPages);
            *num_moves = 0;
        }
        return;
    }
    // 3: hand them out in the entries' order
    __syncthreads();
    int page0 = 0, move0 = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid, w = i < n ? ws.want[i] : 0;
        int sum_p, sum_m;
        int at = page0 + block_exclusive(w & ~kWantCopy, &scan, &sum_p);
        const int mv = move0 + block_exclusive((w & kWantCopy) != 0, &scan, &sum_m);
        page0 += sum_p;
        move0 += sum_m;
        int s = 0, cur = 0, len = 0;
        if (i < n) {
            s = seq(i);
            cur = p.seq_lens[s];
            len = new_lens[i];
        }
        if (w & kWantCopy) {  // the first page: a copy of the shared one
            const int to = ws.free_[at++];
            int32_t *e = entry(s, cur / p.page);
            const int v = *e;
            moves[2 * mv] = v;
            moves[2 * mv + 1] = to;
            *e = to;
            atomicSub(&p.refs[v], 1);
            p.refs[to] = 1;
        }
        const int lo = pages_of(cur, p.page), hi = len > cur ? pages_of(len, p.page) : lo;
        const bool few = hi - lo <= kFewPages;
        if (few)
            for (int k = lo; k < hi; ++k)
                if (*entry(s, k) < 0) {
                    const int to = ws.free_[at++];
                    *entry(s, k) = to;
                    p.refs[to] = 1;
                }
        for (unsigned many = __ballot_sync(0xffffffffu, !few); many; many &= many - 1) {
            const int who = __ffs(many) - 1;
            const int ws_ = __shfl_sync(0xffffffffu, s, who), wlo = __shfl_sync(0xffffffffu, lo, who), whi = __shfl_sync(0xffffffffu, hi, who);
            int wat = __shfl_sync(0xffffffffu, at, who);
            for (int k0 = wlo; k0 < whi; k0 += 32) {
                const bool open = k0 + lane < whi && *entry(ws_, k0 + lane) < 0;
                const unsigned set = __ballot_sync(0xffffffffu, open);
                if (open) {
                    const int to = ws.free_[wat + __popc(set & ((1u << lane) - 1u))];
                    *entry(ws_, k0 + lane) = to;
                    p.refs[to] = 1;
                }
                wat += __popc(set);
            }
        }
        if (len > cur) p.seq_lens[s] = len;
    }
    if (tid == 0) *num_moves = copies;
}

// ---- mla_pages_compact -----------------------------------------------------------------------
// One block decides: with `used` pages in use, the k-th page in use behind the first `used` ids moves to
// the k-th free id among them.  A second kernel follows the ids through the block table.
__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(const __grid_constant__ PageTable p, int32_t *moves, int32_t *num_moves, int32_t *to) {
    dependent_start();
    __shared__ ScanScratch scan;
    const int tid = threadIdx.x;
    int count = 0, used;
    for (int v = tid; v < p.num_blocks; v += kPlanThreads) count += p.refs[v] > 0;
    block_exclusive(count, &scan, &used);
    int holes = 0, movers = 0;
    for (int v0 = 0; v0 < p.num_blocks; v0 += kPlanThreads * kSearch) {  // kSearch consecutive ids a thread
        const int v1 = v0 + tid * kSearch;
        unsigned live = 0, there = 0;
#pragma unroll
        for (int k = 0; k < kSearch; ++k) {
            live |= (unsigned)(v1 + k < p.num_blocks && p.refs[v1 + k] > 0) << k;
            there |= (unsigned)(v1 + k < p.num_blocks) << k;
        }
        const int in_front = min(max(used - v1, 0), kSearch);  // of these ids, those among the first `used`
        const unsigned front = (1u << in_front) - 1u;
        unsigned hole = ~live & there & front, mover = live & ~front;
        int sum;
        int h = holes + block_exclusive(__popc(hole), &scan, &sum);
        holes += sum;
        int m = movers + block_exclusive(__popc(mover), &scan, &sum);
        movers += sum;
#pragma unroll
        for (int k = 0; k < kSearch; ++k)  // where a page is afterwards, -1: nobody holds it (a mover's place follows)
            if (there >> k & 1) to[v1 + k] = live >> k & 1 ? v1 + k : -1;
        for (; hole; hole &= hole - 1) moves[2 * h++ + 1] = v1 + __ffs(hole) - 1;
        for (; mover; mover &= mover - 1) moves[2 * m++] = v1 + __ffs(mover) - 1;
    }
    __syncthreads();
    for (int k = tid; k < movers; k += kPlanThreads) {
        const int s = moves[2 * k], d = moves[2 * k + 1];
        p.refs[d] = p.refs[s];
        p.refs[s] = 0;
        to[s] = d;
    }
    if (tid == 0) *num_moves = movers;
}

constexpr int kFollowThreads = 256;
__global__ void __launch_bounds__(kFollowThreads)
compact_follow_kernel(const __grid_constant__ PageTable p, const int32_t *to) {
    dependent_start();
    const size_t n = (size_t)p.num_seqs * p.max_blocks;
    for (size_t i = (size_t)blockIdx.x * kFollowThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kFollowThreads) {
        const int v = p.bt[i];
        if (v < 0) continue;
        const int d = v < p.num_blocks ? to[v] : -1;
        if (d < 0) record_error(p.err, kErrBadBlock);  // a page that nobody holds: the entry stays
        else if (d != v) p.bt[i] = d;
    }
}

// ---- mla_cache_copy_pages --------------------------------------------------------------------
// Pure copy, 2 x 73728 bytes a page of a bf16 V3 cache: every thread keeps kInFlight 16-byte loads in
// flight.  The moves' number is known on the device only, so a fixed grid walks all of
// (pool, move, piece of a page).
constexpr int kCopyThreads = 256, kInFlight = 6;

struct CopyArgs {
    const int32_t *moves, *num_moves;
    int max_moves, num_blocks, num_pools, pieces;
    unsigned *err;
};

// Piece `piece` of a page of `cols` elements.
template <typename V>
__device__ __forceinline__ void copy_part(char *part, int cols, int s, int d, int piece, int pieces) {
    const int c0 = (int)((int64_t)cols * piece / pieces), c1 = (int)((int64_t)cols * (piece + 1) / pieces);
    const V *src = reinterpret_cast<const V *>(part) + (size_t)s * cols;
    V *dst = reinterpret_cast<V *>(part) + (size_t)d * cols;
    for (int c = c0 + threadIdx.x; c < c1; c += kCopyThreads * kInFlight) {
        V v[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (c + i * kCopyThreads < c1) v[i] = src[c + i * kCopyThreads];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (c + i * kCopyThreads < c1) dst[c + i * kCopyThreads] = v[i];
    }
}

template <typename V>
__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const __grid_constant__ CopyArgs a, const __grid_constant__ PoolSet pools) {
    dependent_start();
    const int count = a.num_moves ? min(max(*a.num_moves, 0), a.max_moves) : a.max_moves;
    const int64_t work = (int64_t)count * a.num_pools * a.pieces;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int piece = (int)(w % a.pieces);
        const int64_t mp = w / a.pieces;
        const int m = (int)(mp % count), q = (int)(mp / count);
        const int s = a.moves[2 * m], d = a.moves[2 * m + 1];
        if (s < 0 || s >= a.num_blocks || d < 0 || d >= a.num_blocks) {
            if (threadIdx.x == 0) record_error(a.err, kErrBadBlock);
            continue;
        }
        if (s == d) continue;
        const PoolRef &pool = pools.pool[q];
        copy_part<V>(pool.part[0], pools.row_bytes[0] / (int)sizeof(V), s, d, piece, a.pieces);
        if (pools.row_bytes[1]) {
            copy_part<V>(pool.part[1], pools.row_bytes[1] / (int)sizeof(V), s, d, piece, a.pieces);
            copy_part<uint32_t>(pool.part[2], pools.row_bytes[2] / 4, s, d, piece, a.pieces);
        }
    }
}

int sm_count() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

struct PagesWs {
    int32_t *a, *b, *c, *d, *e;
    size_t bytes;
};
// fork: lens [n], rows [n][max_blocks].  grow: owner, count, last, want, free.  compact: to (in b).
PagesWs pages_ws(const PageTable &p, int n, void *base) {
    char *w = reinterpret_cast<char *>(base);
    size_t at = 0;
    auto take = [&](size_t ints) {
        int32_t *r = reinterpret_cast<int32_t *>(w + at);
        at += align_up(ints * sizeof(int32_t), 256);
        return r;
    };
    PagesWs s;
    s.a = take(n > p.num_seqs ? n : p.num_seqs);
    s.b = take(p.num_blocks);
    s.c = take(p.num_blocks);
    s.d = take(n > 0 ? n : 1);
    const size_t rows = (size_t)n * p.max_blocks;
    s.e = take(rows > (size_t)p.num_blocks ? rows : (size_t)p.num_blocks);
    s.bytes = at;
    return s;
}

}  // namespace

size_t pages_workspace_bytes(const PageTable &p, int n) { return pages_ws(p, n, nullptr).bytes; }

cudaError_t launch_pages_fork(const PageTable &p, int n, const int32_t *parent, const int32_t *child, void *ws,
                              cudaStream_t st) {
    const PagesWs s = pages_ws(p, n, ws);
    const cudaError_t e = launch_dependent(fork_read_kernel, dim3(n), kForkThreads, 0, st, p, n, parent, child, s.a, s.e);
    return e != cudaSuccess ? e : launch_dependent(fork_write_kernel, dim3(n), kForkThreads, 0, st, p, child, s.a, s.e);
}

cudaError_t launch_pages_grow(const PageTable &p, int n, const int32_t *seqs, const int32_t *new_lens, int32_t *moves,
                              int32_t *num_moves, void *ws, cudaStream_t st) {
    const PagesWs s = pages_ws(p, n, ws);
    return launch_dependent(grow_kernel, dim3(1), kPlanThreads, 0, st, p, n, seqs, new_lens, moves, num_moves,
                            GrowWs{s.a, s.b, s.c, s.d, s.e});
}

cudaError_t launch_pages_trim(const PageTable &p, int n, const int32_t *seqs, const int32_t *new_lens,
                              cudaStream_t st) {
    return launch_dependent(trim_kernel, dim3(n), kForkThreads, 0, st, p, seqs, new_lens);
}

cudaError_t launch_pages_compact(const PageTable &p, int32_t *moves, int32_t *num_moves, void *ws, cudaStream_t st) {
    const PagesWs s = pages_ws(p, 0, ws);
    const cudaError_t e = launch_dependent(compact_plan_kernel, dim3(1), kPlanThreads, 0, st, p, moves, num_moves, s.b);
    if (e != cudaSuccess) return e;
    const size_t n = (size_t)p.num_seqs * p.max_blocks, blocks = (n + kFollowThreads - 1) / kFollowThreads;
    const int most = 4 * sm_count();
    return launch_dependent(compact_follow_kernel, dim3(blocks < (size_t)most ? (int)blocks : most), kFollowThreads, 0, st,
                            p, s.b);
}

cudaError_t launch_copy_pages(const mla_dims_t &d, int num_pools, const mla_pool_t *pools, int num_blocks,
                              const int32_t *moves, const int32_t *num_moves, int max_moves, cudaStream_t st) {
    for (int p0 = 0; p0 < num_pools; p0 += kPoolsPerLaunch) {
        PoolSet set;
        const int n = num_pools - p0 < kPoolsPerLaunch ? num_pools - p0 : kPoolsPerLaunch;
        const int v = make_pool_set(d, d.page_size, pools + p0, n, &set);
        const CopyArgs a{moves, num_moves, max_moves, num_blocks, n, 3, device_error_word()};
        const int64_t work = (int64_t)max_moves * n * a.pieces, most = 8 * sm_count();
        const int grid = (int)(work < most ? work : most);
        const cudaError_t e = launch_dependent(v == 16  ? copy_pages_kernel<uint4>
                                               : v == 4 ? copy_pages_kernel<uint32_t>
                                                        : copy_pages_kernel<uint8_t>,
                                               dim3(grid), kCopyThreads, 0, st, a, set);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mla
