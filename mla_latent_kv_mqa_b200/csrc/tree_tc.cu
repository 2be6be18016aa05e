// Tensor-core (tcgen05, CTA pairs) mla_decode_tree for d_c = 512, d_R = 64, 64-token pages.
//
// MLA article (itwiki "멀티 헤드 잠재 어텐션"), section 분리 RoPE output equation in the absorbed form
// of section 행렬 흡수, for the drafted nodes of a sequence.  All nodes and heads of a sequence attend
// to the same cache rows, so its (node, head) pairs are the rows of two dense contractions, whatever
// the number of heads.  A tile is 128 of them, a step 256 tokens (four pages):
//     S[128 x 256]  = Q[128 x 576] . KV[256 x 576]^T,     O[128 x 512] += P[128 x 256] . V[256 x 512].
//
// Split over a pair of SMs.  O in fp32 for 128 rows fills one SM's tensor memory, so the pair's two CTAs
// take 64 rows each (cta_group::2, M = 128): O is 256 columns, S two buffers of 128.  No score and no P
// crosses the pair, nothing is computed twice, and each operand byte of B is read from one CTA's shared
// memory only: for S each CTA holds the K rows of two of the step's pages, for O the halves of V's
// columns that its half of N takes.  In a CTA's tensor memory lanes 0-63 hold its rows against the
// first half of N and lanes 64-127 the same rows against the second; a softmax thread owns a row against
// one of the step's pages and exchanges the maximum with the three others of its row.
//
// Roles (16 warps a CTA).  One thread loads Q per tile and K, one V, in rings of 16 KB stages; two threads
// of the even CTA issue the MMAs of S and of O for both CTAs, S of the next step while this one's
// softmax runs.  (An MMA costs its thread about 60 clocks, the 64 that it runs, and a stage's wait and
// commit another 170: one thread for both left the tensor cores idle for half the time.)  Eight warps do
// the softmax in log2 units with a lazily moved maximum (O is rescaled when it grows by more than 8),
// write P as the MMA's A operand, and at a tile's end write O; four warps clean the V rows that some row
// of the tile does not see (one warp took 25000 clocks a tile for it).
//
// FP8.  K's codes are operands as they are, at twice the rate, against two e4m3 parts of each query, which
// together are the bf16 query (split_query): no K passes through registers, and S takes as long as in bf16.
// (K's codes converted to bf16 tiles by four more warps took 593 us where this took 420, with 96 registers a
// thread for the softmax, which spilled.)  V would need P in parts too, and a part's range is too small for a
// long context's weights: the cleaning warps turn V's codes into fp16 tiles, exactly, by two instructions for
// four codes (bf16 takes eight), and P is fp16.  Its 11 bits reach from 2^15 down to 2^-14, so m is chosen to
// bound P with the tokens' scales in it; what is below 2^-16 of a row's largest weight times scale loses
// bits, and below 2^-27 is lost (scales below 2^-80, in a row of none larger, sooner).  Content and RoPE scores are apart, since only the first take the token's
// scale: one buffer of S, no second.  What is left to the softmax and the conversion sets the pace (tensor
// pipe 50% busy, clocks not limited): every instruction there shows, so the page's scales come two steps
// after their page's id, without a wait, and what only a sequence's last pages need is out of the common path.
//
// Masks.  Steps before ctx need none.  In the others a row's thread selects by its node's bits.  P is 0
// where a node does not see a token, and 0 times what such a row holds must be 0: the cleaning warps zero
// the rows behind the sequence, and the infinities and NaN of drafted rows (whoever sees such a row has
// them in its scores already, as NaN or as weight 0).  Committed rows are seen by every row of the tile and are
// taken as they are: over bf16 an infinity among them is NaN in its column of O for a row whose score it makes
// -inf too (to clean them would take 16 KB of shared memory once more through registers for each V stage).
//
// Split along the tokens.  All (tile, step) units of the batch are dealt to the pairs in contiguous
// equal runs; a tile that lies in several runs leaves partial (O, m, l), at most two a pair, which a
// second kernel joins.  Where few tiles are spread over many pairs, a tile's steps are turned (tile_turn).
//
// Measured (B200, warm; ten calls after a pause, and in a loop of seconds, which power slows): 24 sequences of
// 1024-8190 tokens, 3-24 nodes, 128 heads 449 us = 1040 TFLOP/s, 505-535 in the loop; 16 of 6000-8192, 64 nodes
// 1.83 ms = 1110, 1.99-2.15; 4 of 131072, 4 nodes 490 us = 1190, 555-577; FP8, 32 of 4097-8192, 2-12 nodes 436 us = 920,
// 471-492.  A step takes ~6800 clocks over bf16, of which the MMAs run 4352.  L2 hands the SMs 5.1 GB a call of the
// first, 11.5 TB/s where loads alone reach 12.5 (557 KB a step and pair: 128 rows a pair use a byte, and O leaves no
// tensor memory for more rows).
//
// Every wait is bounded (2 s).  On give-up both CTAs' abort flags are set, MLA_ERR_DEVICE_TIMEOUT is
// recorded, and both CTAs stay until copies and MMAs in flight have had time to land.  What the join acts on
// (schedule) is written before the first wait; of a pair that gave up it joins whatever the partials hold.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <float.h>
#include <math.h>

#include <mutex>

#include "mla_internal.cuh"
#include "sm100.cuh"
#include "tmap.cuh"
#include "tree.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int DC = 512, ROW = 576, PG = 64, NCB = ROW / 64;
constexpr int TILE = 128, HALF = 64;              // rows of a tile, and of a CTA
constexpr int STEP = 256, SPG = STEP / PG;        // tokens and pages of a step
constexpr int CB = PG * 128;                      // 64 rows x 64 bf16 columns, 128-byte swizzle
constexpr int STAGE = 2 * CB;                     // K: two pages' 128 bytes a row; V: a page's 128 columns
constexpr int F8_KST = DC / 128 + 1;              // FP8: K stages of a step, the codes' and the RoPE keys'
constexpr int MAX_STAGES = 4;
constexpr int Q_OFF = 0, P_OFF = NCB * CB, K_OFF = P_OFF + SPG * CB;
constexpr int RAW = 8192, RAW_STAGES = 2;         // FP8: the codes of a V stage, before their conversion
// Shared memory and tensor memory of the bf16 (F8 = false) and FP8 kernels.
template <bool F8>
struct Lay {
    static constexpr int k_stages = F8 ? 3 : 4, v_stages = 3;
    static constexpr int v_off = K_OFF + k_stages * STAGE, vraw_off = v_off + v_stages * STAGE;
    static constexpr int data = F8 ? vraw_off + RAW_STAGES * RAW : vraw_off;
    static constexpr int s_bufs = F8 ? 1 : 2;     // FP8: content and RoPE scores apart, one buffer of both
};
constexpr int DATA = Lay<false>::data;
static_assert(Lay<true>::data == DATA, "one shared-memory size");
constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int LOAD_K_WARP = 0, LOAD_V_WARP = 1, QK_WARP = 2, PV_WARP = 3, SM_WARP0 = 4, CLEAN_WARP0 = 12;
constexpr int SM_WARPS = 8, SM_THREADS = 32 * SM_WARPS, CLEAN_THREADS = 128;
constexpr uint32_t S_COL = 0, O_COL = 256, TMEM_COLS = 512;
constexpr float RESCALE_LOG2 = 8.0f;
constexpr int BAR_MAX = 1, BAR_CLEAN = 2;

struct __align__(16) Ctrl {
    uint64_t k_full[MAX_STAGES], v_full[MAX_STAGES];    // even CTA: both CTAs' halves are there (landed, cleaned, converted)
    uint64_t k_empty[MAX_STAGES], v_empty[MAX_STAGES];  // each CTA: the MMAs that read the stage are done
    uint64_t land[MAX_STAGES];  // each CTA: a V stage that the cleaning warps have to go over has landed
    uint64_t vraw_full[RAW_STAGES], vraw_empty[RAW_STAGES];  // FP8: each CTA's codes of V
    uint64_t q_land, q_full, q_empty;  // FP8: each CTA's queries have landed; both CTAs' are operands; read by the MMAs
    uint64_t s_full[2], s_free[2];
    uint64_t p_full[SPG], p_free[SPG];  // a page of P: written / its MMAs done
    // By step parity: O read or rescaled as the step needs / the step's MMAs done.  A CTA may be a step ahead of
    // its peer, so one barrier would take its arrivals for two steps as both CTAs' for one.
    uint64_t o_ok[2], pv_done[2];
    uint64_t never_done;  // nothing completes it (MLA_FLAG_TEST_GIVE_UP)
    uint32_t tmem_base, abort;
    int w_b, w_tile, w_step, w_n;
    long long w_units, w_end;  // of the batch; where the pair's run ends
    long long scan_u[WARPS];
    int scan_t[WARPS];
    alignas(16) float scale[SM_WARPS][2][PG];  // FP8: each softmax warp's page's scales, as they are and with 0 for infinities and NaN
    float q_unit[2][HALF];  // FP8, by segment parity: what a row's scores are multiples of
    float top[2][SPG][HALF], sum[SPG][HALF];  // by step parity (a thread may be a step behind its partners), page, row
};
constexpr int SMEM = 1024 + DATA + (int)((sizeof(Ctrl) + 127) / 128 * 128);
static_assert(SMEM <= 232448, "shared memory per block");

// What the join reads: the batch's units and tiles, and for every tile its first row, its rows, the first
// pair that had steps of it and how many pairs from there (0: none, a bad length; negative: that pair began
// with another tile).
struct TreePlan {
    long long *units;
    int *tiles;
    int4 *tile;
    float *o, *m, *l;  // [2 pairs][128 / 8][512 / 4][8 rows][4 columns], [2 pairs][128 rows]
    int pairs;
};

struct Seq {
    int t0, n, L, ctx, tiles, steps;
};
__device__ __forceinline__ Seq seq_of(const TreeArgs &a, int t0, int n, int L) {
    Seq s;
    s.t0 = t0;
    s.n = n;
    s.L = L;
    s.ctx = committed(L, n);
    s.tiles = (int)(((long long)s.n * a.n_h + TILE - 1) / TILE);
    s.steps = s.ctx < 0 || s.L > a.max_seq_len || s.L > a.max_blocks * PG ? 0 : (s.L + STEP - 1) / STEP;
    return s;
}

__device__ __forceinline__ Seq seq_of(const TreeArgs &a, int b) { return seq_of(a, a.cu[b], a.cu[b + 1] - a.cu[b], a.seq_lens[b]); }

// A pair's first unit.  (Batches of fewer than 2^24 units, all but the largest, without a 64-bit division.)
__device__ __forceinline__ long long unit_start(long long c, long long U, int pairs) {
    return U < (1 << 24) ? (uint32_t)c * (uint32_t)U / (uint32_t)pairs : c * U / pairs;
}
__device__ __forceinline__ int pair_of_unit(long long u, long long U, int pairs) {
    int c = U < (1 << 24) ? (int)((uint32_t)u * (uint32_t)pairs / (uint32_t)U) : (int)(u * pairs / U);
    while (c + 1 < pairs && unit_start(c + 1, U, pairs) <= u) ++c;
    while (c > 0 && unit_start(c, U, pairs) > u) --c;
    return c;
}

// Where a tile's steps begin among its sequence's (they go around from there).  Pairs start together and keep pace, so
// where a tile takes several runs, its first whole run begins at the sequence's first step: all tiles of the sequence
// then go over the same places of a long cache at the same time, and L2 hands on what one of them fetched.
// u0: the tile's first unit.
__device__ __noinline__ int tile_turn(long long u0, int steps, long long U, int pairs) {
    if ((long long)steps * pairs <= U + pairs) return 0;  // no longer than a run
    const int c = pair_of_unit(u0, U, pairs);
    return unit_start(c, U, pairs) == u0 ? 0 : steps - (int)(unit_start(c + 1, U, pairs) - u0);
}

// Walks a pair's units; every role walks the same ones.
template <bool TURN>
struct Walk {
    Seq s;
    int b, tile, step, left;
    bool first;  // of its segment (a run of one tile's steps)
    bool head;   // the segment is the pair's first
    int seg0;    // the segment's first step
    int turn;    // TURN: the place of the tile's first step
    __device__ void init(const TreeArgs &a, const TreePlan &pl, const Ctrl *c) {
        b = c->w_b;
        tile = c->w_tile;
        step = seg0 = c->w_step;
        left = c->w_n;
        first = head = true;
        if (left > 0) {
            s = seq_of(a, b);
            if (TURN) turn = tile_turn(c->w_end - left - step, s.steps, c->w_units, pl.pairs);
        }
    }
    // The place of the tile's step k among its sequence's.
    __device__ __forceinline__ int at(int k) const { return !TURN ? k : k + turn >= s.steps ? k + turn - s.steps : k + turn; }
    __device__ bool done() const { return left <= 0; }
    __device__ int pages() const { return min(SPG, (s.L + PG - 1) / PG - at(step) * SPG); }  // of this step
    __device__ bool last() const { return left == 1 || step == s.steps - 1; }
    __device__ __forceinline__ void next(const TreeArgs &a, const TreePlan &pl, const Ctrl *c) {
        first = last();
        if (first) head = false;
        --left;
        if (++step == s.steps) {
            step = 0;
            if (++tile == s.tiles) {
                tile = 0;
                b = next_seq(a, b);
                if (b < a.B) s = seq_of(a, b);
                else left = 0;
            }
            if (TURN && left > 0) turn = tile_turn(c->w_end - left, s.steps, c->w_units, pl.pairs);
        }
        if (first) seg0 = step;
    }
    // The next sequence with units (B: none).  Out of line: the roles call it once a sequence and share the
    // instruction cache.
    static __device__ __noinline__ int next_seq(const TreeArgs &a, int b) {
        while (++b < a.B) {
            const Seq n = seq_of(a, b);
            if (n.steps > 0 && n.tiles > 0) break;
        }
        return b;
    }
};

struct Ring {
    int i;
    uint32_t ph;
    __device__ void adv(int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1u;
        }
    }
};

// The pair's run: every CTA scans the batch's tiles and units (two passes where the batch is larger than
// the block); pair 0 also leaves the offsets for the join.  One sequence that is no tree refuses all: no
// units, and no tiles for the join.
__device__ __noinline__ void schedule(const TreeArgs &a, const TreePlan &pl, int pair, uint32_t rank, Ctrl *c) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    auto block_scan = [&](long long &u, int &t, long long &all_u, int &all_t) {  // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long yu = __shfl_up_sync(0xffffffffu, u, o);
            const int yt = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) {
                u += yu;
                t += yt;
            }
        }
        if (lane == 31) {
            c->scan_u[w] = u;
            c->scan_t[w] = t;
        }
        __syncthreads();
        long long bu = 0;
        int bt = 0;
        all_u = 0;
        all_t = 0;
        for (int k = 0; k < THREADS / 32; ++k) {
            if (k < w) {
                bu += c->scan_u[k];
                bt += c->scan_t[k];
            }
            all_u += c->scan_u[k];
            all_t += c->scan_t[k];
        }
        u += bu;
        t += bt;
        __syncthreads();
    };
    const bool report = pair == 0 && rank == 0;
    if (tid == 0) c->w_n = 0;
    bool bad = false, bad_len = false;
    auto read = [&](int b, Seq &q, long long &u, int &t) {  // sequence b's units and tiles; 0 behind the batch
        u = 0;
        t = 0;
        TreeSpan sp;
        if (b >= a.B) return;
        const int L = a.seq_lens[b];  // beside the offsets
        if (!tree_span(a.cu, b, a.B, a.T, a.max_nodes, &sp)) {
            bad = true;
            return;
        }
        q = seq_of(a, sp.t0, sp.n, L);
        bad_len |= q.n > 0 && q.steps == 0;
        t = q.tiles;
        u = (long long)t * q.steps;
    };
    // Sequence b with `mine` units up to the inclusive sums u1 and t1: the pair's start if it lies there.
    auto place = [&](int b, const Seq &q, long long u1, long long mine, int t1, long long U, bool refuse) {
        const long long s0 = unit_start(pair, U, pl.pairs), s1 = unit_start(pair + 1, U, pl.pairs), u0 = u1 - mine;
        if (b >= a.B) return;
        if (!refuse && mine > 0 && u0 <= s0 && s0 < u1 && s1 > s0) {
            c->w_b = b;
            c->w_tile = (int)((s0 - u0) / q.steps);
            c->w_step = (int)((s0 - u0) % q.steps);
            c->w_n = (int)(s1 - s0);
            c->w_units = U;
            c->w_end = s1;
        }
        // The records of the tiles that begin in the run: every tile has one before any wait, so that the join finds
        // none of an earlier call's after a give-up.
        if (!refuse && rank == 0 && mine > 0 && u0 < s1 && s0 < u1) {
            for (long long k = s0 > u0 ? (s0 - u0 + q.steps - 1) / q.steps : 0; k < q.tiles && u0 + k * q.steps < s1; ++k) {
                const long long v = u0 + k * q.steps, last = v + q.steps - 1;
                const int n = last < s1 ? 1 : pair_of_unit(last, U, pl.pairs) - pair + 1;
                pl.tile[t1 - q.tiles + k] = make_int4(q.t0 * a.n_h + (int)k * TILE, q.n * a.n_h - (int)k * TILE, pair, v == s0 ? n : -n);
            }
        }
        if (report) {
            if (!refuse && q.steps == 0)  // nobody's: the join writes 0 and -inf
                for (int t = 0; t < q.tiles; ++t)
                    pl.tile[t1 - q.tiles + t] = make_int4(q.t0 * a.n_h + t * TILE, q.n * a.n_h - t * TILE, 0, 0);
            if (b == a.B - 1) {
                *pl.units = refuse ? 0 : U;
                *pl.tiles = refuse ? 0 : t1;
            }
        }
    };
    Seq q = {};
    if (a.B <= THREADS) {  // one pass, every length read once
        long long u, all_u;
        int t, all_t;
        read(tid, q, u, t);
        const long long mine = u;
        block_scan(u, t, all_u, all_t);
        bad = __syncthreads_or(bad);
        place(tid, q, u, mine, t, bad ? 0 : all_u, bad);
    } else {
        long long U = 0;
        for (int b0 = 0; b0 < a.B; b0 += THREADS) {
            long long u, all_u;
            int t, all_t;
            read(b0 + tid, q, u, t);
            block_scan(u, t, all_u, all_t);
            U += all_u;
        }
        bad = __syncthreads_or(bad);
        const bool refuse = bad;
        long long cu = 0;
        int ct = 0;
        for (int b0 = 0; b0 < a.B; b0 += THREADS) {
            long long u, all_u;
            int t, all_t;
            read(b0 + tid, q, u, t);
            const long long mine = u;
            block_scan(u, t, all_u, all_t);
            place(b0 + tid, q, cu + u, mine, ct + t, refuse ? 0 : U, refuse);
            cu += all_u;
            ct += all_t;
        }
        bad = refuse;
    }
    if (report && (bad || bad_len)) record_error(a.err, bad ? kErrBadTree : kErrBadSeqLen);
    __syncthreads();
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ bool named_red_or(bool v, int id, int n) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(n)
        : "memory");
    return r != 0;
}

// Four e4m3 codes (low byte first) as fp16 values, exactly (NaN stays NaN).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((unsigned short)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((unsigned short)(w >> 16)));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// At least log2 of a scale's size, by less than 1; a smaller one counts as 2^-80.  (exp2(score - m) reaches 2^(15 + 80)
// then, and the sum of 2^31 of them 2^126: it stays in fp32.)
__device__ __forceinline__ int scale_exponent(float s) { return max((int)(__float_as_uint(s) >> 23 & 255u) - 126, -80); }
// A pair of bf16 values with 0 for infinities and NaN.
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {
    return x & ((x & 0x7f80u) == 0x7f80u ? 0xffff0000u : 0xffffffffu) & ((x & 0x7f800000u) == 0x7f800000u ? 0xffffu : 0xffffffffu);
}

// Two fp32 values an instruction, and a maximum of three: fewer instructions are also less power, which holds the clock
// over bf16 (ragged batch 443 -> 431 us).
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(lo), "r"(hi));
    return x;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) { return pair_of(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 floats_of(uint64_t x) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(x));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void ld_shared_v4(uint32_t at, uint32_t *x) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
}

// A thread's four chunks of codes where they landed, rows row0 (even k) and row0 + 32: 0 behind the sequence, and
// for NaN in drafted rows.  Ahead of the conversion: selects in its loop cost every page 10%, in its registers 2%.
__device__ __noinline__ void clean_codes(uint32_t src, int odd, int row0, int drafted, int end) {
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
        const int row = row0 + 32 * (k & 1);
        const uint32_t at = src + ((k >> 1) ^ odd) * 64 + (k & 1) * 4096;
        if (row < drafted) continue;
        uint32_t w[4];
        ld_shared_v4(at, w);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = row >= end ? 0u : w[q] & ~__vcmpeq4(w[q] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        st_shared_v4(at, w[0], w[1], w[2], w[3]);
    }
}

// FP8: a landed query row (nine blocks of 64 bf16 columns) becomes, in place, 2^k times itself as e4m3 operands
// against the codes: of the row's 128 columns from 128 i, the nearest codes in block 2 i and the codes of
// what is left in block 2 i + 1; the RoPE columns stay bf16.  2^k puts the row's largest content element in
// [128, 256).  A bf16 value has 8 significant bits and a code 4, so both parts together are the value itself,
// down to 2^-9 of the row's largest; below, they are within 2^-17 of that largest.  Scores come out as
// multiples of 2^-k, the row's `unit`.  (A content element that is not finite makes every score of its row NaN.)
// k is 68 at most, so that the RoPE columns stay in range: 2^-61 counts as the largest of a row with less.  Eight
// lanes a row; a lane holds all its 64 columns before it writes.
__device__ __forceinline__ void split_query(uint32_t q, int row, int c, float *unit) {
    const uint32_t at = q + row * 128, key = row & 7, half = c >> 2, ch = 2 * (c & 3);
    uint32_t x[4][8], top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // columns 128 i + 16 c .. + 15
        ld_shared_v4(at + (2 * i + half) * CB + ((ch ^ key) << 4), x[i]);
        ld_shared_v4(at + (2 * i + half) * CB + (((ch + 1) ^ key) << 4), x[i] + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = __vmaxu2(top, x[i][j] & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));  // the row's largest, as bf16 bits
    const int e = min(max((int)(top >> 7), 66), 254);  // its exponent + 127
    const float mul = __uint_as_float(top >= 0x7f80u ? 0x7fc00000u : (uint32_t)(134 + 127 - e) << 23);
    if (c == 0) unit[row] = __uint_as_float((uint32_t)(e - 7) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __half2 v = __floats2half2_rn(__uint_as_float(x[i][j] << 16) * mul, __uint_as_float(x[i][j] & 0xffff0000u) * mul);
            unsigned short h, r;
            uint32_t near;
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(near) : "h"(h));
            const __half2 rest = __hsub2(v, *reinterpret_cast<const __half2 *>(&near));
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&rest)));
            hi[j >> 1] = j & 1 ? hi[j >> 1] | (uint32_t)h << 16 : h;
            lo[j >> 1] = j & 1 ? lo[j >> 1] | (uint32_t)r << 16 : r;
        }
        st_shared_v4(at + 2 * i * CB + ((c ^ key) << 4), hi[0], hi[1], hi[2], hi[3]);
        st_shared_v4(at + (2 * i + 1) * CB + ((c ^ key) << 4), lo[0], lo[1], lo[2], lo[3]);
    }
    const uint32_t rope = at + (NCB - 1) * CB + ((c ^ key) << 4);
    uint32_t y[4];
    ld_shared_v4(rope, y);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = pack_bf16x2(__uint_as_float(y[j] << 16) * mul, __uint_as_float(y[j] & 0xffff0000u) * mul);
    st_shared_v4(rope, y[0], y[1], y[2], y[3]);
}

// Which of the 32 tokens j .. j + 31 a node sees: all before ctx, its mask's bits from there, none behind L.
__device__ __forceinline__ uint32_t sees32(const uint32_t *mask, int words, int j, int ctx, int L) {
    const int rem = L - j, k = j - ctx;
    if (rem <= 0) return 0u;
    uint32_t v = 0xffffffffu;
    if (k > -32) {
        auto word = [&](int w) { return w < words ? mask[w] : 0u; };
        if (k < 0)
            v = (0xffffffffu >> (32 + k)) | (word(0) << -k);
        else
            v = __funnelshift_r(word(k >> 5), word((k >> 5) + 1), k & 31);
    }
    return rem < 32 ? v & (0xffffffffu >> (32 - rem)) : v;
}

// tm_k, tm_v: column blocks of the bf16 cache; FP8: tm_k the RoPE keys, tm_v and tm_c a page's codes as boxes of
// 128 columns, as they are and in the operands' layout (unused in the bf16 kernel).
template <bool F8, bool TURN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_c,
               const __grid_constant__ TreeArgs a, const __grid_constant__ TreePlan pl) {
    constexpr int K_STAGES = Lay<F8>::k_stages, V_STAGES = Lay<F8>::v_stages, V_OFF = Lay<F8>::v_off;
    constexpr int S_BUFS = Lay<F8>::s_bufs, KST = F8 ? F8_KST : NCB;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw), data_s = (raw_s + 1023u) & ~1023u;
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem_raw + (data_s - raw_s) + DATA);
    volatile uint32_t *abort_flag = &ctrl->abort;
    auto bar = [&](uint64_t &b) { return smem_u32(&b); };
    auto lead = [&](uint64_t &b) { return mapa(smem_u32(&b), 0); };  // the even CTA's barrier
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < MAX_STAGES; ++i) {
            mbar_init(bar(ctrl->k_full[i]), 2);
            mbar_init(bar(ctrl->k_empty[i]), 1);
            mbar_init(bar(ctrl->v_full[i]), F8 ? 2 * CLEAN_THREADS / 32 : 2);
            mbar_init(bar(ctrl->v_empty[i]), 1);
            mbar_init(bar(ctrl->land[i]), 1);
        }
        for (int i = 0; i < RAW_STAGES; ++i) {
            mbar_init(bar(ctrl->vraw_full[i]), 1);
            mbar_init(bar(ctrl->vraw_empty[i]), CLEAN_THREADS / 32);
        }
        mbar_init(bar(ctrl->q_land), 1);
        mbar_init(bar(ctrl->q_full), F8 ? 2 * CLEAN_THREADS / 32 : 2);
        mbar_init(bar(ctrl->q_empty), 1);
        mbar_init(bar(ctrl->never_done), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(ctrl->s_full[i]), 1);
            mbar_init(bar(ctrl->s_free[i]), 2 * SM_WARPS);
            mbar_init(bar(ctrl->o_ok[i]), 2 * SM_WARPS);
            mbar_init(bar(ctrl->pv_done[i]), 1);
        }
        for (int i = 0; i < SPG; ++i) {
            mbar_init(bar(ctrl->p_full[i]), 2 * SM_WARPS / SPG);
            mbar_init(bar(ctrl->p_free[i]), 1);
        }
        ctrl->abort = 0;
        fence_mbarrier_init_cluster();
    }
    if (warp == QK_WARP) {
        tmem_alloc_pair(smem_u32(&ctrl->tmem_base), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    pdl_trigger();
    pdl_wait();  // inputs are read from here on
    schedule(a, pl, pair, rank, ctrl);
    const uint32_t tmem = ctrl->tmem_base;
    auto fail = [&]() {
        *abort_flag = 1;
        st_shared_cluster_u32(mapa(smem_u32(&ctrl->abort), rank ^ 1u), 1u);
        record_error(a.err, kErrTimeout);
    };

    if ((warp == LOAD_K_WARP || warp == LOAD_V_WARP) && lane == 0) {  // ================= loads =================
        const bool kw = warp == LOAD_K_WARP;
        Walk<TURN> it;
        it.init(a, pl, ctrl);
        Ring st{0, 0};
        uint32_t q_ph = 1;
        bool ok = true;
        int ids[SPG];
        uint32_t raw = 0;  // FP8: code stages sent so far
        auto pages = [&]() {
#pragma unroll
            for (int p = 0; p < SPG; ++p) {
                const int pg = it.at(it.step) * SPG + p;
                ids[p] = -1;
                if (!it.done() && pg * PG < it.s.L) {
                    int blk = a.bt[(size_t)it.b * a.max_blocks + pg];
                    if (blk < 0 || blk >= a.num_blocks) {
                        record_error(a.err, kErrBadBlock);
                        blk = 0;  // in bounds; the result is flagged
                    }
                    ids[p] = blk;
                }
            }
        };
        if (!it.done()) {
            prefetch_tensormap(&tm_q);
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
            if (F8) prefetch_tensormap(&tm_c);
            pages();
        }
        bool begun = false;
        while (ok && kw && !it.done()) {  // Q per segment; K: the CTA's two pages, a column block a stage
            // the failure path's test: the first step's copies are under way, a short wait runs out
            if (a.test_give_up && begun && !(ok = wait(bar(ctrl->never_done), 0u, abort_flag, 20000ull))) break;
            begun = true;
            if (it.first) {
                if (!(ok = wait(bar(ctrl->q_empty), q_ph, abort_flag))) break;
                q_ph ^= 1u;
                const int q0 = it.s.t0 * a.n_h + it.tile * TILE + (int)rank * HALF;
                if (F8) {
                    mbar_arrive_expect_tx(bar(ctrl->q_land), NCB * CB);
                    tma_load_3d(data_s + Q_OFF, &tm_q, 0, q0, 0, bar(ctrl->q_land));
                } else {
                    mbar_arrive_expect_tx_remote(lead(ctrl->q_full), NCB * CB);
                    tma_load_3d_pair(data_s + Q_OFF, &tm_q, 0, q0, 0, lead(ctrl->q_full));
                }
            }
            const int p0 = rank ? ids[2] : ids[0], p1 = rank ? ids[3] : ids[1];
            it.next(a, pl, ctrl);
            pages();  // of the next step: the table's latency passes under this one's loads
            for (int cb = 0; ok && cb < KST; ++cb) {
                if (!(ok = wait(bar(ctrl->k_empty[st.i]), st.ph ^ 1u, abort_flag))) break;
                const uint32_t dst = data_s + K_OFF + st.i * STAGE, full = lead(ctrl->k_full[st.i]);
                mbar_arrive_expect_tx_remote(full, (p0 >= 0 ? CB : 0) + (p1 >= 0 ? CB : 0));
                if (F8 && cb < KST - 1) {
                    if (p0 >= 0) tma_load_2d_pair(dst, &tm_c, cb * 128, p0 * PG, full);
                    if (p1 >= 0) tma_load_2d_pair(dst + CB, &tm_c, cb * 128, p1 * PG, full);
                } else {
                    if (p0 >= 0) tma_load_3d_pair(dst, &tm_k, 0, p0 * PG, F8 ? 0 : cb, full);
                    if (p1 >= 0) tma_load_3d_pair(dst + CB, &tm_k, 0, p1 * PG, F8 ? 0 : cb, full);
                }
                st.adv(K_STAGES);
            }
        }
        while (ok && !kw && !it.done()) {  // V: a page's 128 columns of each half of O a stage
            int id[SPG];
#pragma unroll
            for (int p = 0; p < SPG; ++p) id[p] = ids[p];
            const int pg0 = it.at(it.step) * SPG, ctx = it.s.ctx, np = it.pages();
            it.next(a, pl, ctrl);
            pages();
#pragma unroll
            for (int p = 0; p < SPG; ++p) {
                const bool clean = (pg0 + p + 1) * PG > ctx;
                for (int nh = 0; ok && p < np && nh < 2; ++nh) {
                    if (F8) {
                        if (!(ok = wait(bar(ctrl->vraw_empty[raw % RAW_STAGES]), ((raw / RAW_STAGES) & 1) ^ 1, abort_flag))) break;
                        const uint32_t land = bar(ctrl->vraw_full[raw % RAW_STAGES]);
                        mbar_arrive_expect_tx(land, RAW);
                        tma_load_2d(data_s + Lay<F8>::vraw_off + (raw % RAW_STAGES) * RAW, &tm_v, nh * 256 + (int)rank * 128, id[p] * PG, land);
                        ++raw;
                        st.adv(V_STAGES);
                        continue;
                    }
                    if (!(ok = wait(bar(ctrl->v_empty[st.i]), st.ph ^ 1u, abort_flag))) break;
                    const uint32_t dst = data_s + V_OFF + st.i * STAGE, full = lead(ctrl->v_full[st.i]);
                    const int z = nh * 4 + (int)rank * 2;
                    if (!clean) {
                        mbar_arrive_expect_tx_remote(full, STAGE);
                        tma_load_3d_pair(dst, &tm_v, 0, id[p] * PG, z, full);
                    } else {
                        mbar_arrive_expect_tx(bar(ctrl->land[st.i]), STAGE);
                        tma_load_3d(dst, &tm_v, 0, id[p] * PG, z, bar(ctrl->land[st.i]));
                    }
                    st.adv(V_STAGES);
                }
            }
        }
        // the last arrivals on this CTA's barriers have come before it may leave (once per stage; a stage
        // that no unit filled passes at once)
        if (ctrl->w_n > 0) {
            for (int i = 0; ok && i < (kw ? K_STAGES : V_STAGES); ++i) {
                ok = wait(bar(kw ? ctrl->k_empty[st.i] : ctrl->v_empty[st.i]), st.ph ^ 1u, abort_flag);
                st.adv(kw ? K_STAGES : V_STAGES);
            }
            if (ok && kw) ok = wait(bar(ctrl->q_empty), q_ph, abort_flag);
        }
        if (!ok) fail();
    } else if (warp == QK_WARP && lane == 0 && rank == 0) {  // ================= S of both CTAs =================
        constexpr uint32_t idesc = idesc_bf16(TILE, STEP, false, false), idesc_f8 = idesc_e4m3(TILE, STEP);
        Walk<TURN> it;
        it.init(a, pl, ctrl);
        Ring st{0, 0};
        uint32_t q_ph = 0;
        constexpr uint32_t HI = sdesc_sw128_hi(1024);
        const uint32_t q_lo = sdesc_sw128_lo(data_s + Q_OFF, 16), k_lo = sdesc_sw128_lo(data_s + K_OFF, 16);
        bool ok = true;
        for (int u = 0; ok && !it.done(); ++u) {
            const int sb = u % S_BUFS;
            if (it.first) {
                if (!(ok = wait(bar(ctrl->q_full), q_ph, abort_flag))) break;
                q_ph ^= 1u;
            }
            if (!(ok = wait(bar(ctrl->s_free[sb]), ((u / S_BUFS) & 1) ^ 1, abort_flag))) break;
#pragma unroll 1
            for (int cb = 0; cb < KST; ++cb) {
                if (!(ok = wait(bar(ctrl->k_full[st.i]), st.ph, abort_flag))) break;
                tc_fence_after();
                const uint32_t kl = k_lo + st.i * (STAGE >> 4);
                if (F8 && cb < KST - 1) {  // 128 columns of codes against both parts of the queries
                    const uint32_t ql = q_lo + 2 * cb * (CB >> 4);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ss_pair_f8(tmem + S_COL, ql + (k >> 2) * (CB >> 4) + 2 * (k & 3), kl + 2 * (k & 3), HI, idesc_f8, cb > 0 || k > 0);
                } else {  // FP8: the RoPE part of the scores apart, it takes no scale
                    const uint32_t ql = q_lo + (F8 ? NCB - 1 : cb) * (CB >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss_pair(tmem + S_COL + (F8 ? 128 : sb * 128), ql + 2 * k, kl + 2 * k, HI, idesc, (!F8 && cb > 0) || k > 0);
                }
                mma_commit_pair(bar(ctrl->k_empty[st.i]));
                st.adv(K_STAGES);
            }
            if (!ok) break;
            mma_commit_pair(bar(ctrl->s_full[sb]));
            if (it.last()) mma_commit_pair(bar(ctrl->q_empty));
            it.next(a, pl, ctrl);
        }
        if (!ok) fail();
    } else if (warp == PV_WARP && lane == 0 && rank == 0) {  // ================= O of both CTAs =================
        constexpr uint32_t idesc = F8 ? idesc_f16(TILE, 256, false, true) : idesc_bf16(TILE, 256, false, true);
        Walk<TURN> it;
        it.init(a, pl, ctrl);
        Ring st{0, 0};
        constexpr uint32_t HI = sdesc_sw128_hi(1024);
        const uint32_t p_lo = sdesc_sw128_lo(data_s + P_OFF, 16), v_lo = sdesc_sw128_lo(data_s + V_OFF, CB);
        uint32_t p_ph = 0;  // a bit per page: a step's last pages may not be there
        bool ok = true;
        for (int u = 0; ok && !it.done(); ++u) {
            if (!(ok = wait(bar(ctrl->o_ok[u & 1]), (u >> 1) & 1, abort_flag))) break;
            const int np = it.pages();
            for (int p = 0; ok && p < np; ++p) {
                if (!(ok = wait(bar(ctrl->p_full[p]), (p_ph >> p) & 1u, abort_flag))) break;
                p_ph ^= 1u << p;
                const uint32_t pl_ = p_lo + p * (CB >> 4);
                const bool acc = !it.first || p > 0;
#pragma unroll 1
                for (int nh = 0; nh < 2; ++nh) {
                    if (!(ok = wait(bar(ctrl->v_full[st.i]), st.ph, abort_flag))) break;
                    tc_fence_after();
                    const uint32_t vl = v_lo + st.i * (STAGE >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss_pair(tmem + O_COL + nh * 128, pl_ + 2 * k, vl + 128 * k, HI, idesc, acc || k > 0);
                    mma_commit_pair(bar(ctrl->v_empty[st.i]));
                    st.adv(V_STAGES);
                }
                if (ok) mma_commit_pair(bar(ctrl->p_free[p]));
            }
            if (!ok) break;
            mma_commit_pair(bar(ctrl->pv_done[u & 1]));
            it.next(a, pl, ctrl);
        }
        if (!ok) fail();
    } else if (F8 && warp >= CLEAN_WARP0) {  // ================= FP8: Q in two parts, V's codes to fp16 tiles =================
        const int t = threadIdx.x - CLEAN_WARP0 * 32;
        Walk<TURN> it;
        it.init(a, pl, ctrl);
        Ring st{0, 0};
        uint32_t q_ph = 0;
        uint32_t raw = 0;
        bool ok = true;
        while (ok && !it.done()) {
            if (it.first) {  // each warp the rows that it splits, and for itself: a warp that gave up waits for no other
                const bool good = wait(bar(ctrl->q_land), q_ph, abort_flag);
                for (int r0 = 0; r0 < HALF; r0 += CLEAN_THREADS / 8) split_query(data_s + Q_OFF, r0 + (t >> 3), t & 7, ctrl->q_unit[q_ph]);
                q_ph ^= 1u;
                fence_proxy_async_smem();
                if (!(ok = __all_sync(0xffffffffu, good))) break;
                __syncwarp();  // a vote orders no memory
                if (lane == 0) mbar_arrive_pair(lead(ctrl->q_full));
            }
            for (int i = 0, n = 2 * it.pages(); i < n; ++i, ++raw, st.adv(V_STAGES)) {
                const bool good = wait(bar(ctrl->vraw_full[raw % RAW_STAGES]), (raw / RAW_STAGES) & 1, abort_flag) &&
                                  wait(bar(ctrl->v_empty[st.i]), st.ph ^ 1u, abort_flag);
                const int j0 = (it.at(it.step) * SPG + (i >> 1)) * PG;        // the page's first token
                const int drafted = it.s.ctx - j0, end = it.s.L - j0;  // the first drafted row, and the sequence's end
                // A thread takes four chunks of 16 codes, columns 16 c of two rows of two blocks, odd rows the blocks the
                // other way round so that eight lanes read 128 different bytes modulo 128.  Its loads come before its
                // stores, each of which would hold the next load back.
                const int c = t & 3, row0 = t >> 2, odd = row0 & 1;
                const uint32_t src = data_s + Lay<F8>::vraw_off + (raw % RAW_STAGES) * RAW + row0 * 128 + c * 16;
                const uint32_t dst = data_s + V_OFF + st.i * STAGE + row0 * 128;
                const uint32_t dst0 = dst + (((2 * c) ^ (row0 & 7)) << 4), dst1 = dst + (((2 * c + 1) ^ (row0 & 7)) << 4);
                if (drafted < PG) clean_codes(src, odd, row0, drafted, end);
                uint32_t w[4][4];
#pragma unroll
                for (int k = 0; k < 4; ++k)  // block k / 2 (odd rows: the other), rows row0 and row0 + 32
                    ld_shared_v4(src + ((k >> 1) ^ odd) * 64 + (k & 1) * 4096, w[k]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t o[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) e4m3x4_to_f16x4(w[k][q], o[2 * q], o[2 * q + 1]);
                    st_shared_v4(dst0 + ((k >> 1) ^ odd) * CB + (k & 1) * 4096, o[0], o[1], o[2], o[3]);
                    st_shared_v4(dst1 + ((k >> 1) ^ odd) * CB + (k & 1) * 4096, o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async_smem();
                if (!(ok = __all_sync(0xffffffffu, good))) break;
                __syncwarp();
                if (lane == 0) {  // each warp for itself: a barrier among the four cost 4% of the whole
                    mbar_arrive_pair(lead(ctrl->v_full[st.i]));
                    mbar_arrive(bar(ctrl->vraw_empty[raw % RAW_STAGES]));
                }
            }
            it.next(a, pl, ctrl);
        }
        if (!ok && lane == 0) fail();
    } else if (warp >= CLEAN_WARP0) {  // ================= V rows not seen by all =================
        const int t = threadIdx.x - CLEAN_WARP0 * 32;
        Walk<TURN> it;
        it.init(a, pl, ctrl);
        Ring st{0, 0};
        uint32_t land_ph = 0;  // a bit per stage: only the stages that are cleaned use their barrier
        bool ok = true;
        while (ok && !it.done()) {
            for (int v = 0; ok && v < 2 * it.pages(); ++v, st.adv(V_STAGES)) {
                const int j0 = (it.at(it.step) * SPG + (v >> 1)) * PG;
                if (j0 + PG <= it.s.ctx) continue;
                const bool good = wait(bar(ctrl->land[st.i]), (land_ph >> st.i) & 1u, abort_flag);
                land_ph ^= 1u << st.i;
                const uint32_t base = data_s + V_OFF + st.i * STAGE + (t & 8) / 8 * CB + (t & 7) * 16;
#pragma unroll
                for (int k = 0; k < PG * 16 / CLEAN_THREADS; ++k) {  // this thread's 16-byte chunk of every eighth row
                    const int row = k * (CLEAN_THREADS / 16) + (t >> 4), j = j0 + row;
                    const uint32_t at = base + row * 128;
                    uint32_t x[4];
                    ld_shared_v4(at, x);
                    bool hit = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t y = j >= it.s.L ? 0u : finite_pair(x[i]);
                        hit |= y != x[i];
                        x[i] = y;
                    }
                    if (hit && j >= it.s.ctx) st_shared_v4(at, x[0], x[1], x[2], x[3]);
                }
                fence_proxy_async_smem();
                if (!(ok = !named_red_or(!good, BAR_CLEAN, CLEAN_THREADS))) break;
                if (t == 0) mbar_arrive_pair(lead(ctrl->v_full[st.i]));
            }
            it.next(a, pl, ctrl);
        }
        if (!ok && lane == 0) fail();
    } else if (warp >= SM_WARP0 && warp < SM_WARP0 + SM_WARPS) {  // ================= softmax, P, O =================
        // thread: row r of the CTA against page pg of the step (64 columns of S), and 128 of O's columns
        const int r = (warp & 1) * 32 + lane, half = (warp >> 1) & 1, cg = (warp - SM_WARP0) >> 2, pg = 2 * half + cg;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t p_row = data_s + P_OFF + (uint32_t)pg * CB + r * 128;
        const uint32_t stage = data_s + P_OFF + (warp - SM_WARP0) * 2048;  // this warp's share of P, between tiles
        Walk<TURN> it;
        it.init(a, pl, ctrl);
        float m = -INFINITY, l = 0.f;
        int before = 0;  // steps so far that had the page pg
        bool ok = true, good = true;
        float sc0 = 0.f, sc1 = 0.f;
        int sc_top = 0;
        bool sc_near = true;
        float(*scales)[PG] = ctrl->scale[warp - SM_WARP0];
        int next_block = -1;  // the page's in the tile's next step
        auto block_of = [&](int step) {
            const int g = it.at(step) * SPG + pg;
            return g * PG < it.s.L ? a.bt[(size_t)it.b * a.max_blocks + g] : -1;
        };
        auto load_scales = [&](int blk) {
            sc0 = sc1 = 0.f;
            if (blk < 0 || blk >= a.num_blocks) return;  // the loader reports a bad one
            const float *src = a.kv_scale + (size_t)blk * PG + lane;
            sc0 = src[0];
            sc1 = src[32];
        };
        float to_log2 = a.scale_log2;  // a score of S to log2 units
        int seg = 0;
        for (int u = 0; ok && !it.done(); ++u) {
            const int row = it.tile * TILE + (int)rank * HALF + r;  // of the sequence's (node, head) pairs
            const bool mine = row < it.s.n * a.n_h;
            const int sb = u & 1, buf = u % S_BUFS;
            if (F8) {  // the page's scales, before S is there
                if (it.first) {
                    load_scales(block_of(it.step));
                    next_block = block_of(it.step + 1);
                }
                scales[0][lane] = sc0;
                scales[0][lane + 32] = sc1;
                sc0 = fabsf(sc0) <= FLT_MAX ? sc0 : 0.f;
                sc1 = fabsf(sc1) <= FLT_MAX ? sc1 : 0.f;
                scales[1][lane] = sc0;
                scales[1][lane + 32] = sc1;
                const int e0 = scale_exponent(sc0), e1 = scale_exponent(sc1);
                sc_top = __shfl_sync(0xffffffffu, e0, 0) + 2;
                sc_near = __all_sync(0xffffffffu, e0 <= sc_top && e0 >= sc_top - 4 && e1 <= sc_top && e1 >= sc_top - 4);
                __syncwarp();
            }
            good = __all_sync(0xffffffffu, good && wait(bar(ctrl->s_full[buf]), (u / S_BUFS) & 1, abort_flag));
            tc_fence_after();
            uint32_t v[PG];
            if (F8 && it.first) to_log2 = a.scale_log2 * ctrl->q_unit[seg++ & 1][r];
            if (good) {
                const uint32_t sa = tmem + lane_base + S_COL + buf * 128 + cg * PG;
                if (F8) {  // content scores times the tokens' scales, and the RoPE scores
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_ld32(sa + 128 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
#pragma unroll
                    for (int c = 0; c < PG / 16; ++c) {
                        uint32_t x[16];
                        tmem_ld16(sa + c * 16, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 sc = *reinterpret_cast<const float4 *>(&scales[0][16 * c + j]);
                            const uint64_t t[2] = {pair_of(sc.x, sc.y), pair_of(sc.z, sc.w)};
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t *y = v + 16 * c + j + 2 * i;
                                const float2 d = floats_of(fma2(pair_of(x[j + 2 * i], x[j + 2 * i + 1]), t[i], pair_of(y[0], y[1])));
                                y[0] = __float_as_uint(d.x);
                                y[1] = __float_as_uint(d.y);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_ld32(sa + c * 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
                    tmem_wait_ld();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(ctrl->s_free[buf]));
            }
            if (F8 && !it.last()) {  // on their way under this step, and the table's entry two steps ahead, so that nothing waits
                load_scales(next_block);
                next_block = block_of(it.step + 2);
            }
            const int j0 = it.at(it.step) * STEP + pg * PG;
            if (j0 + PG > it.s.ctx) {
                const uint32_t *mask = a.mask + (size_t)(it.s.t0 + (mine ? row / a.n_h : 0)) * a.mask_words;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t see = sees32(mask, a.mask_words, j0 + 32 * w, it.s.ctx, it.s.L);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!((see >> j) & 1u)) v[32 * w + j] = 0xff800000u;  // -inf
                }
            }
            // The largest score in log2 units.  FP8: P is exp2(score - m) times the token's scale, in fp16, so m bounds
            // score + log2(scale) - 7.  P's largest is then between 2^2 and 2^7, and below 2^15 when m moves.  The scales
            // of a page count as four times its first where all are within 2^2 of that, else each as it is.
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            float top;
            if (!F8 || sc_near) {
#pragma unroll
                for (int j = 0; j < PG; j += 2) x[j >> 1 & 3] = max3(x[j >> 1 & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                top = max3(fmaxf(x[0], x[1]), x[2], x[3]) * to_log2 + (F8 ? (float)(sc_top - 7) : 0.f);
            } else {
#pragma unroll
                for (int j = 0; j < PG; ++j)
                    x[j & 3] = fmaxf(x[j & 3], fmaf(__uint_as_float(v[j]), to_log2, (float)(scale_exponent(scales[1][j]) - 7)));
                top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
            }
            ctrl->top[sb][pg][r] = top;
            if (named_red_or(!good, BAR_MAX, SM_THREADS)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int k = 0; k < SPG; ++k) top = fmaxf(top, ctrl->top[sb][k][r]);
            float fac = 1.f;
            if (it.first) {
                m = top;
                l = 0.f;
            } else if (top > m + RESCALE_LOG2 || m == -INFINITY) {
                fac = m == -INFINITY ? 0.f : ex2(m - top);
                m = fmaxf(m, top);
            }
            const float base = m == -INFINITY ? 0.f : m;
            uint64_t s0 = 0, s1 = 0;
            const uint64_t mul = pair_of(to_log2, to_log2), sub = pair_of(-base, -base);
#pragma unroll
            for (int j = 0; j < PG / 4; ++j) {  // P as 16-bit pairs, into the front half of v
                const float2 a0 = floats_of(fma2(pair_of(v[4 * j], v[4 * j + 1]), mul, sub));
                const float2 a1 = floats_of(fma2(pair_of(v[4 * j + 2], v[4 * j + 3]), mul, sub));
                uint64_t p0 = pair_of(ex2(a0.x), ex2(a0.y)), p1 = pair_of(ex2(a1.x), ex2(a1.y));
                s0 = add2(s0, p0);
                s1 = add2(s1, p1);
                if (F8) {  // the value product is over the codes: their scales go into P
                    const float4 sc = *reinterpret_cast<const float4 *>(&scales[1][4 * j]);
                    p0 = mul2(p0, pair_of(sc.x, sc.y));
                    p1 = mul2(p1, pair_of(sc.z, sc.w));
                }
                const float2 f0 = floats_of(p0), f1 = floats_of(p1);
                v[2 * j] = F8 ? pack_f16x2(f0.x, f0.y) : pack_bf16x2(f0.x, f0.y);
                v[2 * j + 1] = F8 ? pack_f16x2(f1.x, f1.y) : pack_bf16x2(f1.x, f1.y);
            }
            const float2 sum2 = floats_of(add2(s0, s1));
            l = l * fac + (sum2.x + sum2.y);
            // Every thread waits for every step's MMAs in turn, two steps behind (by then they are done): a wait by
            // parity tells two phases apart, not three.  The next vote hears of a failure.
            if (u >= 2) good = wait(bar(ctrl->pv_done[sb]), ((u >> 1) & 1) ^ 1, abort_flag);
            // a moved maximum rescales O, once the step before is in it
            if (!it.first && __any_sync(0xffffffffu, fac != 1.f)) {
                good = good && wait(bar(ctrl->pv_done[sb ^ 1]), ((u - 1) >> 1) & 1, abort_flag);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    uint32_t o[16];
                    tmem_ld16(tmem + lane_base + O_COL + cg * 128 + c * 16, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac);
                    tmem_st16(tmem + lane_base + O_COL + cg * 128 + c * 16, o);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_pair(lead(ctrl->o_ok[sb]));
            const int np = it.pages();
            if (pg < np) {  // P is 0 behind the last page, and nothing multiplies it
                // its MMAs of the step before (a tile's first step finds all of them done)
                if (!it.first) good = good && wait(bar(ctrl->p_free[pg]), (before - 1) & 1, abort_flag);
#pragma unroll
                for (int c = 0; c < PG / 8; ++c)  // eight tokens: one 16-byte chunk of P's row
                    st_shared_v4(p_row + ((c ^ (r & 7)) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(lead(ctrl->p_full[pg]));
            }
            before += pg < np;

            if (it.last()) {
                ctrl->sum[pg][r] = l;
                good = good && wait(bar(ctrl->pv_done[sb]), (u >> 1) & 1, abort_flag);
                if (named_red_or(!good, BAR_MAX, SM_THREADS)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float total = (ctrl->sum[0][r] + ctrl->sum[1][r]) + (ctrl->sum[2][r] + ctrl->sum[3][r]);
                const bool whole = it.seg0 == 0 && it.step == it.s.steps - 1;
                const int slot = 2 * pair + (it.head ? 0 : 1);
                const float inv = total == 0.f ? 0.f : 1.f / total;
                const int row0 = row - lane;  // this warp's first row of the sequence
                if (pg == 0) {
                    if (!whole) {
                        pl.m[slot * TILE + (int)rank * HALF + r] = total == total ? m : total;  // NaN scores move no maximum
                        pl.l[slot * TILE + (int)rank * HALF + r] = total;
                    } else if (mine && a.lse) {
                        a.lse[(size_t)it.s.t0 * a.n_h + row] =
                            total == 0.f ? -INFINITY : (base + log2f(total)) * 0.69314718055994531f;
                    }
                }
                if (!whole) {  // partial rows: a warp's store is four columns of 32 rows, four times 128 bytes
                    float *dst = pl.o + (((size_t)slot * (TILE / 8) + ((int)rank * HALF + r) / 8) * DC + cg * 256 + half * 128) * 8 + (r & 7) * 4;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tmem + lane_base + O_COL + cg * 128 + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            __stcg(reinterpret_cast<uint4 *>(dst + (c * 32 + i) * 8), make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
                    }
                } else {
                    // O's rows pass through 2 KB of P (its MMAs are done) a warp, 64 bytes of each of the 32 rows at a
                    // time, so that a store instruction writes whole sectors of eight rows, not 16 bytes of 32
                    const bool narrow = a.out_bf16;
                    const size_t width = narrow ? DC * 2 : DC * 4;
                    char *dst = reinterpret_cast<char *>(a.o) + ((size_t)it.s.t0 * a.n_h + row0) * width +
                                (cg * 256 + half * 128) * (narrow ? 2 : 4);
                    const int rows_left = it.s.n * a.n_h - row0;
                    const uint32_t mine_s = stage + lane * 64, key = (lane >> 1) & 3;
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {  // 16 of the 128 columns
                        uint32_t o[16];
                        tmem_ld16(tmem + lane_base + O_COL + cg * 128 + c * 16, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
                        if (narrow) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                o[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < 2 || !narrow)
                                st_shared_v4(mine_s + ((((narrow ? 2 * (c & 1) : 0) + i) ^ key) << 4), o[4 * i], o[4 * i + 1],
                                             o[4 * i + 2], o[4 * i + 3]);
                        if (narrow && !(c & 1)) continue;
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int rr = 8 * i + (lane >> 2), ch = lane & 3;
                            uint32_t x[4];
                            ld_shared_v4(stage + rr * 64 + ((ch ^ ((rr >> 1) & 3)) << 4), x);
                            if (rr < rows_left)
                                *reinterpret_cast<uint4 *>(dst + rr * width + (narrow ? c >> 1 : c) * 64 + ch * 16) =
                                    make_uint4(x[0], x[1], x[2], x[3]);
                        }
                        __syncwarp();
                    }
                }
            }
            it.next(a, pl, ctrl);
        }
        if (!(ok && good)) fail();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (*abort_flag) {  // copies and MMAs in flight land within microseconds
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 5000000ull) {
        }
        __syncthreads();
        cluster_sync();
    }
    if (warp == QK_WARP) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// Joins the tiles that lie in several pairs' runs: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.  A block
// takes eight rows, 16 contiguous KB of a slot's partials; a thread a row in 16 columns.  The block finds the
// slots and weights of its rows side by side first, so that the partials are read without waiting for one
// another.  Rows of a sequence without steps (a bad length) are 0 and -inf.
constexpr int JOIN_ROWS = 8, JOIN_THREADS = 256, JOIN_SLOTS = 128;
__global__ void __launch_bounds__(JOIN_THREADS)
tree_tc_join_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ TreePlan pl) {
    __shared__ float weight[JOIN_SLOTS][JOIN_ROWS];
    __shared__ int slots[JOIN_SLOTS];
    pdl_trigger();
    pdl_wait();
    const int g = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int4 t = __ldcg(&pl.tile[g]);  // beside the other two; of no use behind the last tile
    const long long U = *pl.units;
    if (g >= *pl.tiles) return;
    const int r0 = blockIdx.y * JOIN_ROWS, left = t.y, c0 = t.z, n = abs(t.w);
    if (r0 >= left || n == 1) return;
    // A pair without units left nothing: it counts with weight 0 and any slot of the tile's.  The first pair may
    // have begun with another tile.
    const int first = 2 * c0 + (t.w < 0);
    for (int i = tid; i < n; i += JOIN_THREADS)
        slots[i] = i == 0 ? first : unit_start(c0 + i, U, pl.pairs) == unit_start(c0 + i + 1, U, pl.pairs) ? -1 : 2 * (c0 + i);
    __syncthreads();
    // a warp per row: its maximum, weights and sum
    float M = -INFINITY, l = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float m = slots[i] < 0 ? -INFINITY : pl.m[slots[i] * TILE + r0 + warp];
        if (i < 32 && slots[i] >= 0) l = pl.l[slots[i] * TILE + r0 + warp];  // on its way beside m
        weight[i][warp] = m;
        M = fmaxf(M, m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float base = M == -INFINITY ? 0.f : M;
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float w = exp2f(weight[i][warp] - base);
        weight[i][warp] = w;
        if (w != 0.f) sum += w * (i < 32 ? l : pl.l[slots[i] * TILE + r0 + warp]);
    }
    l = sum;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    __syncwarp();
    if (l != 0.f) {
        for (int i = lane; i < n; i += 32) weight[i][warp] /= l;
    }
    if (a.lse && lane == 0 && r0 + warp < left)
        a.lse[(size_t)t.x + r0 + warp] = l == 0.f ? -INFINITY : (base + log2f(l)) * 0.69314718055994531f;
    __syncthreads();
    const int row = tid & 7, quad = tid >> 3;  // columns 4 quad .. + 3, + 128 k
    const float *src = pl.o + ((size_t)(r0 / 8) * DC + quad * 4) * 8 + row * 4;
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float w = weight[i][row];
        const float *part = src + (size_t)(slots[i] < 0 ? first : slots[i]) * TILE * DC;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(part + k * 128 * 8));
            acc[k].x = w == 0.f ? acc[k].x : fmaf(w, x.x, acc[k].x);
            acc[k].y = w == 0.f ? acc[k].y : fmaf(w, x.y, acc[k].y);
            acc[k].z = w == 0.f ? acc[k].z : fmaf(w, x.z, acc[k].z);
            acc[k].w = w == 0.f ? acc[k].w : fmaf(w, x.w, acc[k].w);
        }
    }
    if (r0 + row >= left) return;
    const size_t at = ((size_t)t.x + r0 + row) * DC + quad * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (a.out_bf16)
            *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.o) + at + 128 * k) =
                make_uint2(pack_bf16x2(acc[k].x, acc[k].y), pack_bf16x2(acc[k].z, acc[k].w));
        else
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.o) + at + 128 * k) = acc[k];
    }
}

// Pairs that run at once on the current device (0: it cannot be queried), looked up once.  All variants
// have the same launch shape and shared memory.
int tree_pairs() {
    static int known[64];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (known[dev]) return known[dev];
    int sms = 148, most = 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    for (auto kern : {tree_tc_kernel<false, false>, tree_tc_kernel<true, false>, tree_tc_kernel<false, true>, tree_tc_kernel<true, true>}) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (sms / 2));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = SMEM;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = sms / 2;
        }
        if (most == 0 || n < most) most = n;
    }
    return known[dev] = most < JOIN_SLOTS ? most : JOIN_SLOTS;
}

// Tiles of a batch at most: a sequence's last one may be part-filled.
int64_t tree_tiles(int B, int64_t rows) { return B + rows / TILE; }

size_t tree_tc_layout(int pairs, int B, int64_t rows, char *base, TreePlan *pl) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = base ? base + off : nullptr;
        off += align_up(bytes, 256);
        return p;
    };
    TreePlan t;
    t.pairs = pairs;
    t.units = reinterpret_cast<long long *>(take(sizeof(long long)));
    t.tiles = reinterpret_cast<int *>(take(sizeof(int)));
    t.tile = reinterpret_cast<int4 *>(take((size_t)tree_tiles(B, rows) * sizeof(int4)));
    t.o = reinterpret_cast<float *>(take((size_t)2 * pairs * TILE * DC * sizeof(float)));
    t.m = reinterpret_cast<float *>(take((size_t)2 * pairs * TILE * sizeof(float)));
    t.l = reinterpret_cast<float *>(take((size_t)2 * pairs * TILE * sizeof(float)));
    if (pl) *pl = t;
    return off;
}

}  // namespace

bool tree_tc_supported(const mla_dims_t &d) {
    return d.d_c == DC && d.d_r == ROW - DC && d.page_size == PG && d.act_dtype == MLA_DTYPE_BF16 &&
           (d.kv_dtype == MLA_DTYPE_BF16 || d.kv_dtype == MLA_DTYPE_FP8_E4M3) && !(d.flags & MLA_FLAG_SIMT_DECODE);
}

size_t tree_tc_workspace_bytes(const mla_dims_t &d, int B, int T) {
    const int pairs = tree_pairs();
    return pairs < 1 ? 0 : tree_tc_layout(pairs, B, (int64_t)T * d.n_h, nullptr, nullptr);
}

cudaError_t launch_tree_tc(const mla_dims_t &d, const TreeArgs &a, void *ws, cudaStream_t st) {
    const int pairs = tree_pairs();
    if (pairs < 1) return cudaErrorNotSupported;
    TreePlan pl;
    tree_tc_layout(pairs, a.B, (int64_t)a.T * a.n_h, reinterpret_cast<char *>(ws), &pl);
    const uint64_t pool_rows = (uint64_t)a.num_blocks * PG, q_rows = (uint64_t)a.T * a.n_h;
    const bool f8 = d.kv_dtype == MLA_DTYPE_FP8_E4M3;
    CUtensorMap tm_q, tm_k, tm_v, tm_c;
    const bool maps = f8 ? tmap_bf16_colblocks(&tm_k, a.kr_pool, pool_rows, ROW - DC, (ROW - DC) * 2, PG, 1) &&
                               tmap_u8_rows(&tm_v, a.kv_pool, DC, pool_rows, DC, 128, PG) &&
                               tmap_2d(&tm_c, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.kv_pool, DC, pool_rows, DC, 128, PG)
                         : tmap_bf16_colblocks(&tm_k, a.kv_pool, pool_rows, ROW, ROW * 2, PG, 1) &&
                               tmap_bf16_colblocks(&tm_v, a.kv_pool, pool_rows, ROW, ROW * 2, PG, 2);
    if (!maps || !tmap_bf16_colblocks(&tm_q, a.q_abs, q_rows, ROW, ROW * 2, HALF, NCB)) return cudaErrorInvalidValue;
    if (!f8) tm_c = tm_v;
    cudaLaunchAttribute pdl;
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    // Turned where few tiles are each spread over several pairs, a sequence has two tiles or more to share what L2 holds
    // (their mean: the host knows no more), and it may be long.  Measured, turned against as they come (us, 74 pairs):
    //   bf16, 128 heads   8 x 32768, 2 tiles 156-180 / 176-189   4 x 65536, 4 tiles 270-282 / 318-330   4 x 131072 556 / 650
    //                     4 x 16384, 4 tiles 119-137 / 116-126   8 x 32768, 1 tile   98 / 92
    //   FP8               4 x 65536, 4 tiles 303-311 / 316-319   4 x 131072 602-608 / 641-648
    //                     4 x 32768, 4 tiles 169 / 165-167       8 x 32768, 2 tiles 171 / 169-171       8 x 32768, 1 tile 103 / 100
    // Many tiles have nothing to share, and the turns' instructions cost them 3% (24 ragged sequences).  max_seq_len is the
    // caller's bound: short sequences under a long one are turned for nothing (4 x 2000 under 131072: bf16 46 / 49, FP8 45 / 44).
    const bool turn = 2 * tree_tiles(a.B, (int64_t)q_rows) <= pairs && q_rows >= (uint64_t)a.B * 2 * TILE &&
                      a.max_seq_len >= (f8 ? 65536 : 32768);
    auto kern = f8 ? turn ? tree_tc_kernel<true, true> : tree_tc_kernel<true, false>
                   : turn ? tree_tc_kernel<false, true> : tree_tc_kernel<false, false>;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm_q, tm_k, tm_v, tm_c, a, pl);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)tree_tiles(a.B, (int64_t)q_rows), TILE / JOIN_ROWS);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, tree_tc_join_kernel, a, pl);
}

}  // namespace mla
