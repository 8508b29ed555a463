// Attention of one decode token of every sequence of a batch over a prefix that
// all of them share, joined with each sequence's own suffix.
//
// Method: the split-K reduction of the SinkRouter README's decode-time procedure
// list, carried across two caches: softmax attention over a union of position
// ranges is sum_r exp(lse_r - lse) o_r with lse = log sum_r exp(lse_r). Over the
// prefix the query heads of every active sequence of a KV head are the rows of
// one matrix Q_g [rows x 128], so S = Q_g K_g^T and O = P V_g are matrix products,
// and every prefix tile is read once for up to 256 rows.
//
// Three launches:
//  * plan: one CTA lists the active sequences of each KV head and cuts each head's
//    rows into items of up to 256.
//  * scan: one persistent CTA per SM takes a contiguous share of the (item, tile
//    of positions) sequence, in which a tile weighs 2 for an item of more than 128
//    rows and 1 for a smaller one, and leaves one partial (m, l, O) a row for every
//    item its share touches.
//  * join: the partials of every query head are combined, and the suffix's.
//
// scan, per CTA: two streams, each with a softmax warpgroup (a thread a row), its
// logits S in TMEM (128 x 128 fp32 columns in all) and its output O (128 x 128); a copy
// warp; and the warps that issue the MMAs. With more than 128 rows the streams are
// the item's two halves over the same tiles; with fewer they are the same rows over
// alternate tiles, and leave a partial each. P goes to the second product in bf16,
// written over S. A warpgroup rescales O only when a row's maximum has grown by more
// than 2^8 since the reference it uses (the weights stay below 2^8 of their row's sum,
// far inside bf16 and fp32), once the previous tile's product is complete.
//
// It has two forms. The wide form works in 128-position tiles (an S product of 128
// columns reads Q from shared memory half as often: 75 cycles a 128x128x16 step
// against 57 a 128x64x16), and one MMA warp issues P0 V and S0 of the next tile, then
// P1 V and S1 of the next tile, which keeps the streams half a turn apart: one has the
// tensor cores while the other has the exponentials. Many rows are bound by those two,
// few rows by the prefix's bytes. A short prefix with at most 128 rows a KV head gives
// a CTA only a few tiles, whose latency counts: the narrow form works in 64-position
// tiles, with two S buffers a stream and an MMA warp each, so that a copied tile is
// used as soon as it has landed and the shares are cut half as coarse.
//
// Every wait is bounded in time; a timeout sets a device error bit, and the CTA
// leaves once its own copies and MMAs have landed.
#include <climits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "sinkrouter.h"
#include "sr_internal.h"
#include "sr_ptx.cuh"
#include "sr_tc.cuh"

namespace sr {
namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull; // 2 s: far above any legitimate wait
constexpr float kScaleLog2 = 0.12751743082459868f; // log2(e) / sqrt(128)
constexpr float kLn2 = 0.6931471805599453f;
constexpr unsigned kFull = 0xffffffffu;

constexpr int kRows = 128;           // rows a stream
constexpr int kItemRows = 2 * kRows; // rows an item
constexpr int kGridCap = 256;        // persistent CTAs never exceed this (sizes the workspace)
constexpr int kQHalfBytes = kRows * 128, kQBytes = 2 * kQHalfBytes;

constexpr int kThreads = 384;        // two softmax warpgroups, one for copies and MMAs:
                                     // 168 registers a thread, of which the last gives some up
constexpr int kSoftmaxWarps = 8;
constexpr int kCopyWarp = 8, kMmaWarp = 9;

// The scan's two forms, by the positions of a tile.
template <int TILE> struct Form {
    static constexpr int kStages = TILE == 64 ? 10 : 4;
    static constexpr int kHalfBytes = TILE * 128;      // [TILE positions x 64 bf16], 128B swizzle
    static constexpr int kTileBytes = 2 * kHalfBytes;  // [TILE x 128]
    static constexpr int kOffQ = 0, kOffRing = 2 * kQBytes, kOffBar = kOffRing + kStages * kTileBytes;
    static constexpr int kSmem = kOffBar + 512 + 1024; // and room to align the base to 1024 B
    static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};
constexpr float kGrowth = 8.f; // log2 growth of a row's maximum that O is rescaled for

// Workspace: [error word | total weight | left alone | first item of each KV head | active
// sequences of each head | rank of each unit | items | item at each weight | (m, l) | O].
// What is left alone is where a decode workspace keeps its units' arrival counters,
// which have to stay 0 between launches: one buffer serves both kinds of call in turn.
struct Layout {
    size_t first, list, rank, items, item_of, ml, o, total;
    int row_cap; // rows of a stream's partial
    long long max_items, slots;
};

Layout layout(int B, int Hq, int Hkv)
{
    Layout w;
    const long long rows = (long long)B * (Hq / Hkv);
    const size_t U = (size_t)B * Hkv;
    w.row_cap = rows < kRows ? (int)((rows + 7) / 8 * 8) : kRows;
    w.max_items = Hkv * ((rows + kItemRows - 1) / kItemRows);
    w.slots = kGridCap + w.max_items;
    size_t at = WorkspaceLayout{}.cnt_off + sizeof(int32_t) * SR_MAX_UNITS;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = align_up(at + bytes, 256);
        return here;
    };
    w.first = take(4 * (size_t)Hkv);
    w.list = take(4 * U);
    w.rank = take(4 * U);
    w.items = take(16 * (size_t)w.max_items);
    w.item_of = take(4 * 2 * (size_t)w.max_items);
    w.ml = take(8 * 2 * (size_t)w.slots * w.row_cap);
    w.o = take(4 * 2 * (size_t)w.slots * w.row_cap * kHeadDim);
    w.total = at;
    return w;
}

struct Params {
    const __nv_bfloat16 *q, *v0;
    const uint8_t *mask;
    int32_t *err;
    int32_t *weight; // word 1 of the workspace: sum of the items' weights
    int32_t *first, *list, *rank;
    int4 *items;      // KV head, first row of the head's rows, rows, weights before it
    int32_t *item_of; // item at each unit of weight
    float2 *ml;  // [slot][stream][row] (m in log2 units, l)
    float *o;    // [slot][stream][16][row][8]
    const float *o_suffix, *lse_suffix;
    __nv_bfloat16 *out;
    float *out_f32, *lse;
    int B, Hq, Hkv, M, prefix_len, row_cap, grid;
    int tile; // positions a tile
};

// An item's weight: its tiles take two row tiles' products or one.
__device__ __forceinline__ int weight_of(int rows) { return rows > kRows ? 2 : 1; }

// Cost of an item for each unit of its weight, in tiles of weight 1: an entry that
// stands for what a CTA spends on beginning an item (its queries, its partial), then its
// tiles. Even, so that with even shares no tile of weight 2 lies across two shares.
// Entries of 2, 4, 6 and 8: 121, 117, 121 and 118 us for 128 sequences of 8 KV heads over
// 32K (M = 8), 68, 70, 74 and 74 for 512 over 8K (M = 4); nothing where an item is spread
// over many CTAs.
constexpr int kEntry = 4;
__device__ __forceinline__ long long item_cost(int nt) { return kEntry + ((nt + 1) & ~1); }

// Cost that one CTA takes of `weight` items of weight 1.
__device__ __forceinline__ long long share_of(int weight, int nt, int grid)
{
    return max(((long long)weight * item_cost(nt) + grid - 1) / grid + 1 & ~1ll, 2ll);
}

// ---- plan -------------------------------------------------------------------------------

constexpr int kPlanThreads = 512, kPlanRounds = 4;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Params p)
{
    __shared__ int2 warp_sum[kPlanThreads / 32];
    __shared__ int2 carry; // items, weight
    __shared__ int count[kPlanThreads];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0)
        carry = make_int2(0, 0);
    for (int g0 = 0; g0 < p.Hkv; g0 += kPlanThreads) {
        // A warp a KV head: ranks of its active sequences, in order. The loads of four
        // rounds go out together.
        for (int g = g0 + warp; g < min(p.Hkv, g0 + kPlanThreads); g += kPlanThreads / 32) {
            int n = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32 * kPlanRounds) {
                bool act[kPlanRounds];
#pragma unroll
                for (int i = 0; i < kPlanRounds; ++i) {
                    const int b = b0 + 32 * i + lane;
                    act[i] = b < p.B && p.mask[(size_t)b * p.Hkv + g] == 0;
                }
#pragma unroll
                for (int i = 0; i < kPlanRounds; ++i) {
                    const int b = b0 + 32 * i + lane;
                    const unsigned ball = __ballot_sync(kFull, act[i]);
                    const int r = n + __popc(ball & ((1u << lane) - 1u));
                    if (act[i])
                        p.list[(size_t)g * p.B + r] = b;
                    if (b < p.B)
                        p.rank[(size_t)b * p.Hkv + g] = act[i] ? r : -1;
                    n += __popc(ball);
                }
            }
            if (lane == 0)
                count[g - g0] = n;
        }
        __syncthreads();
        const int g = g0 + (int)threadIdx.x;
        const int rows = g < p.Hkv ? count[threadIdx.x] * p.M : 0;
        const int n = (rows + kItemRows - 1) / kItemRows, last = rows - (n - 1) * kItemRows;
        const int2 mine = make_int2(n, n ? 2 * (n - 1) + weight_of(last) : 0);
        int2 incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl.x, o), z = __shfl_up_sync(kFull, incl.y, o);
            if (lane >= o) {
                incl.x += y;
                incl.y += z;
            }
        }
        if (lane == 31)
            warp_sum[warp] = incl;
        __syncthreads();
        int2 before = carry, all = make_int2(0, 0);
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const int2 x = warp_sum[w];
            if (w < warp) {
                before.x += x.x;
                before.y += x.y;
            }
            all.x += x.x;
            all.y += x.y;
        }
        const int first = before.x + incl.x - mine.x, weight = before.y + incl.y - mine.y;
        if (g < p.Hkv)
            p.first[g] = first;
        for (int i = 0; i < n; ++i) {
            p.items[first + i] = make_int4(g, i * kItemRows, min(kItemRows, rows - i * kItemRows), weight + 2 * i);
            p.item_of[weight + 2 * i] = first + i;
            if (i + 1 < n || weight_of(last) == 2)
                p.item_of[weight + 2 * i + 1] = first + i;
        }
        __syncthreads();
        if (threadIdx.x == 0)
            carry = make_int2(carry.x + all.x, carry.y + all.y);
        __syncthreads();
    }
    if (threadIdx.x == 0)
        *p.weight = carry.y;
}

// ---- scan -------------------------------------------------------------------------------

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (*abort_flag)
            return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            return false;
        }
    }
}

// The same for a whole warp: true in every lane or in none.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    return __all_sync(kFull, wait_bar(bar, parity, abort_flag));
}

// Largest of three, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A CTA's part of one item: tiles [j0, j1).
struct Segment {
    int item, j0, j1;
    int4 it;
};

// The segments of a share: costs [at, end) of the items' sequence.
struct Walk {
    const Params &p;
    long long at, end, cost;
    int nt;
    __device__ __forceinline__ Walk(const Params &p_) : p(p_)
    {
        nt = (p.prefix_len + p.tile - 1) / p.tile;
        cost = item_cost(nt);
        const int weight = __ldcg(p.weight);
        const long long share = share_of(weight, nt, gridDim.x);
        at = min((long long)blockIdx.x * share, weight * cost);
        end = min(at + share, weight * cost);
    }
    __device__ __forceinline__ bool next(Segment &s)
    {
        while (at < end) {
            s.item = __ldcg(p.item_of + at / cost);
            s.it = __ldcg(p.items + s.item);
            const int w = weight_of(s.it.z);
            const long long begin = s.it.w * cost;
            s.j0 = (int)max((at - begin) / w - kEntry, 0ll);
            s.j1 = (int)min((long long)nt, (end - begin) / w - kEntry);
            at = min(end, begin + w * cost);
            if (s.j0 < s.j1) // else only of the entry, or the padding of an odd number of tiles
                return true;
        }
        return false;
    }
};

// How a segment of n tiles runs on the two streams.
struct Streams {
    bool two; // the streams are two row tiles over the same tiles; else alternate tiles of one
    int n;
    __device__ __forceinline__ int steps(int s) const { return two ? n : (n + 1 - s) / 2; }
    __device__ __forceinline__ int tile(int s, int t) const { return two ? t : 2 * t + s; }
};

// Copies come in the order of their first use: the keys of the first `look` steps (or
// tiles), then each one's values and the next keys. Places of the keys and values of
// number t of n in that sequence of 2 n copies.
__device__ __forceinline__ int key_at(int look, int t) { return t < look ? t : 2 * t + 1 - look; }
__device__ __forceinline__ int value_at(int look, int t, int n)
{
    return min(look, n) + t + min(t, max(n - look, 0));
}

// Narrow form: each stream has a ring of half the stages to itself, so that its MMA
// warp waits for every copy of the ring, in order, and a barrier's parity is never two
// phases off.
constexpr int kRing = Form<64>::kStages / 2;

// Narrow form: the barrier that step t of stream s uses, of the pair that its steps
// use in turn, as a byte offset, and the parity of its phase. done: steps of earlier
// segments on each of the pair.
struct Turn {
    uint32_t off, parity;
};
__device__ __forceinline__ Turn turn_of(int s, int t, uint32_t done0, uint32_t done1)
{
    return {(uint32_t)(16 * s + 8 * (t & 1)), (((t & 1) ? done1 : done0) + (t >> 1)) & 1};
}

struct Shared {
    uint64_t full[10], empty[10];
    uint64_t s_full[2][2], p_full[2][2], o_full[2][2]; // stream; step parity (narrow; wide: the first)
    uint64_t q_full, seg_done, drain[2];
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(Shared) <= 512, "barrier block");

// Barriers, TMEM and the dependency on the plan; returns the TMEM base.
template <int TILE>
__device__ __forceinline__ uint32_t scan_prologue(Shared *sh, const CUtensorMap *tmK, const CUtensorMap *tmV, int warp,
                                                  int lane)
{
    if (threadIdx.x == 0) {
        for (int s = 0; s < Form<TILE>::kStages; ++s) {
            mbar_init(smem_u32(&sh->full[s]), 1);
            mbar_init(smem_u32(&sh->empty[s]), 1);
        }
        mbar_init(smem_u32(&sh->q_full), kSoftmaxWarps);
        mbar_init(smem_u32(&sh->seg_done), kSoftmaxWarps + (TILE == 64 ? 2 : 0)); // narrow: and its MMA warps
        for (int s = 0; s < 2; ++s) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&sh->s_full[s][i]), 1);
                mbar_init(smem_u32(&sh->p_full[s][i]), kSoftmaxWarps / 2);
                mbar_init(smem_u32(&sh->o_full[s][i]), 1);
            }
            mbar_init(smem_u32(&sh->drain[s]), 1);
        }
        sh->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kCopyWarp && lane == 0) {
        prefetch_tensormap(tmK);
        prefetch_tensormap(tmV);
    }
    if (warp == kMmaWarp)
        tmem_alloc(smem_u32(&sh->tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    grid_dependency_wait();
    grid_launch_dependents();
    return tmem;
}

// All warps: a timeout is reported, TMEM given back.
__device__ __forceinline__ void scan_epilogue(const Params &p, bool ok, uint32_t tmem, int warp, int lane)
{
    if (!ok && lane == 0)
        atomicOr(p.err, SR_DEVERR_TIMEOUT);
    __syncthreads();
    __syncwarp();
    if (warp == kMmaWarp)
        tmem_dealloc(tmem, 512);
}

// A warp's MMAs in flight finish before it leaves on a timeout.
__device__ __forceinline__ void drain_mmas(uint32_t bar)
{
    volatile int never = 0;
    if (elect_one())
        mma_commit(bar);
    __syncwarp();
    (void)wait_bar(bar, 0, &never);
}

// One arrival a warp, behind every lane's work (a lane's own arrival each would be
// served one after another).
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane)
{
    tc_fence_before();
    __syncwarp();
    if (lane == 0)
        mbar_arrive(bar);
}

// The two 64-column boxes of TILE positions into a stage.
template <int TILE>
__device__ __forceinline__ void copy_tile(uint8_t *smem, const CUtensorMap *map, uint32_t stage, uint32_t full_bar, int j, int g)
{
    using F = Form<TILE>;
    const uint32_t dst = smem_u32(smem + F::kOffRing + stage * F::kTileBytes);
    if (elect_one()) {
        mbar_arrive_expect_tx(full_bar, F::kTileBytes);
        tma_load_3d_plain(dst, map, full_bar, 0, j * TILE, g);
        tma_load_3d_plain(dst + F::kHalfBytes, map, full_bar, 64, j * TILE, g);
    }
    __syncwarp();
}

// S[128 x TILE] = Q K^T, the elected lane.
template <int TILE> __device__ __forceinline__ void issue_logits(uint32_t d, uint32_t sq, uint32_t sk)
{
    const uint64_t a = smem_desc_sw128(sq, 16, 1024), b = smem_desc_sw128(sk, 16, 1024);
#pragma unroll
    for (int k = 0; k < 8; ++k) // 16 of the 128 dimensions each
        mma_ss(d, a + (k >> 2) * (kQHalfBytes >> 4) + (k & 3) * 2, b + (k >> 2) * (Form<TILE>::kHalfBytes >> 4) + (k & 3) * 2,
               bf16_idesc(kRows, TILE, false), k > 0);
}

// O[128 x 128] (+)= P V over a tile, the elected lane.
template <int TILE> __device__ __forceinline__ void issue_output(uint32_t d, uint32_t tp, uint32_t sv, bool accumulate)
{
    const uint64_t b = smem_desc_sw128(sv, Form<TILE>::kHalfBytes, 1024);
#pragma unroll
    for (int k = 0; k < TILE / 16; ++k) // 16 positions each
        mma_ts(d, tp + k * 8, b + k * (2048 >> 4), bf16_idesc(kRows, kHeadDim, true), accumulate || k > 0);
}

// The row of a segment's item in a softmax thread's lane (past the item: none). Of two
// streams over the same rows, at most 64, the second's start at lane 64, so that the
// streams' rows fall to different schedulers.
__device__ __forceinline__ int row_of(bool two, int rows, int s, int row)
{
    const int shift = !two && rows <= kRows / 2 ? s * (kRows / 2) : 0;
    return two ? s * kRows + row : (row + kRows - shift) % kRows;
}

// Stages the query rows of a warp's 32 threads (zeros for none) in stream s's swizzled
// tile, half a warp a row. (A row a thread, each load touching 32 lines: 48.5 us against
// 45.4 for 1024 rows over 32K, 43.0 against 39.7 for 10240 over 2K.)
__device__ __forceinline__ void stage_query(const Params &p, uint8_t *tile, const int4 &it, int qrow, int row, int lane)
{
    uint4 *dst = reinterpret_cast<uint4 *>(tile);
    int from = -1; // b * Hq + h of this thread's row
    if (qrow < it.z) {
        const int r = it.y + qrow, a = r / p.M;
        from = __ldcg(p.list + (size_t)it.x * p.B + a) * p.Hq + it.x * p.M + (r - a * p.M);
    }
    const int c = lane & 15, r0 = (row & ~31) + (lane >> 4);
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int f = __shfl_sync(kFull, from, 2 * (h + i) + (lane >> 4));
            x[i] = f >= 0 ? ld_dep(reinterpret_cast<const uint4 *>(p.q) + (size_t)f * (kHeadDim / 8) + c)
                          : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 2 * (h + i);
            dst[(c >> 3) * (kQHalfBytes / 16) + r * 8 + ((c & 7) ^ (r & 7))] = x[i];
        }
    }
    fence_proxy_async_smem();
}

// Logits behind the prefix count as -inf: columns c >= left of N.
template <int N> __device__ __forceinline__ void mask_columns(uint32_t (&x)[N / 32][32], int left)
{
#pragma unroll
    for (int c = 0; c < N; ++c)
        if (c >= left)
            x[c / 32][c % 32] = 0xff800000u;
}

// Largest of N logits, NaN if one is: N / 16 chains, so that one warp alone on its
// scheduler does not wait for each comparison.
template <int N> __device__ __forceinline__ float largest(const uint32_t (&x)[N / 32][32])
{
    constexpr int kChains = N / 16;
    float mx[kChains];
#pragma unroll
    for (int c = 0; c < kChains; ++c)
        mx[c] = max_nan(__uint_as_float(x[c / 2][c % 2 * 16]), __uint_as_float(x[c / 2][c % 2 * 16 + 1]),
                        __uint_as_float(x[c / 2][c % 2 * 16 + 2]));
#pragma unroll
    for (int i = 3; i < 15; i += 2)
#pragma unroll
        for (int c = 0; c < kChains; ++c)
            mx[c] = max_nan(mx[c], __uint_as_float(x[c / 2][c % 2 * 16 + i]), __uint_as_float(x[c / 2][c % 2 * 16 + i + 1]));
#pragma unroll
    for (int c = 0; c < kChains; c += 2)
        mx[c] = max_nan(mx[c], __uint_as_float(x[c / 2][15]), __uint_as_float(x[c / 2][31]));
    float top = mx[0];
#pragma unroll
    for (int c = 1; c + 1 < kChains; c += 2)
        top = max_nan(top, mx[c], mx[c + 1]);
    return max_nan(top, mx[kChains - 1], mx[kChains - 1]);
}

// A row's reference m takes its new largest logit: l and O follow it.
__device__ __forceinline__ void raise_reference(float top, float &m, float &l, uint32_t tO)
{
    const float mn = max_nan(m, top, top);
    const float f = mn == m ? 1.f : exp2_approx((m - mn) * kScaleLog2);
    m = mn;
    l *= f;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld16(o, tO + 16 * c);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st16(tO + 16 * c, o);
    }
}

// Weights 2^(s * scale - sub) of 64 logits as bf16 pairs, and their fp32 sum.
__device__ __forceinline__ float weights64(const uint32_t (&x0)[32], const uint32_t (&x1)[32], float sub, uint32_t (&w)[32])
{
    const uint64_t scale2 = pack2(kScaleLog2, kScaleLog2), nsub2 = pack2(-sub, -sub);
    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t(&src)[32] = i < 16 ? x0 : x1;
        const uint64_t y =
            fma2(pack2(__uint_as_float(src[(2 * i) & 31]), __uint_as_float(src[(2 * i + 1) & 31])), scale2, nsub2);
        float a, b;
        unpack2(y, a, b);
        a = exp2_approx(a);
        b = exp2_approx(b);
        sum[i & 1] = add2(sum[i & 1], pack2(a, b));
        w[i] = pack_bf16x2(a, b);
    }
    float s0, s1;
    unpack2(add2(sum[0], sum[1]), s0, s1);
    return s0 + s1;
}

// What the weights' exponents are taken against. A row without a finite logit yet
// keeps weights of 0; an infinite maximum makes them NaN.
__device__ __forceinline__ float subtrahend(float m) { return m == -INFINITY ? 0.f : fmaf(m, kScaleLog2, m - m); }

// 32 bytes in one store: whole sectors. (Two of 16 bytes: 45.4 us against 42.1 for 1024
// rows over 32K.)
__device__ __forceinline__ void st_global_v8(float *at, const uint32_t *x)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// The segment's O of a row: eight elements a row and block of 16.
__device__ __forceinline__ void store_partial(const Params &p, size_t part, uint32_t tO, int prow, bool mine)
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(o, tO + 32 * c);
        tmem_wait_ld();
        if (mine) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                st_global_v8(p.o + part * kHeadDim + ((size_t)(4 * c + i) * p.row_cap + prow) * 8, o + 8 * i);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
scan_narrow_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p)
{
    using F = Form<64>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared *sh = reinterpret_cast<Shared *>(smem + F::kOffBar);
    volatile int *abort_flag = &sh->abort_flag;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const uint32_t full0 = smem_u32(sh->full), empty0 = smem_u32(sh->empty), q_full = smem_u32(&sh->q_full);
    const uint32_t s_full = smem_u32(sh->s_full), p_full = smem_u32(sh->p_full), o_full = smem_u32(sh->o_full);
    const uint32_t seg_done = smem_u32(&sh->seg_done);
    const uint32_t tmem = scan_prologue<64>(sh, &tmK, &tmV, warp, lane);

    Walk walk(p);
    Segment seg{};
    bool ok = true;

    // The copy and MMA warps run converged and elect the issuing lane at each issue:
    // the instructions take their descriptors from uniform registers, which code under
    // a divergent branch has to fill one by one.
    if (warp >= kSoftmaxWarps) {
        regs_dec<120>();
        if (warp == kCopyWarp) {
            // ------------------------------------------------------------ copies
            uint32_t used0 = 0, used1 = 0; // copies issued to each ring
            auto copy = [&](const CUtensorMap *map, int j) -> bool { // tile j of the segment
                const int ring = j & 1;
                const uint32_t i = ring ? used1 : used0, st = ring * kRing + i % kRing;
                if (!wait_warp(empty0 + 8 * st, ((i / kRing) & 1) ^ 1, abort_flag))
                    return false;
                copy_tile<64>(smem, map, st, full0 + 8 * st, seg.j0 + j, seg.it.x);
                ++(ring ? used1 : used0);
                return true;
            };
            while (ok && walk.next(seg)) {
                const int n = seg.j1 - seg.j0; // each stream looks two steps ahead: four tiles
                for (int j = 0; ok && j < min(4, n); ++j)
                    ok = copy(&tmK, j);
                for (int j = 0; ok && j < n; ++j)
                    ok = copy(&tmV, j) && (j + 4 >= n || copy(&tmK, j + 4));
            }
            // Copies in flight land before the CTA can leave.
            volatile int never = 0;
            if (!ok)
                for (int ring = 0; ring < 2; ++ring) {
                    const uint32_t n = ring ? used1 : used0;
                    for (uint32_t i = n > kRing ? n - kRing : 0; i < n; ++i)
                        (void)wait_bar(full0 + 8 * (ring * kRing + i % kRing), (i / kRing) & 1, &never);
                }
        } else if (warp <= kMmaWarp + 1) {
            // ---------------------------------------------- MMAs, a warp a stream
            const int s = warp - kMmaWarp;
            const uint32_t tO = tmem + 256 + s * 128, sq = smem_u32(smem + F::kOffQ + s * kQBytes);
            const uint32_t ring = smem_u32(smem + F::kOffRing + s * kRing * F::kTileBytes);
            const uint32_t full = full0 + 8 * s * kRing, empty = empty0 + 8 * s * kRing;
            uint32_t used = 0, nseg = 0;   // copies of earlier segments in the ring; segments
            uint32_t done0 = 0, done1 = 0; // steps of earlier segments, by their parity
            while (ok && walk.next(seg)) {
                const int steps = Streams{false, seg.j1 - seg.j0}.steps(s);
                if (!(ok = wait_warp(q_full, nseg & 1, abort_flag)))
                    break;
                tc_fence_after();
                // S of step t into its buffer
                auto logits = [&](int t) -> bool {
                    const uint32_t i = used + key_at(2, t), stage = i % kRing;
                    if (!wait_warp(full + 8 * stage, (i / kRing) & 1, abort_flag))
                        return false;
                    if (elect_one()) {
                        issue_logits<64>(tmem + s * 128 + (t & 1) * 64, sq, ring + stage * F::kTileBytes);
                        mma_commit(s_full + turn_of(s, t, done0, done1).off);
                        mma_commit(empty + 8 * stage);
                    }
                    __syncwarp();
                    return true;
                };
                ok = (steps < 1 || logits(0)) && (steps < 2 || logits(1));
                for (int t = 0; ok && t < steps; ++t) {
                    const uint32_t i = used + value_at(2, t, steps), stage = i % kRing;
                    const Turn turn = turn_of(s, t, done0, done1);
                    if (!(ok = wait_warp(full + 8 * stage, (i / kRing) & 1, abort_flag) &&
                               wait_warp(p_full + turn.off, turn.parity, abort_flag)))
                        break;
                    tc_fence_after();
                    if (elect_one()) {
                        issue_output<64>(tO, tmem + s * 128 + (t & 1) * 64, ring + stage * F::kTileBytes, t > 0);
                        mma_commit(o_full + turn.off);
                        mma_commit(empty + 8 * stage);
                    }
                    __syncwarp();
                    if (t + 2 < steps)
                        ok = logits(t + 2);
                }
                if (!ok)
                    break;
                used += 2 * (uint32_t)steps;
                done0 += (steps + 1) / 2;
                done1 += steps / 2;
                ++nseg;
                // A segment of one tile gives the second stream's warp no step, and nobody
                // else waits for it: without its arrival q_full could complete twice
                // before the warp has seen it once.
                if (lane == 0)
                    mbar_arrive(seg_done);
                __syncwarp();
            }
            if (!ok)
                drain_mmas(smem_u32(&sh->drain[s]));
        }
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<192>();
        const int s = warp >> 2, row = tid & (kRows - 1);  // stream, row of its tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21; // this warp's TMEM lanes
        const uint32_t tO = tmem + 256 + s * 128 + lanes;
        uint32_t done0 = 0, done1 = 0, nseg = 0; // steps of earlier segments, by their parity; segments
        while (walk.next(seg)) {
            const Streams st{false, seg.j1 - seg.j0};
            const int qrow = row_of(false, seg.it.z, s, row);
            const bool mine = qrow < seg.it.z;
            const bool busy = __any_sync(kFull, mine); // a warp without a row only keeps the barriers' count
            // Every earlier MMA that read Q is complete (both groups have met below).
            stage_query(p, smem + F::kOffQ + s * kQBytes, seg.it, qrow, row, lane);
            arrive_warp(q_full, lane);

            float m = -INFINITY, l = 0.f; // m in the logits' units
            const int steps = st.steps(s);
            for (int t = 0; t < steps; ++t) {
                const Turn turn = turn_of(s, t, done0, done1);
                const uint32_t tS = tmem + s * 128 + (t & 1) * 64 + lanes;
                if (!wait_warp(s_full + turn.off, turn.parity, abort_flag)) {
                    ok = false;
                    break;
                }
                if (busy) {
                    tc_fence_after();
                    uint32_t x[2][32];
                    tmem_ld32(x[0], tS);
                    tmem_ld32(x[1], tS + 32);
                    tmem_wait_ld();
                    const int left = p.prefix_len - (seg.j0 + st.tile(s, t)) * 64;
                    if (left < 64)
                        mask_columns<64>(x, left);
                    const float top = largest<64>(x);
                    if (t == 0) {
                        m = top;
                    } else if (__any_sync(kFull, !((top - m) * kScaleLog2 <= kGrowth))) { // also for a NaN
                        // This S means that the product before the last is complete:
                        // wait for the last one.
                        const Turn last = turn_of(s, t - 1, done0, done1);
                        if (!wait_warp(o_full + last.off, last.parity, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        raise_reference(top, m, l, tO);
                    }
                    uint32_t w[32];
                    l += weights64(x[0], x[1], subtrahend(m), w);
                    tmem_st32(tS, w);
                    tmem_wait_st();
                }
                arrive_warp(p_full + turn.off, lane);
            }
            if (!ok)
                break;
            const size_t part = (((size_t)blockIdx.x + seg.item) * 2 + s) * p.row_cap;
            const int prow = qrow % kRows;
            if (steps > 0) {
                const Turn last = turn_of(s, steps - 1, done0, done1);
                if (!wait_warp(o_full + last.off, last.parity, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                store_partial(p, part, tO, prow, mine);
            }
            if (mine)
                __stcg(p.ml + part + prow, make_float2(m * kScaleLog2, l));
            done0 += (steps + 1) / 2;
            done1 += steps / 2;
            // Both groups are done with the segment's Q, S and O, and both MMA warps have
            // issued all of it.
            arrive_warp(seg_done, lane);
            if (!wait_warp(seg_done, nseg & 1, abort_flag)) {
                ok = false;
                break;
            }
            ++nseg;
        }
    }
    scan_epilogue(p, ok, tmem, warp, lane);
}

__global__ void __launch_bounds__(kThreads, 1)
scan_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p)
{
    using F = Form<128>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared *sh = reinterpret_cast<Shared *>(smem + F::kOffBar);
    volatile int *abort_flag = &sh->abort_flag;
    const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
    const uint32_t full0 = smem_u32(sh->full), empty0 = smem_u32(sh->empty), q_full = smem_u32(&sh->q_full);
    const uint32_t s_full = smem_u32(sh->s_full), p_full = smem_u32(sh->p_full), o_full = smem_u32(sh->o_full);
    const uint32_t seg_done = smem_u32(&sh->seg_done);
    const uint32_t tmem = scan_prologue<128>(sh, &tmK, &tmV, warp, lane);

    Walk walk(p);
    Segment seg{};
    bool ok = true;

    if (warp >= kSoftmaxWarps) {
        regs_dec<88>();
        if (warp == kCopyWarp) {
            // ------------------------------------------------------------ copies
            uint32_t used = 0; // copies issued
            auto copy = [&](const CUtensorMap *map, int g, int j) -> bool {
                const uint32_t st = used % F::kStages;
                if (!wait_warp(empty0 + 8 * st, ((used / F::kStages) & 1) ^ 1, abort_flag))
                    return false;
                copy_tile<128>(smem, map, st, full0 + 8 * st, j, g);
                ++used;
                return true;
            };
            while (ok && walk.next(seg)) {
                const Streams st{seg.it.z > kRows, seg.j1 - seg.j0};
                const int g = seg.it.x, lead = st.two ? 1 : 2;
                for (int j = 0; ok && j < min(lead, st.n); ++j)
                    ok = copy(&tmK, g, seg.j0 + j);
                for (int j = 0; ok && j < st.n; ++j)
                    ok = copy(&tmV, g, seg.j0 + j) && (j + lead >= st.n || copy(&tmK, g, seg.j0 + j + lead));
            }
            volatile int never = 0;
            if (!ok)
                for (uint32_t i = used > F::kStages ? used - F::kStages : 0; i < used; ++i)
                    (void)wait_bar(full0 + 8 * (i % F::kStages), (i / F::kStages) & 1, &never);
        } else if (warp == kMmaWarp) {
            // ---------------------------------------- MMAs of both streams in turn
            // A wait costs this warp about as much as two MMAs even when it is over, and
            // its issues are what keeps the tensor cores busy: so a turn waits for all
            // that it needs (its P, its values and the next keys; streams over the same
            // tiles wait for these once) and issues both products in one go.
            const uint32_t ring = smem_u32(smem + F::kOffRing), sq = smem_u32(smem + F::kOffQ);
            uint32_t used = 0, seg_parity = 0, np0 = 0, np1 = 0; // copies before; parities
            while (ok && walk.next(seg)) {
                const Streams st{seg.it.z > kRows, seg.j1 - seg.j0};
                const int look = st.two ? 1 : 2, steps0 = st.steps(0), steps1 = st.steps(1);
                if (!(ok = wait_warp(q_full, seg_parity, abort_flag)))
                    break;
                tc_fence_after();
                auto stage_at = [&](int at) { return (used + at) % F::kStages; };
                auto landed = [&](int at) {
                    return wait_warp(full0 + 8 * stage_at(at), ((used + at) / F::kStages) & 1, abort_flag);
                };
                // S of stream s, step t, by the elected lane
                auto logits = [&](int s, int t, bool release) {
                    const uint32_t stage = stage_at(key_at(look, st.tile(s, t)));
                    issue_logits<128>(tmem + s * 128, sq + s * kQBytes, ring + stage * F::kTileBytes);
                    mma_commit(s_full + 16 * s);
                    if (release)
                        mma_commit(empty0 + 8 * stage);
                };
                auto turn = [&](int s, int t, int steps, uint32_t &np) -> bool {
                    const int at = value_at(look, st.tile(s, t), st.n);
                    const bool more = t + 1 < steps, mine = !st.two || s == 1;
                    if (!st.two || s == 0)
                        if (!landed(at) || (more && !landed(key_at(look, st.tile(s, t + 1)))))
                            return false;
                    if (!wait_warp(p_full + 16 * s, np, abort_flag))
                        return false;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t stage = stage_at(at);
                        issue_output<128>(tmem + 256 + s * 128, tmem + s * 128, ring + stage * F::kTileBytes, t > 0);
                        if (mine)
                            mma_commit(empty0 + 8 * stage);
                        if (more)
                            logits(s, t + 1, mine);
                        else
                            mma_commit(o_full + 16 * s);
                    }
                    __syncwarp();
                    np ^= 1;
                    return true;
                };
                ok = landed(key_at(look, 0)) && (st.two || steps1 == 0 || landed(key_at(look, 1)));
                if (ok && elect_one()) {
                    logits(0, 0, !st.two);
                    if (steps1)
                        logits(1, 0, true);
                }
                __syncwarp();
                for (int t = 0; ok && t < steps0; ++t)
                    ok = turn(0, t, steps0, np0) && (t >= steps1 || turn(1, t, steps1, np1));
                used += 2 * (uint32_t)st.n;
                seg_parity ^= 1;
            }
            if (!ok)
                drain_mmas(smem_u32(&sh->drain[0]));
        }
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<208>();
        const int s = warp >> 2, row = tid & (kRows - 1);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t tO = tmem + 256 + s * 128 + lanes, tS = tmem + s * 128 + lanes;
        uint32_t ns = 0, no = 0, nseg = 0; // S tiles, O results and segments consumed
        while (walk.next(seg)) {
            const Streams st{seg.it.z > kRows, seg.j1 - seg.j0};
            const int qrow = row_of(st.two, seg.it.z, s, row);
            const bool mine = qrow < seg.it.z;
            const bool busy = __any_sync(kFull, mine);
            stage_query(p, smem + F::kOffQ + s * kQBytes, seg.it, qrow, row, lane);
            arrive_warp(q_full, lane);

            float m = -INFINITY, l = 0.f;
            const int steps = st.steps(s);
            for (int t = 0; t < steps; ++t) {
                if (!wait_warp(s_full + 16 * s, ns & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                ++ns;
                if (!busy) {
                    arrive_warp(p_full + 16 * s, lane);
                    continue;
                }
                tc_fence_after();
                uint32_t x[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(x[c], tS + 32 * c);
                tmem_wait_ld();
                const int left = p.prefix_len - (seg.j0 + st.tile(s, t)) * 128;
                if (left < 128)
                    mask_columns<128>(x, left);
                const float top = largest<128>(x);
                // This S means that every earlier product of the stream is complete.
                if (t == 0)
                    m = top;
                else if (__any_sync(kFull, !((top - m) * kScaleLog2 <= kGrowth)))
                    raise_reference(top, m, l, tO);
                const float sub = subtrahend(m);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
                    l += weights64(x[2 * h], x[2 * h + 1], sub, w);
                    tmem_st32(tS + 32 * h, w);
                }
                tmem_wait_st();
                arrive_warp(p_full + 16 * s, lane);
            }
            if (!ok)
                break;
            const size_t part = (((size_t)blockIdx.x + seg.item) * 2 + s) * p.row_cap;
            const int prow = qrow % kRows;
            if (steps > 0) {
                if (!wait_warp(o_full + 16 * s, no & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                ++no;
                tc_fence_after();
                store_partial(p, part, tO, prow, mine);
            }
            if (mine)
                __stcg(p.ml + part + prow, make_float2(m * kScaleLog2, l));
            arrive_warp(seg_done, lane);
            if (!wait_warp(seg_done, nseg & 1, abort_flag)) {
                ok = false;
                break;
            }
            ++nseg;
        }
    }
    scan_epilogue(p, ok, tmem, warp, lane);
}

// ---- join -------------------------------------------------------------------------------

constexpr int kJoinWarps = 8;
constexpr int kJoinBatch = 4; // partials in flight a thread, four loads each
constexpr int kJoinRows = 4;  // query heads a warp: eight lanes each

// A row's partials (m, l, acc) += k0, k0 + step, ... below n, `stride` rows of (m, l)
// apart from `ml` on, their columns from `o` on. Eight lanes (the low bits, `sub`) share
// a row: element i of acc is columns 32 i + 4 sub .. + 3. Lane i of them fetches the
// batch's i-th (m, l), and the weights reach the others by shuffles. A part with l = 0
// has no O. n may differ between the rows of a warp.
__device__ __forceinline__ void add_parts(const float2 *ml, const float *o, size_t stride, int row_cap, int k0, int step,
                                          int n, int lane, float &m, float &l, float4 (&acc)[4])
{
    const int sub = lane & 7;
    o += (size_t)(sub >> 1) * row_cap * 8 + (sub & 1) * 4;
    for (; __any_sync(kFull, k0 < n); k0 += step * 8) {
        float2 x = make_float2(-INFINITY, 0.f);
        if (k0 + sub * step < n)
            x = __ldcg(ml + (k0 + sub * step) * stride);
        float mb = x.y == 0.f ? -INFINITY : x.x;
#pragma unroll
        for (int b = 4; b > 0; b >>= 1)
            mb = fmaxf(mb, __shfl_xor_sync(kFull, mb, b));
        const float mn = fmaxf(m, mb);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float w = x.y == 0.f ? 0.f : exp2f(x.x - mn);
        float ls = x.y * w;
#pragma unroll
        for (int b = 4; b > 0; b >>= 1)
            ls += __shfl_xor_sync(kFull, ls, b);
        l = l * keep + ls;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[c].x *= keep, acc[c].y *= keep, acc[c].z *= keep, acc[c].w *= keep;
        const unsigned used = __ballot_sync(kFull, w != 0.f); // NaN too
#pragma unroll 1
        for (int i0 = 0; i0 < 8; i0 += kJoinBatch) {
            // A batch that weighs nothing in any of the rows is skipped; the next one
            // may hold all the weight (its maxima far above this one's).
            if (!(used >> i0 & 0x01010101u * ((1u << kJoinBatch) - 1u)))
                continue;
            float4 y[kJoinBatch][4];
            float wi[kJoinBatch];
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i) {
                wi[i] = __shfl_sync(kFull, w, (lane & 24) + i0 + i);
                const float4 *from = reinterpret_cast<const float4 *>(o + (k0 + (i0 + i) * step) * stride * kHeadDim);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    y[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (wi[i] != 0.f)
                        y[i][c] = __ldcg(from + (size_t)c * 8 * row_cap);
                }
            }
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc[c].x = fmaf(y[i][c].x, wi[i], acc[c].x);
                    acc[c].y = fmaf(y[i][c].y, wi[i], acc[c].y);
                    acc[c].z = fmaf(y[i][c].z, wi[i], acc[c].z);
                    acc[c].w = fmaf(y[i][c].w, wi[i], acc[c].w);
                }
        }
        m = mn;
    }
}

// How the query heads are spread. Four heads a warp where there are enough of them:
// the partials keep eight columns of consecutive rows side by side, so that the heads
// of a group make whole lines of them.
enum class Join {
    kWarpFour, // a warp four heads, all partials
    kCtaFour,  // a CTA four heads, its warps every eighth partial
    kCtaOne    // a CTA one head, eight lanes every 32nd partial
};

template <Join J> __global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Params p)
{
    constexpr bool one = J == Join::kCtaOne, split = J != Join::kWarpFour;
    constexpr int kParts = J == Join::kCtaFour ? 4 : 1; // float4 of a thread's that meet in shared memory
    __shared__ float4 sh_acc[kJoinWarps][kParts][32];
    __shared__ float2 sh_ml[kJoinWarps][kJoinRows];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane >> 3;
    const long long rows = (long long)p.B * p.Hq;
    const long long row0 = one ? blockIdx.x : kJoinRows * (split ? blockIdx.x : (long long)blockIdx.x * kJoinWarps + warp);
    const long long row = one ? row0 : row0 + group; // b * Hq + h
    if (row0 >= rows)
        return;
    const int b = (int)(row / p.Hq), h = (int)(row - (long long)b * p.Hq), g = h / p.M;
    const size_t u = (size_t)b * p.Hkv + g;
    const int rank = row < rows ? __ldcg(p.rank + u) : -1;
    const int nt = (p.prefix_len + p.tile - 1) / p.tile;
    float m = -INFINITY, l = 0.f;
    float4 acc[4] = {};
    int n = 0, pr = 0;
    size_t first = 0, stride = 0; // of its partials
    if (rank >= 0 && nt > 0) {
        const int r = rank * p.M + (h - g * p.M);
        const int item = __ldcg(p.first + g) + r / kItemRows, ir = r % kItemRows;
        const int4 it = __ldcg(p.items + item);
        const bool two = it.z > kRows;
        const long long share = share_of(__ldcg(p.weight), nt, p.grid), begin = it.w * item_cost(nt);
        const int w = weight_of(it.z);
        const int c0 = (int)((begin + (long long)kEntry * w) / share);
        const int c1 = (int)((begin + (long long)(kEntry + nt - 1) * w) / share);
        // CTAs c0 .. c1: one partial each, of the stream that has the row, or both streams'
        n = two ? c1 - c0 + 1 : 2 * (c1 - c0 + 1);
        first = ((size_t)(c0 + item) * 2 + (two ? ir / kRows : 0)) * p.row_cap;
        stride = (size_t)(two ? 2 : 1) * p.row_cap;
        pr = ir % kRows;
    }
    add_parts(p.ml + first + pr, p.o + first * kHeadDim + pr * 8, stride, p.row_cap,
              one ? kJoinRows * warp + group : split ? warp : 0, one ? kJoinRows * kJoinWarps : split ? kJoinWarps : 1, n,
              lane, m, l, acc);
    if constexpr (one) { // the warp's four
        float top = m;
#pragma unroll
        for (int d = 8; d < 32; d <<= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
        const float f = l == 0.f ? 0.f : exp2f(m - top);
        m = top;
        l *= f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[c].x *= f, acc[c].y *= f, acc[c].z *= f, acc[c].w *= f;
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) {
            l += __shfl_xor_sync(kFull, l, d);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[c].x += __shfl_xor_sync(kFull, acc[c].x, d);
                acc[c].y += __shfl_xor_sync(kFull, acc[c].y, d);
                acc[c].z += __shfl_xor_sync(kFull, acc[c].z, d);
                acc[c].w += __shfl_xor_sync(kFull, acc[c].w, d);
            }
        }
    }
    if constexpr (split) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if constexpr (one) {
                if (group == c)
                    sh_acc[warp][0][lane] = acc[c];
            } else {
                sh_acc[warp][c % kParts][lane] = acc[c];
            }
        }
        if ((lane & 7) == 0)
            sh_ml[warp][group] = make_float2(m, l);
        __syncthreads();
        if (warp >= kParts) // the others finish, with a float4 of the row a thread
            return;
        m = -INFINITY;
        l = 0.f;
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
            m = fmaxf(m, sh_ml[w][group].x);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float2 ml = sh_ml[w][group];
            const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - m);
            const float4 o = sh_acc[w][warp][lane];
            l = fmaf(ml.y, f, l);
            acc[0].x = fmaf(o.x, f, acc[0].x);
            acc[0].y = fmaf(o.y, f, acc[0].y);
            acc[0].z = fmaf(o.z, f, acc[0].z);
            acc[0].w = fmaf(o.w, f, acc[0].w);
        }
    }
    if (row >= rows)
        return;
    // acc and l are in units of 2^m; join the suffix's normalised part
    float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    float wp = l == 0.f ? 0.f : 1.f / l, ws = 0.f;
    bool suffix = false;
    if (p.o_suffix && rank >= 0) {
        const float ls = ld_dep(p.lse_suffix + row), top = fmaxf(lse, ls);
        if ((suffix = ls != -INFINITY)) {
            const float ep = expf(lse - top), es = expf(ls - top), tot = ep + es;
            wp *= ep / tot;
            ws = es / tot;
            lse = top + logf(tot);
        }
    }
#pragma unroll
    for (int c = 0; c < (split ? 1 : 4); ++c) {
        const int at = one ? lane : 8 * (split ? warp : c) + (lane & 7); // of the row's 32 float4
        float4 x = acc[c];
        if (rank < 0) { // a sink head
            const uint2 v = ld_dep(reinterpret_cast<const uint2 *>(p.v0 + u * kHeadDim) + at);
            x = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                            __uint_as_float(v.y & 0xffff0000u));
        } else {
            float4 os = make_float4(0.f, 0.f, 0.f, 0.f);
            if (suffix)
                os = ld_dep(reinterpret_cast<const float4 *>(p.o_suffix + (size_t)row * kHeadDim) + at);
            x.x = x.x * wp + os.x * ws;
            x.y = x.y * wp + os.y * ws;
            x.z = x.z * wp + os.z * ws;
            x.w = x.w * wp + os.w * ws;
        }
        if (p.out_f32)
            reinterpret_cast<float4 *>(p.out_f32 + (size_t)row * kHeadDim)[at] = x;
        else
            reinterpret_cast<uint2 *>(p.out + (size_t)row * kHeadDim)[at] =
                make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
    if (p.lse && (one ? lane == 0 : (lane & 7) == 0) && (!split || warp == 0))
        p.lse[row] = rank < 0 ? __int_as_float(0x7fc00000) : lse;
}

// ---- host side ------------------------------------------------------------------------

cudaError_t grid_of(int *grid)
{
    static std::mutex mu;
    static int known[64]; // 0: not configured
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (!known[dev]) {
        int sms = 0;
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(scan_narrow_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Form<64>::kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(scan_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Form<128>::kSmem);
        if (e != cudaSuccess)
            return e;
        known[dev] = sms < kGridCap ? sms : kGridCap;
    }
    *grid = known[dev];
    return cudaSuccess;
}

constexpr long long kJoinOne = 384, kJoinFour = 4096;
constexpr int kShortPrefix = 4096;

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                   const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace

size_t prefix_workspace_bytes(int batch, int n_q_heads, int n_kv_heads)
{
    return layout(batch, n_q_heads, n_kv_heads).total;
}

cudaError_t launch_prefix(const PrefixArgs &a, cudaStream_t stream)
{
    Params p;
    cudaError_t e = grid_of(&p.grid);
    if (e != cudaSuccess)
        return e;
    const Layout w = layout(a.batch, a.n_q_heads, a.n_kv_heads);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.v0 = static_cast<const __nv_bfloat16 *>(a.v0);
    p.mask = a.mask;
    p.err = reinterpret_cast<int32_t *>(ws);
    p.weight = p.err + 1;
    p.first = reinterpret_cast<int32_t *>(ws + w.first);
    p.list = reinterpret_cast<int32_t *>(ws + w.list);
    p.rank = reinterpret_cast<int32_t *>(ws + w.rank);
    p.items = reinterpret_cast<int4 *>(ws + w.items);
    p.item_of = reinterpret_cast<int32_t *>(ws + w.item_of);
    p.ml = reinterpret_cast<float2 *>(ws + w.ml);
    p.o = reinterpret_cast<float *>(ws + w.o);
    p.o_suffix = a.o_suffix;
    p.lse_suffix = a.lse_suffix;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.out_f32 = a.out_f32;
    p.lse = a.lse;
    p.B = a.batch;
    p.Hq = a.n_q_heads;
    p.Hkv = a.n_kv_heads;
    p.M = a.n_q_heads / a.n_kv_heads;
    p.prefix_len = a.prefix_len;
    p.row_cap = w.row_cap;
    // At most 128 rows a KV head, narrow form against wide, the whole call in us: 14.0 /
    // 16.1 for 32 KV heads over 577 positions, 23.6 / 25.8 for 32 over 2048, 15.1 / 15.0 for
    // 8 over 4096, 22.9 / 21.3 for 8 over 8192, 58.9 / 52.4 for 8 over 32768 (128 rows).
    p.tile = a.batch * p.M <= kRows && a.prefix_len < kShortPrefix ? 64 : 128;

    e = launch(plan_kernel, 1, kPlanThreads, 0, stream, p);
    if (e == cudaSuccess && a.prefix_len > 0) {
        CUtensorMap tmK, tmV;
        if (!make_cache_map(&tmK, a.k_prefix, a.n_kv_heads, a.max_seq_len, p.tile, false, a.prefix_len) ||
            !make_cache_map(&tmV, a.v_prefix, a.n_kv_heads, a.max_seq_len, p.tile, false, a.prefix_len))
            return cudaErrorInvalidValue;
        if (p.tile == 64)
            e = launch(scan_narrow_kernel, (unsigned)p.grid, kThreads, Form<64>::kSmem, stream, tmK, tmV, p);
        else
            e = launch(scan_wide_kernel, (unsigned)p.grid, kThreads, Form<128>::kSmem, stream, tmK, tmV, p);
    }
    if (e == cudaSuccess) {
        // The fewer the rows, the more partials each has (the grid is spread over fewer
        // items), and the more of the GPU a row needs. The whole call in us with a CTA a
        // row, a CTA four, a warp four: 90.8 / 93.4 / 122 for 256 rows over 128K; 40.5 /
        // 40.0 / 64.5 for 512, 53.5 / 48.3 / 73.5 for 1024, 108 / 86 / 85 for 4096
        // and 192 / 145 / 135 for 8192 over 32K.
        const long long rows = (long long)a.batch * a.n_q_heads, quads = (rows + kJoinRows - 1) / kJoinRows;
        if (rows <= kJoinOne)
            e = launch(join_kernel<Join::kCtaOne>, (unsigned)rows, 32 * kJoinWarps, 0, stream, p);
        else if (rows <= kJoinFour)
            e = launch(join_kernel<Join::kCtaFour>, (unsigned)quads, 32 * kJoinWarps, 0, stream, p);
        else
            e = launch(join_kernel<Join::kWarpFour>, (unsigned)((quads + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0,
                       stream, p);
    }
    return e;
}

} // namespace sr
