// Routing kernel: cosine of each query head with its group's position-0 key,
// minimum over the group's heads, threshold, and ordered compaction of the
// active units into a work list.
//
// Method: SinkRouter README (github.com/streamer-AP/SinkRouter), decode-time
// procedure list -- the RoPE query is compared with the cached position-0 key
// and every GQA KV group is routed before the long cache scan; README routing
// controls -- the threshold is a cosine threshold. The min over heads and ">="
// are this library's reading of what the pages leave open.
//
// Layout: one CTA of 256 threads. One warp per GQA group (M >= 4; a warp takes
// 4 / M groups when M < 4): each lane loads its blocks of the query rows and of
// the key row straight from global memory, and shuffle reductions give each
// pair's cosine and the group's minimum (sr_route_math.cuh). A warp with more
// groups to route issues the loads of its next group before reducing the
// current one. Launches of more than kOneCtaRows<M> query rows give every warp one
// chunk of units on as many CTAs as that takes, and compact in a second launch.
// The compaction writes active units in ascending order with warp
// ballots and a block prefix, so no CTA of the decode kernel is ever bound to a
// sink unit. No asynchronous copy is used, so nothing is in flight when the
// kernel ends.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sinkrouter.h"
#include "sr_internal.h"
#include "sr_ptx.cuh"
#include "sr_route_math.cuh"
#include "sr_timeline.cuh"

SR_TL_DEFINE(tl_route)
#ifdef SR_TIMELINE
// set by the host to the decode kernel's last-exit word (sr_timeline_last_exit_addr)
static __device__ unsigned long long *tl_exit_ptr;
static __device__ unsigned int tl_route_launch; // ring of per-launch stamps in rows 1 .. 64
extern "C" int sr_timeline_set_exit_ptr(void *p) { return (int)cudaMemcpyToSymbol(tl_exit_ptr, &p, sizeof(p)); }
#endif

namespace sr {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;

// M = query heads per KV head (compile time). The dynamic shared memory holds
// one sink flag per unit.
template <int M>
__global__ void __launch_bounds__(kRouteThreads, 1)
route_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *k0, float tau, uint8_t *mask, int32_t *active, int B, int Hkv)
{
    extern __shared__ uint8_t sink_flag[]; // [B*Hkv]
    __shared__ int32_t warp_cnt[kRouteWarps];
    __shared__ int32_t warp_off[kRouteWarps + 1];

    const int U = B * Hkv;
    if (threadIdx.x == 0)
        SR_STAMP(tl_route, 0);
    // Inputs may come from the previous kernel in the stream, and the previous
    // decode step may still read route_mask / active_list: wait for it, then
    // let the decode kernel that follows launch and run its prologue.
    grid_dependency_wait();
    grid_launch_dependents();
    if (threadIdx.x == 0)
        SR_STAMP(tl_route, 1);
#ifdef SR_TIMELINE
    if (threadIdx.x == 0) {
        const unsigned long long pe = tl_exit_ptr ? *(volatile unsigned long long *)tl_exit_ptr : 0ull;
        tl_route[0][5] = pe;
        const unsigned int ring = 1 + atomicAdd(&tl_route_launch, 1u) % 64u;
        tl_route[ring][1] = tl_route[0][1];
        tl_route[ring][5] = pe;
        tl_route[ring][0] = tl_route[0][0];
    }
#endif

    route_units_warp<M>(reinterpret_cast<const uint4 *>(q), reinterpret_cast<const uint4 *>(k0), U, tau,
                              (int)threadIdx.x >> 5, kRouteWarps, [&](int u, bool sink) {
                                  sink_flag[u] = sink ? 1 : 0;
                                  mask[u] = sink ? 1 : 0;
                              });
    __syncthreads();
    if (threadIdx.x == 0)
        SR_STAMP(tl_route, 3);
    compact_active<kRouteThreads>(sink_flag, U, active, warp_cnt, warp_off);
    if (threadIdx.x == 0)
        SR_STAMP(tl_route, 4);
}

// The mask alone: each CTA routes kRouteWarps * RouteLanes<M>::UNITS units, one
// group (or 4 / M) a warp, with the same arithmetic.
template <int M>
__global__ void __launch_bounds__(kRouteThreads)
wide_route_kernel(const __nv_bfloat16 *q, const __nv_bfloat16 *k0, float tau, uint8_t *mask, int U)
{
    constexpr int kUnits = kRouteWarps * RouteLanes<M>::UNITS;
    grid_dependency_wait();
    grid_launch_dependents();
    const int u0 = blockIdx.x * kUnits;
    route_units_warp<M>(reinterpret_cast<const uint4 *>(q) + (size_t)u0 * M * 16,
                              reinterpret_cast<const uint4 *>(k0) + (size_t)u0 * 16, min(kUnits, U - u0), tau,
                              (int)threadIdx.x >> 5, kRouteWarps, [&](int u, bool sink) { mask[u0 + u] = sink ? 1 : 0; });
}

// Ordered compaction of a mask (and the lengths' advance of the append step) by
// one CTA: a thread's units are consecutive, so its list entries are too.
constexpr int kCompactThreads = 1024;
constexpr int kCompactMost = SR_MAX_UNITS / kCompactThreads;

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(CompactArgs a)
{
    __shared__ int warp_sum[kCompactThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int per = (a.units + kCompactThreads - 1) / kCompactThreads, u0 = t * per;
    uint32_t act = 0;
#pragma unroll
    for (int i = 0; i < kCompactMost; ++i)
        if (i < per && u0 + i < a.units && __ldcg(a.mask + u0 + i) == 0)
            act |= 1u << i;
    if (a.seq_lens)
        for (int b = t; b < a.batch; b += kCompactThreads) {
            const int slot = a.seq_lens[b];
            const bool ok = slot >= 0 && slot < a.max_seq_len && (long long)slot + a.pos_offset < a.max_pos;
            a.seq_lens_out[b] = slot + (ok ? 1 : 0);
        }
    int incl = __popc(act);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += y;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    const int mine = warp_sum[lane];
    int before = lane < warp ? mine : 0, all = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    int at = 1 + before + incl - __popc(act);
#pragma unroll
    for (int i = 0; i < kCompactMost; ++i)
        if (act & (1u << i))
            a.active[at++] = u0 + i;
    if (t == 0)
        a.active[0] = all;
}

// Query rows up to which one CTA routes and compacts. Measured back to back, one
// CTA against two launches: 1.3 us against 3.5 at 32 rows, 3.5 / 3.5 at 192 (M = 4), 3.4 /
// 3.7 at 192 (M = 1), 4.0 / 3.7 at 256 (M = 1); M = 8: 3.3 / 3.9 at 256, 4.4 / 3.8 at 384,
// 58.8 / 4.1 at 8192.
template <int M> constexpr int kOneCtaRows = M == 8 ? 256 : 192;

template <int M>
cudaError_t launch_route_m(const RouteArgs &a, cudaStream_t stream)
{
    const int U = a.batch * a.n_kv_heads;
    const bool wide = U * M > kOneCtaRows<M>;
    constexpr int kUnits = kRouteWarps * RouteLanes<M>::UNITS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(wide ? (unsigned)((U + kUnits - 1) / kUnits) : 1u);
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = wide ? 0 : (size_t)U;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (wide) {
        const cudaError_t e = cudaLaunchKernelEx(&cfg, wide_route_kernel<M>, static_cast<const __nv_bfloat16 *>(a.q),
                                                 static_cast<const __nv_bfloat16 *>(a.k0), a.tau, a.mask, U);
        if (e != cudaSuccess)
            return e;
        CompactArgs c{};
        c.mask = a.mask;
        c.active = a.active;
        c.units = U;
        return launch_compact(c, stream);
    }
    return cudaLaunchKernelEx(&cfg, route_kernel<M>, static_cast<const __nv_bfloat16 *>(a.q),
                              static_cast<const __nv_bfloat16 *>(a.k0), a.tau, a.mask, a.active, a.batch,
                              a.n_kv_heads);
}

} // namespace

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kCompactThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, compact_kernel, a);
}

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream)
{
    cudaError_t e;
    switch (a.n_q_heads / a.n_kv_heads) {
    case 1:
        e = launch_route_m<1>(a, stream);
        break;
    case 2:
        e = launch_route_m<2>(a, stream);
        break;
    case 4:
        e = launch_route_m<4>(a, stream);
        break;
    case 8:
        e = launch_route_m<8>(a, stream);
        break;
    default:
        return cudaErrorInvalidValue;
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace sr
