// The step just before the cache scan, in one launch: rotary position
// embedding of the query heads and of the new key, the append of the new key /
// value at each sequence's next slot, the position-0 capture that prefill
// leaves for routing, the routing decision and the ordered active list, and the
// length update.
//
// Method: SinkRouter README (github.com/streamer-AP/SinkRouter), decode-time
// procedure list -- routing compares the RoPE'd query with the cached
// position-0 key (recorded when the first token is written) and the new
// token's key and value join the cache before the scan. The rotation is the
// rotate-half form (element i pairs with element i + 64 of a 128-wide head)
// driven by caller-supplied cos / sin tables, so no frequency schedule is
// built in.
//
// Exactness: each rotated element is a*c - b*s (or b*c + a*s) with a, b bf16
// and c, s fp32, so both products are exact in fp64 and one fp64 rounding of
// their sum is the only error before the narrowing. The narrowing to bf16
// rounds to odd into fp32 and then to nearest-even into bf16, which equals a
// single round-to-nearest-even of the fp64 value (Boldo and Melquiond, rounding
// to odd: an intermediate with at least two more bits than the target, at every
// exponent, makes the double rounding innocuous; fp32 has sixteen more than
// bf16). The result is the correctly rounded bf16 of the fp64 rotation.
//
// The same step writes the 8-bit cache (sr_quant.cuh): the new key is the
// correctly rounded bf16 rotation first and is quantised from that, by the
// eight lanes that hold it, so the position-0 key is the bf16 row in either case.
//
// Layout: one CTA of 512 threads for the smallest launches; else a cluster of eight
// with a share of the units each, whose sink flags go to CTA 0's shared memory for
// the compaction; launches of more than kClusterItems items a CTA use as many CTAs
// as give every item a thread, and the routing kernel's compaction launch, which
// then also advances the lengths. Per CTA, in one pass where each thread takes its own item:
// eight threads per new key rotate it (each takes 8 elements and their 8
// partners), write the cache slot, and stage the group's position-0 key (the
// captured one at slot 0, else the stored k0); eight threads per query row
// rotate it into q_out and the staged rows; the staged rows are routed with the routing kernel's own
// routine (one warp per GQA group), so the decision equals sr_route on
// (q_out, k0) bit for bit. Lengths advance after every read of
// them; the compaction is the routing kernel's.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sinkrouter.h"
#include "sr_internal.h"
#include "sr_ptx.cuh"
#include "sr_quant.cuh"
#include "sr_route_math.cuh"

namespace sr {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterCtas = 8;
// How a launch is spread, by its items (eight per query row and per new key; a CTA
// has 512 threads). Measured back to back:
//   one CTA against a cluster of eight: 3.8 us against 4.0 at 320 items (8 units, M = 4);
//   4.6 / 3.3 at 512 (32 units, M = 1), 5.2 / 4.1 at 576 (8 units, M = 8) -- the fp64
//   rotations spread over more SMs;
//   cluster against two launches: 3.7 / 6.5 at 1280 items (32 units, M = 4), 6.0 / 6.6 at
//   5120, 8.3 / 6.6 at 10240, 25.9 / 6.8 at 40960; M = 8: 6.1 / 7.7 at 4608, 8.1 / 7.8 at 9216;
//   M = 1: 5.0 / 6.5 at 4096, 7.3 / 6.6 at 8192.
enum Spread { kOne, kCluster, kWide };
constexpr int kOneItems = 384;
constexpr int kClusterItems = 768; // a CTA

struct PrestepParams {
    const __nv_bfloat16 *q_in, *k_new, *v_new;
    const float *rope_cos, *rope_sin;
    const int32_t *seq_lens;
    int32_t *seq_lens_out;           // may be seq_lens
    uint8_t *k_cache, *v_cache;      // rows of 256 (bf16) or 128 bytes
    float2 *scales;                  // 8-bit caches only
    __nv_bfloat16 *k0, *v0, *q_out;
    uint8_t *mask;
    int32_t *active;
    int32_t *error;
    float tau;
    int B, Hkv, Lmax, max_pos, pos_offset;
};

// Correctly rounded fp64 -> bf16 (nearest, ties to even) through round-to-odd
// into fp32: truncate, and if the truncation was inexact force the last fp32
// bit to 1; the fp32 -> bf16 step then rounds to nearest even.
__device__ __forceinline__ uint32_t bf16_bits_rn(double x)
{
    float f = __double2float_rz(x);
    if ((double)f != x)
        f = __uint_as_float(__float_as_uint(f) | 1u);
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f));
}

__device__ __forceinline__ double bf16_lo(uint32_t w) { return (double)__uint_as_float(w << 16); }
__device__ __forceinline__ double bf16_hi(uint32_t w) { return (double)__uint_as_float(w & 0xffff0000u); }

// Rotate 8 elements x_lo (positions 8j .. 8j+7) against their partners x_hi
// (positions 64+8j ..) with c, s the table entries for those 8 pairs:
//   lo' = lo c - hi s,  hi' = hi c + lo s.
__device__ __forceinline__ void rope8(uint4 x_lo, uint4 x_hi, const float4 (&c)[2], const float4 (&s)[2], uint4 &o_lo,
                                      uint4 &o_hi)
{
    const uint32_t lw[4] = {x_lo.x, x_lo.y, x_lo.z, x_lo.w};
    const uint32_t hw[4] = {x_hi.x, x_hi.y, x_hi.z, x_hi.w};
    const float cf[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
    const float sf[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
    uint32_t ol[4], oh[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t rl[2], rh[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const double a = e ? bf16_hi(lw[k]) : bf16_lo(lw[k]);
            const double b = e ? bf16_hi(hw[k]) : bf16_lo(hw[k]);
            const double cc = (double)cf[2 * k + e], ss = (double)sf[2 * k + e];
            rl[e] = bf16_bits_rn(fma(a, cc, -(b * ss)));
            rh[e] = bf16_bits_rn(fma(b, cc, a * ss));
        }
        ol[k] = rl[0] | (rl[1] << 16);
        oh[k] = rh[0] | (rh[1] << 16);
    }
    o_lo = make_uint4(ol[0], ol[1], ol[2], ol[3]);
    o_hi = make_uint4(oh[0], oh[1], oh[2], oh[3]);
}

// Slot of sequence b, or -1 when it is outside [0, min(Lmax, max_pos -
// pos_offset)). Plain loads: this kernel may write seq_lens at the end.
__device__ __forceinline__ int slot_of(const PrestepParams &p, int b)
{
    const int slot = p.seq_lens[b];
    return (slot >= 0 && slot < p.Lmax && (long long)slot + p.pos_offset < p.max_pos) ? slot : -1;
}

// Writes elements 8j .. 8j+7 (lo) and 64+8j .. 64+8j+7 (hi) of a cache row. For
// an 8-bit cache the eight lanes that hold the row agree on its scale, which is
// returned.
template <int KV> __device__ __forceinline__ float store_row(uint8_t *cache, size_t row, int j, uint4 lo, uint4 hi)
{
    if constexpr (KV == SR_KV_BF16) {
        uint4 *d = reinterpret_cast<uint4 *>(cache + row * (kHeadDim * 2));
        d[j] = lo;
        d[j + 8] = hi;
        return 0.f;
    } else {
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t m = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            m = abs_max_bf16x2(m, w[e]);
        const unsigned lanes = 0xffu << (threadIdx.x & 24);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
            m = __vmaxu2(m, __shfl_xor_sync(lanes, m, o));
        const RowQuant r = row_quant<KV>(max(m & 0xffffu, m >> 16));
        uint2 *d = reinterpret_cast<uint2 *>(cache + row * kHeadDim);
        d[j] = make_uint2(quant4<KV>(w[0], w[1], r), quant4<KV>(w[2], w[3], r));
        d[j + 8] = make_uint2(quant4<KV>(w[4], w[5], r), quant4<KV>(w[6], w[7], r));
        return r.scale;
    }
}

__device__ __forceinline__ void load_table8(const float *tab, int pos, int j, float4 (&v)[2])
{
    const float4 *t = reinterpret_cast<const float4 *>(tab + (size_t)pos * (kHeadDim / 2) + 8 * j);
    v[0] = ld_dep(t);
    v[1] = ld_dep(t + 1);
}

template <int M, int KV, int SPREAD>
__global__ void __launch_bounds__(kThreads, 1) rope_append_route_kernel(PrestepParams p, int cu)
{
    extern __shared__ __align__(128) uint8_t dsm[]; // [cu*(M+1)*256 staged rows][B*Hkv sink flags, unless wide]
    __shared__ int32_t warp_cnt[kWarps];
    __shared__ int32_t warp_off[kWarps + 1];

    const int U = p.B * p.Hkv;
    // This CTA's units
    const int u0 = min((int)blockIdx.x * cu, U);
    const int nu = min(cu, U - u0);
    uint4 *rows = reinterpret_cast<uint4 *>(dsm);
    uint8_t *sink_flag = dsm + (size_t)cu * (M + 1) * 256;
    uint8_t *all_flags = sink_flag; // CTA 0's, which compacts the active list
    if constexpr (SPREAD == kCluster) {
        all_flags = cooperative_groups::this_cluster().map_shared_rank(sink_flag, 0);
        cooperative_groups::this_cluster().barrier_arrive();
    }
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

    // Every input may come from the preceding kernel, and the previous decode
    // step may still read the cache, seq_lens and the routing outputs: wait for
    // it. The decode kernel that follows reads all of its inputs after its own
    // dependency wait, so it may launch now and run its prologue.
    grid_dependency_wait();
    grid_launch_dependents();

    // Query row item `it`: rotate into q_out and the staged rows; a sequence with no
    // valid slot gets a zero query.
    auto query_item = [&](int it) {
        const int r = it >> 3, j = it & 7;
        const int u = u0 + r / M;
        const size_t row = ((size_t)u0 * M + r) * kHeadDim;
        // plain loads: q_out may be q_in (rotated in place)
        const uint4 *qi = reinterpret_cast<const uint4 *>(p.q_in + row);
        const uint4 qlo = qi[j], qhi = qi[j + 8];
        const int pos = slot_of(p, u / p.Hkv);
        uint4 *qs = rows + r * 16;
        uint4 *qd = reinterpret_cast<uint4 *>(p.q_out + row);
        uint4 lo = zero, hi = zero;
        if (pos >= 0) {
            float4 c[2], s[2];
            load_table8(p.rope_cos, pos + p.pos_offset, j, c);
            load_table8(p.rope_sin, pos + p.pos_offset, j, s);
            rope8(qlo, qhi, c, s, lo, hi);
        }
        qs[j] = lo;
        qs[j + 8] = hi;
        qd[j] = lo;
        qd[j + 8] = hi;
    };

    bool bad_slot = false;
    uint4 *krows = rows + (size_t)nu * M * 16;
    // One pass over the items, each thread on its own item (at the 8B shape every
    // item has a thread), so that no thread takes a key and a query row one after
    // the other: items [0, nu*8) are the new keys, the rest the query rows.
    for (int it = threadIdx.x; it < nu * 8 + nu * M * 8; it += kThreads) {
        if (it >= nu * 8) {
            query_item(it - nu * 8);
            continue;
        }
        // New key: rotate, append, capture or stage k0. New value: append.
        const int lu = it >> 3, j = it & 7;
        const int u = u0 + lu;
        // The new key and value do not depend on the slot: load them in the
        // same round trip as the slot itself.
        const uint4 *kn = reinterpret_cast<const uint4 *>(p.k_new + (size_t)u * kHeadDim);
        const uint4 *vn = reinterpret_cast<const uint4 *>(p.v_new + (size_t)u * kHeadDim);
        const uint4 klo = ld_dep(kn + j), khi = ld_dep(kn + j + 8);
        const uint4 vlo = ld_dep(vn + j), vhi = ld_dep(vn + j + 8);
        const int pos = slot_of(p, u / p.Hkv);
        uint4 *ks = krows + lu * 16;
        uint4 *k0g = reinterpret_cast<uint4 *>(p.k0 + (size_t)u * kHeadDim);
        if (pos < 0) {
            bad_slot = true;
            ks[j] = k0g[j];
            ks[j + 8] = k0g[j + 8];
            continue;
        }
        float4 c[2], s[2];
        load_table8(p.rope_cos, pos + p.pos_offset, j, c);
        load_table8(p.rope_sin, pos + p.pos_offset, j, s);
        uint4 lo, hi;
        rope8(klo, khi, c, s, lo, hi);
        const size_t slot = (size_t)u * p.Lmax + pos;
        const float sk = store_row<KV>(p.k_cache, slot, j, lo, hi);
        const float sv = store_row<KV>(p.v_cache, slot, j, vlo, vhi);
        if (KV != SR_KV_BF16 && j == 0)
            p.scales[slot] = make_float2(sk, sv);
        if (pos + p.pos_offset == 0) {
            uint4 *v0g = reinterpret_cast<uint4 *>(p.v0 + (size_t)u * kHeadDim);
            k0g[j] = lo;
            k0g[j + 8] = hi;
            v0g[j] = vlo;
            v0g[j + 8] = vhi;
            ks[j] = lo;
            ks[j + 8] = hi;
        } else {
            ks[j] = k0g[j];
            ks[j + 8] = k0g[j + 8];
        }
    }
    __syncthreads();
    if constexpr (SPREAD == kCluster)
        cooperative_groups::this_cluster().barrier_wait(); // CTA 0 runs: its shared memory may be written
    route_units_warp<M>(rows, krows, nu, p.tau, (int)threadIdx.x >> 5, kWarps, [&](int lu, bool sink) {
        if constexpr (SPREAD != kWide)
            all_flags[u0 + lu] = sink ? 1 : 0;
        p.mask[u0 + lu] = sink ? 1 : 0;
    });
    __syncthreads(); // every read of the lengths is done

    if (p.error && __syncthreads_or(bad_slot) && threadIdx.x == 0)
        atomicOr(p.error, SR_DEVERR_APPEND_SLOT);
    if constexpr (SPREAD != kWide) {
        if constexpr (SPREAD == kCluster) {
            cooperative_groups::this_cluster().sync();
            if (blockIdx.x != 0)
                return;
        }
        // Every other read of seq_lens, and every flag, is behind the barriers above.
        for (int b = threadIdx.x; b < p.B; b += kThreads)
            p.seq_lens_out[b] = p.seq_lens[b] + (slot_of(p, b) >= 0 ? 1 : 0);
        compact_active<kThreads>(sink_flag, U, p.active, warp_cnt, warp_off);
    }
}

template <int M, int KV, int SPREAD>
cudaError_t launch_m(const PrestepArgs &a, cudaStream_t stream)
{
    const int U = a.batch * a.n_kv_heads;
    // Units a CTA. Wide: one thread an item.
    const int cu = SPREAD == kWide ? kThreads / (8 * (M + 1)) : SPREAD == kOne ? U : (U + kClusterCtas - 1) / kClusterCtas;
    const size_t smem = (size_t)cu * (M + 1) * 256 + (SPREAD == kWide ? 0 : (size_t)U);
    PrestepParams p;
    p.q_in = static_cast<const __nv_bfloat16 *>(a.q_in);
    p.k_new = static_cast<const __nv_bfloat16 *>(a.k_new);
    p.v_new = static_cast<const __nv_bfloat16 *>(a.v_new);
    p.rope_cos = a.rope_cos;
    p.rope_sin = a.rope_sin;
    p.seq_lens = a.seq_lens;
    p.seq_lens_out = a.seq_lens_out;
    p.k_cache = static_cast<uint8_t *>(a.k_cache);
    p.v_cache = static_cast<uint8_t *>(a.v_cache);
    p.scales = reinterpret_cast<float2 *>(a.scales);
    p.k0 = static_cast<__nv_bfloat16 *>(a.k0);
    p.v0 = static_cast<__nv_bfloat16 *>(a.v0);
    p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
    p.mask = a.mask;
    p.active = a.active;
    p.error = a.error;
    p.tau = a.tau;
    p.B = a.batch;
    p.Hkv = a.n_kv_heads;
    p.Lmax = a.max_seq_len;
    p.max_pos = a.max_pos;
    p.pos_offset = a.pos_offset;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SPREAD == kWide ? (unsigned)((U + cu - 1) / cu) : SPREAD == kOne ? 1u : (unsigned)kClusterCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kClusterCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPREAD == kCluster ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_append_route_kernel<M, KV, SPREAD>, p, cu);
    if (e != cudaSuccess || SPREAD != kWide)
        return e;
    CompactArgs c{};
    c.mask = a.mask;
    c.active = a.active;
    c.units = U;
    c.seq_lens = a.seq_lens;
    c.seq_lens_out = a.seq_lens_out;
    c.batch = a.batch;
    c.max_seq_len = a.max_seq_len;
    c.max_pos = a.max_pos;
    c.pos_offset = a.pos_offset;
    return launch_compact(c, stream);
}

template <int M, int KV> cudaError_t launch_kv(const PrestepArgs &a, cudaStream_t stream)
{
    const int units = a.batch * a.n_kv_heads;
    if (units * 8 * (M + 1) <= kOneItems)
        return launch_m<M, KV, kOne>(a, stream);
    return (units + kClusterCtas - 1) / kClusterCtas * 8 * (M + 1) <= kClusterItems ? launch_m<M, KV, kCluster>(a, stream)
                                                                                    : launch_m<M, KV, kWide>(a, stream);
}

template <int M> cudaError_t launch_group(const PrestepArgs &a, cudaStream_t stream)
{
    switch (a.kv) {
    case SR_KV_BF16:
        return launch_kv<M, SR_KV_BF16>(a, stream);
    case SR_KV_E4M3:
        return launch_kv<M, SR_KV_E4M3>(a, stream);
    default:
        return launch_kv<M, SR_KV_INT8>(a, stream);
    }
}

} // namespace

cudaError_t launch_rope_append_route(const PrestepArgs &a, cudaStream_t stream)
{
    cudaError_t e;
    switch (a.n_q_heads / a.n_kv_heads) {
    case 1:
        e = launch_group<1>(a, stream);
        break;
    case 2:
        e = launch_group<2>(a, stream);
        break;
    case 4:
        e = launch_group<4>(a, stream);
        break;
    case 8:
        e = launch_group<8>(a, stream);
        break;
    default:
        return cudaErrorInvalidValue;
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace sr
