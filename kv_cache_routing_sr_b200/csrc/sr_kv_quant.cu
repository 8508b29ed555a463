// Bulk writes into the 8-bit KV cache and reads back out of it.
//
// Method: the cache that the SinkRouter README's decode-time procedure list
// scans (position-0 key and value recorded when the first token is written),
// held in 8 bits a value with one scale a row (sr_quant.cuh gives the format).
//
// write: T new tokens a sequence, any of them fewer, as rows of strided bf16
// tensors [B, T, Hkv, 128], go to slots start[b] .. of the cache [B, Hkv, Lmax,
// 128] with their scales [B, Hkv, Lmax, 2] (key, value). read: n[b] positions
// from start[b] on come back as bf16 [B, Hkv, T, 128].
//
// Both move each row once (256 bytes one side, 132 the other) and are bound by
// that. Layout: eight lanes a row, lane j with the values 8j .. 8j + 7 and 64 + 8j ..
// 64 + 8j + 7, so that every load and store of a warp covers whole sectors; a warp
// takes four consecutive tokens of one KV head (four rows that are neighbours in the
// cache, 512 contiguous bytes, whose scale pairs fill one 32-byte sector) and both the
// key and the value of each, and neighbouring warps take neighbouring heads, which are
// neighbours in the projection's layout. One item a warp at a time, and many warps:
// two or four items in flight were slower. Nothing is read twice, so loads and stores
// are streaming ones.
//
// Measured, inputs larger than L2: 129 us for the 128K x 8 rows of a prompt (814 MB,
// 6.3 TB/s) in bursts, 151 (5.4 TB/s) when run for seconds; with 58 registers and four
// blocks per SM in place of 40 and six 144 in bursts. To int8, whose quotients take five
// operations a value, 151 in bursts and 181 for seconds (162 in bursts with four blocks);
// with an operation a value in place of one for two, and scales by three divisions, 173.
// Reading 32K x 8 rows back takes 33.5 us (203 MB, 6.1 TB/s), 34.6 for seconds; with
// cached loads 38.0, and with 16 consecutive values a lane, whose stores cover half
// sectors, 39.7.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sinkrouter.h"
#include "sr_internal.h"
#include "sr_ptx.cuh"
#include "sr_quant.cuh"

namespace sr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerWarp = 4;

struct Item {
    int b, g, t; // sequence, KV head, token of this lane's row
};

// Warp item i: KV heads fastest, then blocks of four tokens, then sequences.
__device__ __forceinline__ Item item_of(long long i, int Hkv, int nblk, int lane)
{
    const long long gb = i / Hkv;
    Item r;
    r.g = (int)(i - gb * Hkv);
    const long long b = gb / nblk;
    r.b = (int)b;
    r.t = (int)(gb - b * nblk) * kRowsPerWarp + (lane >> 3);
    return r;
}

// Rows a sequence really has: n clamped to [0, T], reported when it was not in it.
__device__ __forceinline__ int clamp_count(int n, int T, int32_t *err)
{
    if (n >= 0 && n <= T)
        return n;
    if (err)
        atomicOr(err, SR_DEVERR_ROW_COUNT);
    return n < 0 ? 0 : T;
}

template <int KV> __global__ void __launch_bounds__(kThreads, 6) write_kernel(KvWriteArgs a, long long items, int nblk)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, j = lane & 7;
    const long long nw = (long long)gridDim.x * kWarps;
    for (long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < items; i += nw) {
        const Item it = item_of(i, a.n_kv_heads, nblk, lane);
        const int n = clamp_count(ld_dep(a.n + it.b), a.n_tokens, a.error);
        const long long slot = (long long)ld_dep(a.start + it.b) + it.t;
        bool live = it.t < n;
        if (live && (slot < 0 || slot >= a.max_seq_len)) {
            live = false;
            if (a.error)
                atomicOr(a.error, SR_DEVERR_APPEND_SLOT);
        }
        if (!__any_sync(0xffffffffu, live))
            continue;
        uint4 x[2][2] = {};
        if (live) {
            const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.k_new) +
                                                             it.b * a.ks.batch + it.t * a.ks.token + it.g * a.ks.head);
            const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.v_new) +
                                                             it.b * a.vs.batch + it.t * a.vs.token + it.g * a.vs.head);
            x[0][0] = __ldcs(k + j);
            x[0][1] = __ldcs(k + j + 8);
            x[1][0] = __ldcs(v + j);
            x[1][1] = __ldcs(v + j + 8);
        }
        uint32_t w[2][8], top = 0u; // top: of the key in the low half, of the value in the high one
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint32_t m = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint4 &y = x[s][e >> 2];
                w[s][e] = e % 4 == 0 ? y.x : e % 4 == 1 ? y.y : e % 4 == 2 ? y.z : y.w;
                m = abs_max_bf16x2(m, w[s][e]);
            }
            top |= max(m & 0xffffu, m >> 16) << (16 * s);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const RowQuant rq[2] = {row_quant<KV>(top & 0xffffu), row_quant<KV>(top >> 16)};
        uint2 codes[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                codes[s][h] = make_uint2(quant4<KV>(w[s][4 * h], w[s][4 * h + 1], rq[s]),
                                         quant4<KV>(w[s][4 * h + 2], w[s][4 * h + 3], rq[s]));
        if (!live)
            continue;
        const size_t u = (size_t)it.b * a.n_kv_heads + it.g;
        const size_t row = u * a.max_seq_len + (size_t)slot;
        uint2 *kc = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.k_cache) + row * kHeadDim);
        uint2 *vc = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.v_cache) + row * kHeadDim);
        __stcs(kc + j, codes[0][0]);
        __stcs(kc + j + 8, codes[0][1]);
        __stcs(vc + j, codes[1][0]);
        __stcs(vc + j + 8, codes[1][1]);
        if (j == 0)
            __stcs(reinterpret_cast<float2 *>(a.scales) + row, make_float2(rq[0].scale, rq[1].scale));
        if (slot == 0 && a.k0) {
            uint4 *k0 = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.k0) + u * kHeadDim);
            uint4 *v0 = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.v0) + u * kHeadDim);
            k0[j] = x[0][0];
            k0[j + 8] = x[0][1];
            v0[j] = x[1][0];
            v0[j + 8] = x[1][1];
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float4 &a, const float4 &b)
{
    return make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
}

// c * s is rounded to fp32 and then to bf16. For e4m3 (and a scale this library
// wrote) both are exact; for int8 the product has up to 31 bits and the first
// rounding moves the second one only where the product lies within 2^-25 of
// itself of a bf16 tie.
template <int KV> __global__ void __launch_bounds__(kThreads) read_kernel(KvReadArgs a, long long items, int nblk)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, j = lane & 7;
    const long long nw = (long long)gridDim.x * kWarps;
    for (long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < items; i += nw) {
        const Item it = item_of(i, a.n_kv_heads, nblk, lane);
        const int n = clamp_count(ld_dep(a.n + it.b), a.n_rows, a.error);
        const long long pos = (long long)ld_dep(a.start + it.b) + it.t;
        if (it.t >= n)
            continue;
        if (pos < 0 || pos >= a.max_seq_len) {
            if (a.error)
                atomicOr(a.error, SR_DEVERR_APPEND_SLOT);
            continue;
        }
        const size_t u = (size_t)it.b * a.n_kv_heads + it.g;
        const size_t row = u * a.max_seq_len + (size_t)pos;
        const uint2 *kc = reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.k_cache) + row * kHeadDim);
        const uint2 *vc = reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.v_cache) + row * kHeadDim);
        const uint2 k_lo = __ldcs(kc + j), k_hi = __ldcs(kc + j + 8), v_lo = __ldcs(vc + j), v_hi = __ldcs(vc + j + 8);
        const float2 s = __ldcs(reinterpret_cast<const float2 *>(a.scales) + row);
        const size_t to = (u * a.n_rows + it.t) * kHeadDim;
        uint4 *ko = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.k_out) + to);
        uint4 *vo = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.v_out) + to);
        __stcs(ko + j, pack8(dequant4<KV>(k_lo.x, s.x), dequant4<KV>(k_lo.y, s.x)));
        __stcs(ko + j + 8, pack8(dequant4<KV>(k_hi.x, s.x), dequant4<KV>(k_hi.y, s.x)));
        __stcs(vo + j, pack8(dequant4<KV>(v_lo.x, s.y), dequant4<KV>(v_lo.y, s.y)));
        __stcs(vo + j + 8, pack8(dequant4<KV>(v_hi.x, s.y), dequant4<KV>(v_hi.y, s.y)));
    }
}

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args, long long, int), const Args &a, int rows, int blocks_per_sm,
                        cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const int nblk = rows / kRowsPerWarp + (rows % kRowsPerWarp != 0); // rows may be INT_MAX
    const long long items = (long long)a.batch * a.n_kv_heads * nblk;
    const long long want = (items + kWarps - 1) / kWarps, cap = (long long)blocks_per_sm * sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(want < cap ? want : cap));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, items, nblk);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace

cudaError_t launch_kv_write(const KvWriteArgs &a, cudaStream_t stream)
{
    // 8 blocks per SM take 152 us for a 128K prompt in bursts, 16 134, 32 129
    return a.kv == SR_KV_E4M3 ? launch_rows(write_kernel<SR_KV_E4M3>, a, a.n_tokens, 32, stream)
                              : launch_rows(write_kernel<SR_KV_INT8>, a, a.n_tokens, 32, stream);
}

cudaError_t launch_kv_read(const KvReadArgs &a, cudaStream_t stream)
{
    return a.kv == SR_KV_E4M3 ? launch_rows(read_kernel<SR_KV_E4M3>, a, a.n_rows, 64, stream)
                              : launch_rows(read_kernel<SR_KV_INT8>, a, a.n_rows, 64, stream);
}

} // namespace sr
