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
// that. Layout: eight lanes a row, 16 values a lane, so that a lane's codes are
// one 16-byte word; a warp takes four consecutive tokens of one KV head (four
// rows that are neighbours in the cache, 512 contiguous bytes, whose scale
// pairs fill one 32-byte sector) and both the key and the value of each, and
// neighbouring warps take neighbouring heads, which are neighbours in the
// projection's layout.
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

template <int KV> __global__ void __launch_bounds__(kThreads) write_kernel(KvWriteArgs a, long long items, int nblk)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, j = lane & 7;
    const long long nw = (long long)gridDim.x * kWarps;
    for (long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); i < items; i += nw) {
        const Item it = item_of(i, a.n_kv_heads, nblk, lane);
        const int n = clamp_count(__ldg(a.n + it.b), a.n_tokens, a.error);
        const long long slot = (long long)__ldg(a.start + it.b) + it.t;
        bool live = it.t < n;
        if (live && (slot < 0 || slot >= a.max_seq_len)) {
            live = false;
            if (a.error)
                atomicOr(a.error, SR_DEVERR_APPEND_SLOT);
        }
        uint4 x[2][2] = {};
        if (live) {
            const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.k_new) +
                                                             it.b * a.ks.batch + it.t * a.ks.token + it.g * a.ks.head);
            const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.v_new) +
                                                             it.b * a.vs.batch + it.t * a.vs.token + it.g * a.vs.head);
            x[0][0] = __ldg(k + 2 * j);
            x[0][1] = __ldg(k + 2 * j + 1);
            x[1][0] = __ldg(v + 2 * j);
            x[1][1] = __ldg(v + 2 * j + 1);
        }
        RowQuant rq[2];
        uint4 codes[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t w[8] = {x[s][0].x, x[s][0].y, x[s][0].z, x[s][0].w,
                                   x[s][1].x, x[s][1].y, x[s][1].z, x[s][1].w};
            uint32_t m = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                m = abs_max_bf16x2(m, w[e]);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
            rq[s] = row_quant<KV>(max(m & 0xffffu, m >> 16));
            codes[s] = make_uint4(quant4<KV>(w[0], w[1], rq[s]), quant4<KV>(w[2], w[3], rq[s]),
                                  quant4<KV>(w[4], w[5], rq[s]), quant4<KV>(w[6], w[7], rq[s]));
        }
        if (!live)
            continue;
        const size_t u = (size_t)it.b * a.n_kv_heads + it.g;
        const size_t row = u * a.max_seq_len + (size_t)slot;
        reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.k_cache) + row * kHeadDim)[j] = codes[0];
        reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.v_cache) + row * kHeadDim)[j] = codes[1];
        if (j == 0)
            reinterpret_cast<float2 *>(a.scales)[row] = make_float2(rq[0].scale, rq[1].scale);
        if (slot == 0 && a.k0) {
            uint4 *k0 = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.k0) + u * kHeadDim);
            uint4 *v0 = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.v0) + u * kHeadDim);
            k0[2 * j] = x[0][0];
            k0[2 * j + 1] = x[0][1];
            v0[2 * j] = x[1][0];
            v0[2 * j + 1] = x[1][1];
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
        const int n = clamp_count(__ldg(a.n + it.b), a.n_rows, a.error);
        const long long pos = (long long)__ldg(a.start + it.b) + it.t;
        if (it.t >= n)
            continue;
        if (pos < 0 || pos >= a.max_seq_len) {
            if (a.error)
                atomicOr(a.error, SR_DEVERR_APPEND_SLOT);
            continue;
        }
        const size_t u = (size_t)it.b * a.n_kv_heads + it.g;
        const size_t row = u * a.max_seq_len + (size_t)pos;
        const uint4 kc = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.k_cache) + row * kHeadDim) + j);
        const uint4 vc = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.v_cache) + row * kHeadDim) + j);
        const float2 s = __ldg(reinterpret_cast<const float2 *>(a.scales) + row);
        const size_t to = (u * a.n_rows + it.t) * kHeadDim;
        uint4 *ko = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.k_out) + to);
        uint4 *vo = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.v_out) + to);
        ko[2 * j] = pack8(dequant4<KV>(kc.x, s.x), dequant4<KV>(kc.y, s.x));
        ko[2 * j + 1] = pack8(dequant4<KV>(kc.z, s.x), dequant4<KV>(kc.w, s.x));
        vo[2 * j] = pack8(dequant4<KV>(vc.x, s.y), dequant4<KV>(vc.y, s.y));
        vo[2 * j + 1] = pack8(dequant4<KV>(vc.z, s.y), dequant4<KV>(vc.w, s.y));
    }
}

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args, long long, int), const Args &a, int rows, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    const int nblk = (rows + kRowsPerWarp - 1) / kRowsPerWarp;
    const long long items = (long long)a.batch * a.n_kv_heads * nblk;
    const long long want = (items + kWarps - 1) / kWarps, cap = 64ll * sms;
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
    return a.kv == SR_KV_E4M3 ? launch_rows(write_kernel<SR_KV_E4M3>, a, a.n_tokens, stream)
                              : launch_rows(write_kernel<SR_KV_INT8>, a, a.n_tokens, stream);
}

cudaError_t launch_kv_read(const KvReadArgs &a, cudaStream_t stream)
{
    return a.kv == SR_KV_E4M3 ? launch_rows(read_kernel<SR_KV_E4M3>, a, a.n_rows, stream)
                              : launch_rows(read_kernel<SR_KV_INT8>, a, a.n_rows, stream);
}

} // namespace sr
