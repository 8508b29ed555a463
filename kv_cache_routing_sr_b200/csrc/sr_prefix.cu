// Attention of one decode token of every sequence of a batch over a prefix that
// all of them share, joined with each sequence's own suffix.
//
// Method: the split-K reduction of the SinkRouter README's decode-time procedure
// list, carried across two caches: softmax attention over a union of position
// ranges is sum_r exp(lse_r - lse) o_r with lse = log sum_r exp(lse_r).
//
// One CTA of 128 threads per query row: 128 positions at a time, each thread
// takes one position's logit and then one output column, with a running maximum
// and sum in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sinkrouter.h"
#include "sr_internal.h"
#include "sr_ptx.cuh"

namespace sr {
namespace {

constexpr float kScale = 0.08838834764831845f; // 1 / sqrt(128)

template <typename Op> __device__ __forceinline__ float block_reduce(float x, float *sm, Op op)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sm[threadIdx.x >> 5] = x;
    __syncthreads();
    return op(op(sm[0], sm[1]), op(sm[2], sm[3]));
}

__global__ void __launch_bounds__(kHeadDim) prefix_rows_kernel(PrefixArgs a)
{
    __shared__ float qs[kHeadDim], ps[kHeadDim], red[4];
    grid_dependency_wait();
    grid_launch_dependents();
    const int row = blockIdx.x, t = threadIdx.x; // row = b * Hq + h
    const int M = a.n_q_heads / a.n_kv_heads;
    const int b = row / a.n_q_heads, g = (row - b * a.n_q_heads) / M;
    const int u = b * a.n_kv_heads + g;
    const __nv_bfloat16 *v0 = static_cast<const __nv_bfloat16 *>(a.v0) + (size_t)u * kHeadDim;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out);
    const size_t at = (size_t)row * kHeadDim + t;
    if (a.mask[u]) {
        if (a.out_f32)
            a.out_f32[at] = __bfloat162float(v0[t]);
        else
            out[at] = v0[t];
        if (a.lse && t == 0)
            a.lse[row] = __int_as_float(0x7fc00000);
        return;
    }
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k_prefix) + (size_t)g * a.max_seq_len * kHeadDim;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_prefix) + (size_t)g * a.max_seq_len * kHeadDim;
    qs[t] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[at]) * kScale;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int p0 = 0; p0 < a.prefix_len; p0 += kHeadDim) {
        const int n = min(kHeadDim, a.prefix_len - p0);
        __syncthreads();
        float s = -INFINITY;
        if (t < n) {
            s = 0.f;
            const __nv_bfloat162 *kr = reinterpret_cast<const __nv_bfloat162 *>(k + (size_t)(p0 + t) * kHeadDim);
            for (int i = 0; i < kHeadDim / 2; ++i) {
                const float2 x = __bfloat1622float2(kr[i]);
                s = fmaf(qs[2 * i], x.x, s);
                s = fmaf(qs[2 * i + 1], x.y, s);
            }
        }
        const float mn = fmaxf(m, block_reduce(s, red, [](float x, float y) { return fmaxf(x, y); }));
        const float w = t < n ? expf(s - mn) : 0.f, keep = expf(m - mn);
        ps[t] = w;
        l = l * keep + block_reduce(w, red, [](float x, float y) { return x + y; });
        o *= keep;
        for (int i = 0; i < n; ++i)
            o = fmaf(ps[i], __bfloat162float(v[(size_t)(p0 + i) * kHeadDim + t]), o);
        m = mn;
    }
    float lse = l > 0.f ? m + logf(l) : (l == 0.f ? -INFINITY : l);
    o = l == 0.f ? 0.f : o / l;
    if (a.o_suffix) {
        const float ls = a.lse_suffix[row], top = fmaxf(lse, ls);
        if (top == -INFINITY) {
            o = 0.f;
        } else {
            const float wp = expf(lse - top), ws = expf(ls - top);
            o = (wp * o + ws * a.o_suffix[at]) / (wp + ws);
            lse = top + logf(wp + ws);
        }
    }
    if (a.out_f32)
        a.out_f32[at] = o;
    else
        out[at] = __float2bfloat16_rn(o);
    if (a.lse && t == 0)
        a.lse[row] = lse;
}

} // namespace

size_t prefix_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_prefix(const PrefixArgs &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.batch * a.n_q_heads));
    cfg.blockDim = dim3(kHeadDim);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, prefix_rows_kernel, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace sr
