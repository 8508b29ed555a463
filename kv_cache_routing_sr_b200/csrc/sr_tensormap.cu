// Tensor maps of the KV caches for the TMA copies.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "sr_internal.h"

namespace sr {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

} // namespace

// 3-D view [units][Lmax][128] of a cache; a box is 128 bytes of a row (64 bf16
// values, or all 128 codes; swizzled 128B) by `rows` positions of one unit. Rows
// past `len` (at most Lmax) read as zero.
bool make_cache_map(CUtensorMap *map, const void *base, int units, int lmax, int rows, bool quant, int len)
{
    auto fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t row_bytes = quant ? kHeadDim : kHeadDim * 2;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)len, (cuuint64_t)units};
    cuuint64_t strides[2] = {row_bytes, (cuuint64_t)lmax * row_bytes};
    cuuint32_t box[3] = {quant ? 128u : 64u, (cuuint32_t)rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                          const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

} // namespace sr
