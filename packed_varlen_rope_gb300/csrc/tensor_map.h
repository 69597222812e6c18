// Host side: TMA tensor maps over bf16 views.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "attn_internal.h"

namespace pvr {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, looked up once through the runtime (NULL without a driver).
inline EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// A map of `rank` axes, the first one contiguous; strides (elements) of the others.  Boxes
// are 64 elements of the first axis, in the 128-byte swizzle; what lies outside reads as 0.
inline bool make_map(CUtensorMap *map, const void *base, int rank, const int64_t *extent, const int64_t *stride,
                     const int *box)
{
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr) return false;
    cuuint64_t dims[5], bytes[4];
    cuuint32_t boxes[5], ones[5];
    for (int i = 0; i < rank; ++i) {
        dims[i] = static_cast<cuuint64_t>(extent[i]);
        boxes[i] = static_cast<cuuint32_t>(box[i]);
        ones[i] = 1;
        // an axis of one element is never stepped along: any valid stride will do
        if (i > 0) bytes[i - 1] = extent[i] > 1 ? static_cast<cuuint64_t>(stride[i]) * 2 : 16;
    }
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, bytes, boxes, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows: boxes of `tile` tokens x the heads of a group, the heads side by side.
inline bool make_q_map(CUtensorMap *map, const AttnProblem &p, int tile)
{
    const int64_t ext[3] = {p.d, p.hq, p.n_tokens}, st[3] = {1, p.q.hs, p.q.ts};
    const int box[3] = {64, p.group, tile};
    return make_map(map, p.q.p, 3, ext, st, box);
}

// Keys and values in pages, boxes of `rows` slots; an empty pool becomes a map over one page
// that no coordinate in use reaches.
inline bool make_page_maps(CUtensorMap *k, CUtensorMap *v, const AttnProblem &p, int rows)
{
    const bool none = p.pages.n_pages == 0;
    const int64_t ext[4] = {p.d, p.pages.page_size, p.hkv, none ? 1 : p.pages.n_pages};
    const int64_t ks[4] = {1, p.pages.k_ts, p.pages.k_hs, p.pages.k_ps};
    const int64_t vs[4] = {1, p.pages.v_ts, p.pages.v_hs, p.pages.v_ps};
    const int box[4] = {64, rows, 1, 1};
    return make_map(k, none ? p.q.p : p.pages.k, 4, ext, ks, box) && make_map(v, none ? p.q.p : p.pages.v, 4, ext, vs, box);
}

// Lets `kernel` use `bytes` of dynamic shared memory on the current device (set once each).
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

}  // namespace pvr
