// Tensor maps of the TMA kernels, encoded on the host at launch.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace moe {
namespace {

// The driver's encoder: looked up by the first launch, by one thread where
// several launch at once, and again after a look-up that failed.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found{nullptr};
    static std::mutex mutex;
    if (auto fn = found.load(std::memory_order_acquire)) return fn;
    std::lock_guard<std::mutex> lock(mutex);
    if (auto fn = found.load(std::memory_order_relaxed)) return fn;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        found.store(reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p), std::memory_order_release);
    return found.load(std::memory_order_relaxed);
}

// 2-D tensor map over a row-major [rows, cols] matrix of bf16 (or, with
// bytes = true, of 8-bit codes) with the 128-byte swizzle; box = box_cols x
// box_rows (box_cols elements must span 128 bytes).
bool make_tmap(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_cols,
               uint32_t box_rows, bool bytes = false) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * (bytes ? 1 : 2)};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t es[2] = {1, 1};
    const CUresult r = fn(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                          const_cast<void *>(ptr), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moe
