// Tensor maps of byte matrices for tiled TMA loads.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace moe {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  // the driver entry point is looked up once per process (or twice, by two host threads whose first calls meet); it holds no
  // device state
  static std::atomic<EncodeTiledFn> known{nullptr};
  EncodeTiledFn fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
      known.store(fn, std::memory_order_release);
    }
  }
  return fn;
}

// 2D uint8 map over `rows` rows of `row_bytes` bytes, `stride` bytes apart, box = 128 bytes x box_rows, 128B swizzle.
// Columns past row_bytes and rows past `rows` read as zero.
inline bool encode_rows(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint64_t stride,
                        uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {stride};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t es[2] = {1, 1};
  const auto encode = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult result = encode();
  if (result == CUDA_ERROR_INVALID_CONTEXT) {
    // A host thread whose first call of CUDA this is has no context yet, which a call of the driver's needs and does not
    // make; setting the device that it has anyway makes its context current.
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
    result = encode();
  }
  return result == CUDA_SUCCESS;
}

}  // namespace moe
