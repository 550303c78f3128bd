// BF16 rows to E4M3 with FP32 scales: one per row and 128 columns (activations), or one per 128 x 128
// block (weights).
//
// Per scale group scale = amax|x| / 448 (1 when amax is 0), y = e4m3(x * (448 / amax)): the rule of the
// norm's E4M3 output.
#include <math.h>

#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kGroup = MOE_FP8_GROUP;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float bf16_at(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ float scale_of(float amax) { return amax == 0.0f ? 1.0f : __fdiv_rn(amax, 448.0f); }
// x * (448 / amax) with the quotient kept finite for the smallest amax (up is a power of two)
struct Inverse {
  float up, inv;
};
__device__ __forceinline__ Inverse inverse_of(float amax) {
  const float up = amax < 0x1p-64f ? 0x1p64f : 1.0f;
  return {up, amax == 0.0f ? 1.0f : __fdiv_rn(448.0f, amax * up)};
}

struct QuantArgs {
  const uint16_t* x;
  uint8_t* y;
  float* scale;
  int64_t ld_x;
  int M, K, groups;
};

// one warp per scale group, four values a lane
__global__ void __launch_bounds__(256) quantize_fp8_rows_kernel(QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(a.M) * a.groups) return;
  const int64_t m = item / a.groups;
  const int col = static_cast<int>(item - m * a.groups) * kGroup;
  float v[4], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = col + lane + 32 * i;
    v[i] = c < a.K ? bf16_at(a.x + m * a.ld_x + c) : 0.0f;
    top = max_nan(top, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) a.scale[item] = scale_of(top);
  const Inverse inv = inverse_of(top);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = col + lane + 32 * i;
    if (c < a.K) a.y[m * a.K + c] = static_cast<uint8_t>(f32_to_e4m3(__fmul_rn(v[i] * inv.up, inv.inv)));
  }
}

// one block of 8 warps per 128 x 128 values, 16 rows a warp
__global__ void __launch_bounds__(256) quantize_fp8_blocks_kernel(QuantArgs a) {
  __shared__ float red[8];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kGroup;
  const int64_t row = static_cast<int64_t>(blockIdx.y) * kGroup;
  float v[16][4], top = 0.0f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t m = row + warp + 8 * r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = col + lane + 32 * i;
      v[r][i] = m < a.M && c < a.K ? bf16_at(a.x + m * a.ld_x + c) : 0.0f;
      top = max_nan(top, fabsf(v[r][i]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = max_nan(top, red[w]);
  if (threadIdx.x == 0) a.scale[static_cast<int64_t>(blockIdx.y) * a.groups + blockIdx.x] = scale_of(top);
  const Inverse inv = inverse_of(top);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t m = row + warp + 8 * r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = col + lane + 32 * i;
      if (m < a.M && c < a.K) a.y[m * a.K + c] = static_cast<uint8_t>(f32_to_e4m3(__fmul_rn(v[r][i] * inv.up, inv.inv)));
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_quantize_fp8(const uint16_t* x, int64_t ld_x, int32_t M, int32_t K, int32_t block_rows,
                                         uint8_t* y, float* y_scale, moe_stream_t stream) {
  MOE_CHECK(M >= 0 && K > 0 && ld_x >= K, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(block_rows == 1 || block_rows == kGroup, MOE_ERR_INVALID_ARGUMENT);
  if (M == 0) return MOE_OK;
  MOE_CHECK(x && y && y_scale, MOE_ERR_INVALID_ARGUMENT);
  const int groups = (K - 1) / kGroup + 1;
  const int64_t strips = (M - 1) / block_rows + 1;
  MOE_CHECK(block_rows == 1 ? strips * groups <= (int64_t(8) << 31) - 8 : strips <= 65535, MOE_ERR_UNSUPPORTED_SHAPE);
  MOE_CHECK((reinterpret_cast<uintptr_t>(x) & 1) == 0 && (reinterpret_cast<uintptr_t>(y_scale) & 3) == 0, MOE_ERR_MISALIGNED);
  const size_t in_bytes = (static_cast<size_t>(M - 1) * ld_x + K) * 2, y_bytes = static_cast<size_t>(M) * K;
  const size_t scale_bytes = static_cast<size_t>(strips) * groups * 4;
  MOE_CHECK(!overlaps(y, y_bytes, x, in_bytes) && !overlaps(y_scale, scale_bytes, x, in_bytes) &&
                !overlaps(y, y_bytes, y_scale, scale_bytes),
            MOE_ERR_OVERLAP);
  const QuantArgs a = {x, y, y_scale, ld_x, M, K, groups};
  if (block_rows == 1) {
    const dim3 grid(static_cast<unsigned>((strips * groups + 7) / 8));
    return launch_pdl(quantize_fp8_rows_kernel, grid, dim3(256), 0, as_stream(stream), a);
  }
  const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(strips));
  return launch_pdl(quantize_fp8_blocks_kernel, grid, dim3(256), 0, as_stream(stream), a);
}
