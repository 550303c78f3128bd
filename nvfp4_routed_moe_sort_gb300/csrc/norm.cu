// Root-mean-square norm with the residual's addition, and its scaled E4M3 output.
//
// Per row: h = x + r, f = h * rsqrt(sum(h^2) / H + eps) * w; bf16(h), bf16(f), and per scale
// group scale = amax|f| / 448, e4m3(f * (448 / amax)).
#include <math.h>

#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormMaxCols = 32768;

// maximum that lets a NaN through (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

struct NormArgs {
  const uint16_t* x;
  const uint16_t* r;
  const uint16_t* w;
  uint16_t* y;
  uint16_t* r_out;
  uint8_t* y8;
  float* scale;
  int64_t ld_x, ld_r;
  int M, H, groups, group;  // group: columns of one scale
  float eps;
};

__global__ void __launch_bounds__(kNormThreads) norm_rows_kernel(NormArgs a) {
  extern __shared__ float row[];  // h, then f
  __shared__ float red[kNormThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t m = blockIdx.x;
  float sum = 0.0f;
  for (int i = tid; i < a.H; i += kNormThreads) {
    float h = bf16_to_f32(a.x[m * a.ld_x + i]);
    if (a.r) h = __fadd_rn(h, bf16_to_f32(a.r[m * a.ld_r + i]));
    if (a.r_out) a.r_out[m * a.H + i] = f32_to_bf16(h);
    row[i] = h;
    sum += h * h;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 32; ++i) sum += red[i];
  const float rstd = rsqrtf(sum / static_cast<float>(a.H) + a.eps);
  for (int i = tid; i < a.H; i += kNormThreads) {
    const float f = __fmul_rn(__fmul_rn(row[i], rstd), bf16_to_f32(a.w[i]));
    row[i] = f;
    if (a.y) a.y[m * a.H + i] = f32_to_bf16(f);
  }
  if (!a.y8) return;
  __syncthreads();
  for (int g = warp; g < a.groups; g += kNormThreads / 32) {
    const int end = min(a.H, (g + 1) * a.group);
    float amax = 0.0f;
    for (int i = g * a.group + lane; i < end; i += 32) amax = max_nan(amax, fabsf(row[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float inv = amax == 0.0f ? 1.0f : __fdiv_rn(448.0f, amax);
    if (lane == 0) a.scale[m * a.groups + g] = amax == 0.0f ? 1.0f : __fdiv_rn(amax, 448.0f);
    for (int i = g * a.group + lane; i < end; i += 32)
      a.y8[m * a.H + i] = static_cast<uint8_t>(f32_to_e4m3(__fmul_rn(row[i], inv)));
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_add_rmsnorm(const uint16_t* x, int64_t ld_x, const uint16_t* residual, int64_t ld_r,
                                        const uint16_t* weight, int32_t M, int32_t H, float eps, int32_t fp8_scale,
                                        uint16_t* y, uint16_t* residual_out, uint8_t* y8, float* y8_scale,
                                        moe_stream_t stream) {
  MOE_CHECK(M >= 0 && H > 0 && ld_x >= H && isfinite(eps) && eps >= 0.0f, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(fp8_scale >= MOE_FP8_NONE && fp8_scale <= MOE_FP8_PER_GROUP, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(H <= kNormMaxCols, MOE_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return MOE_OK;
  MOE_CHECK(x && weight && (y || y8), MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(residual ? ld_r >= H : residual_out == nullptr, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK((y8 != nullptr) == (fp8_scale != MOE_FP8_NONE) && (y8 != nullptr) == (y8_scale != nullptr),
            MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(y) && aligned16(residual_out) &&
                aligned16(y8) && aligned16(y8_scale),
            MOE_ERR_MISALIGNED);
  const int groups = fp8_scale == MOE_FP8_PER_GROUP ? (H + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP : 1;
  const size_t n = static_cast<size_t>(M) * H;
  const void* in[3] = {x, residual, weight};
  const size_t in_bytes[3] = {(static_cast<size_t>(M - 1) * ld_x + H) * 2,
                              residual ? (static_cast<size_t>(M - 1) * ld_r + H) * 2 : 0, static_cast<size_t>(H) * 2};
  const void* out[4] = {residual_out, y, y8, y8_scale};
  const size_t out_bytes[4] = {n * 2, n * 2, n, static_cast<size_t>(M) * groups * 4};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j) {
      if (i == 0 && j == 1 && residual_out == residual && ld_r == H) continue;  // in place
      MOE_CHECK(!overlaps(out[i], out_bytes[i], in[j], in_bytes[j]), MOE_ERR_OVERLAP);
    }
    for (int j = 0; j < i; ++j) MOE_CHECK(!overlaps(out[i], out_bytes[i], out[j], out_bytes[j]), MOE_ERR_OVERLAP);
  }
  NormArgs a = {x, residual, weight, y, residual_out, y8, y8_scale, ld_x, ld_r, M, H, groups,
                fp8_scale == MOE_FP8_PER_GROUP ? MOE_FP8_GROUP : H, eps};
  const size_t smem = static_cast<size_t>(H) * 4;
  MOE_CUDA(cudaFuncSetAttribute(norm_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxCols * 4));
  return launch_pdl(norm_rows_kernel, dim3(M), dim3(kNormThreads), smem, as_stream(stream), a);
}
