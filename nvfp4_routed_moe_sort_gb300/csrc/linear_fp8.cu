// Products of E4M3 activations with an E4M3 matrix that has one FP32 scale per 128 x 128 block.
//
//   y[m, n] = act(sum_b xs[m, b] * ws[n / 128, b] * sum_{k in block b} x[m, k] * w[n, k])
#include <math.h>

#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kGroup = MOE_FP8_GROUP;
constexpr int kTile = 16;

__device__ __forceinline__ float e4m3_value(uint32_t b) {
  return (b & 0x7F) == 0x7F ? __uint_as_float(0x7FFFFFFFu) : e4m3_to_f32(b);
}
__device__ __forceinline__ float silu(float g) { return __fdiv_rn(g, __fadd_rn(1.0f, expf(-g))); }
__device__ __forceinline__ float gelu(float x) {
  return __fmul_rn(__fmul_rn(0.5f, x), __fadd_rn(1.0f, erff(__fmul_rn(x, 0.70710678118654752f))));
}
__device__ __forceinline__ float relu(float x) { return x < 0.0f ? 0.0f : x; }  // lets a NaN through
__device__ __forceinline__ float activate(int act, float g, float u) {
  switch (act) {
    case MOE_ACT_SWIGLU: return __fmul_rn(silu(g), u);
    case MOE_ACT_GEGLU: return __fmul_rn(gelu(g), u);
    case MOE_ACT_RELU2: {
      const float r = relu(g);
      return __fmul_rn(r, r);
    }
    case MOE_ACT_GELU: return gelu(g);
    case MOE_ACT_RELU: return relu(g);
    case MOE_ACT_SILU: return silu(g);
    default: return g;
  }
}

struct Fp8Args {
  const uint8_t* x;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  uint16_t* out;
  int64_t ld_x;
  int M, N, K, groups, act;
  int xs_step, xs_ld;  // per 128 columns and per row: 1 and groups, or 0 and 1
  int cols;            // of out: N, or N / 2
};

__global__ void __launch_bounds__(256) linear_fp8_plain_kernel(Fp8Args a) {
  __shared__ float sx[kTile][kGroup + 1], sw[2][kTile][kGroup + 1];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kTile + ty, n0 = static_cast<int64_t>(blockIdx.y) * kTile;
  const int kinds = a.cols == a.N ? 1 : 2;
  float sum[2] = {0.0f, 0.0f};
  for (int b = 0; b < a.groups; ++b) {
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kGroup; i += 256) {
      const int r = i / kGroup, k = b * kGroup + i % kGroup;
      const int64_t mm = static_cast<int64_t>(blockIdx.x) * kTile + r;
      sx[r][i % kGroup] = mm < a.M && k < a.K ? e4m3_value(a.x[mm * a.ld_x + k]) : 0.0f;
      for (int h = 0; h < kinds; ++h)
        sw[h][r][i % kGroup] = n0 + r < a.cols && k < a.K
                                   ? e4m3_value(a.w[(n0 + r + static_cast<int64_t>(h) * a.cols) * a.K + k]) : 0.0f;
    }
    __syncthreads();
    if (m < a.M && n0 + tx < a.cols) {
      for (int h = 0; h < kinds; ++h) {
        float part = 0.0f;
        for (int k = 0; k < kGroup; ++k) part = fmaf(sx[ty][k], sw[h][tx][k], part);
        const int64_t n = n0 + tx + static_cast<int64_t>(h) * a.cols;
        sum[h] = fmaf(part, a.xs[m * a.xs_ld + b * a.xs_step] * a.ws[n / kGroup * a.groups + b], sum[h]);
      }
    }
  }
  if (m < a.M && n0 + tx < a.cols)
    a.out[m * a.cols + n0 + tx] = __bfloat16_as_ushort(__float2bfloat16_rn(activate(a.act, sum[0], sum[1])));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_linear_fp8(const uint8_t* x, int64_t ld_x, const float* x_scale, int32_t x_scale_mode,
                                       int32_t M, int32_t K, const uint8_t* w, const float* w_scale, int32_t N,
                                       int32_t activation, uint16_t* out, int32_t* dev_status, moe_stream_t stream) {
  MOE_CHECK(M >= 0 && K > 0 && N > 0 && ld_x >= K, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(x_scale_mode == MOE_FP8_PER_TOKEN || x_scale_mode == MOE_FP8_PER_GROUP, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(activation >= MOE_ACT_SWIGLU && activation <= MOE_ACT_IDENTITY, MOE_ERR_INVALID_ARGUMENT);
  const bool gated = activation == MOE_ACT_SWIGLU || activation == MOE_ACT_GEGLU;
  MOE_CHECK(K % 16 == 0 && K <= 65536 && M <= (1 << 22) && N <= (1 << 22), MOE_ERR_UNSUPPORTED_SHAPE);
  MOE_CHECK(!gated || N % (2 * kGroup) == 0, MOE_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return MOE_OK;
  MOE_CHECK(x && x_scale && w && w_scale && out, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(aligned16(x) && aligned16(w) && aligned16(out) && ld_x % 16 == 0 &&
                ((reinterpret_cast<uintptr_t>(x_scale) | reinterpret_cast<uintptr_t>(w_scale)) & 3) == 0,
            MOE_ERR_MISALIGNED);
  const int groups = (K - 1) / kGroup + 1, cols = gated ? N / 2 : N;
  const bool per_token = x_scale_mode == MOE_FP8_PER_TOKEN;
  const size_t out_bytes = static_cast<size_t>(M) * cols * 2;
  MOE_CHECK(!overlaps(out, out_bytes, x, static_cast<size_t>(M - 1) * ld_x + K) &&
                !overlaps(out, out_bytes, w, static_cast<size_t>(N) * K) &&
                !overlaps(out, out_bytes, x_scale, static_cast<size_t>(M) * (per_token ? 1 : groups) * 4) &&
                !overlaps(out, out_bytes, w_scale, static_cast<size_t>((N - 1) / kGroup + 1) * groups * 4),
            MOE_ERR_OVERLAP);
  const Fp8Args a = {x, x_scale, w, w_scale, out, ld_x, M, N, K, groups, activation, per_token ? 0 : 1, per_token ? 1 : groups, cols};
  const dim3 grid(static_cast<unsigned>((M - 1) / kTile + 1), static_cast<unsigned>((cols - 1) / kTile + 1));
  MOE_CHECK(grid.y <= 65535, MOE_ERR_UNSUPPORTED_SHAPE);
  return launch_pdl(linear_fp8_plain_kernel, grid, dim3(256), 0, as_stream(stream), a);
}
