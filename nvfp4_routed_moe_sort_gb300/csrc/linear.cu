// A few tokens times one dense NVFP4 matrix: y[m, n] = act(alpha * sum_k x[m, k] * w[n, k]).
//
// A weight is code * scale of its 16-value block, both read in their linear layout. Products
// with bf16 or e4m3 activations are exact in FP32, sums are FP32, and alpha, the activation
// and the BF16 rounding come once at the end.
#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kLinThreads = 256;
constexpr int kLinTokens = 16;

struct LinArgs {
  const void* x;
  const float* x_scale;
  const uint8_t* w;
  const uint8_t* sf;
  const float* alpha;
  uint16_t* out;
  int64_t ld_x;
  int x_mode, M, K, N, n_out, act, x_groups;  // N: rows of w; n_out: columns of out
  bool gated;
};

__device__ __forceinline__ float silu(float g) { return __fdiv_rn(g, __fadd_rn(1.0f, expf(-g))); }
__device__ __forceinline__ float gelu(float x) {
  return __fmul_rn(__fmul_rn(0.5f, x), __fadd_rn(1.0f, erff(__fmul_rn(x, 0.70710678118654752f))));
}

// act(g) * u for the gated kinds, act(g) otherwise
__device__ __forceinline__ float activate(int act, float g, float u) {
  switch (act) {
    case MOE_ACT_SWIGLU: return __fmul_rn(silu(g), u);
    case MOE_ACT_GEGLU: return __fmul_rn(gelu(g), u);
    case MOE_ACT_RELU2: {
      const float r = fmaxf(g, 0.0f);
      return __fmul_rn(r, r);
    }
    case MOE_ACT_GELU: return gelu(g);
    case MOE_ACT_RELU: return fmaxf(g, 0.0f);
    case MOE_ACT_SILU: return silu(g);
    default: return g;
  }
}

__device__ __forceinline__ float e2m1_to_f32(uint32_t c) {
  const uint32_t e = (c >> 1) & 3, m = c & 1;
  const float v = e == 0 ? 0.5f * m : (1.0f + 0.5f * m) * static_cast<float>(1u << (e - 1));
  return (c & 8) ? -v : v;
}

__device__ __forceinline__ float load_x(const LinArgs& a, int64_t m, int k) {
  if (a.x_mode == MOE_FP8_NONE)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.x)[m * a.ld_x + k]) << 16);
  const uint32_t b = static_cast<const uint8_t*>(a.x)[m * a.ld_x + k];
  const float v = (b & 0x7F) == 0x7F ? __uint_as_float(0x7FFFFFFFu) : e4m3_to_f32(b);
  return v * a.x_scale[m * a.x_groups + (a.x_mode == MOE_FP8_PER_GROUP ? k / MOE_FP8_GROUP : 0)];
}

// one warp per output column and token, lanes over the 16-value blocks of its weight rows
__global__ void __launch_bounds__(kLinThreads) linear_kernel(LinArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kLinThreads + threadIdx.x) >> 5;
  const int m = blockIdx.y;
  if (i >= a.n_out) return;
  float y[2] = {0.0f, 0.0f};
  for (int h = 0; h < (a.gated ? 2 : 1); ++h) {
    const int64_t n = i + (h ? a.n_out : 0);
    float acc = 0.0f;
    for (int b = lane; b < a.K / kBlock; b += 32) {
      const float s = e4m3_to_f32(a.sf[n * (a.K / kBlock) + b]);
      for (int k = 0; k < kBlock; ++k) {
        const uint32_t c = a.w[n * (a.K / 2) + b * 8 + k / 2] >> (4 * (k & 1));
        acc += load_x(a, m, b * kBlock + k) * (e2m1_to_f32(c & 15) * s);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    y[h] = acc * *a.alpha;
  }
  if (lane == 0)
    a.out[static_cast<int64_t>(m) * a.n_out + i] =
        __bfloat16_as_ushort(__float2bfloat16_rn(activate(a.act, y[0], y[1])));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_linear_fp4(const void* x, int64_t ld_x, const float* x_scale, int32_t x_scale_mode,
                                       int32_t M, int32_t K, const uint8_t* w, const uint8_t* w_sf,
                                       const float* alpha, int32_t N, int32_t activation, uint16_t* out,
                                       moe_stream_t stream) {
  MOE_CHECK(M >= 0 && N >= 1 && K > 0 && ld_x >= K, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(x_scale_mode >= MOE_FP8_NONE && x_scale_mode <= MOE_FP8_PER_GROUP, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(activation >= MOE_ACT_SWIGLU && activation <= MOE_ACT_IDENTITY, MOE_ERR_INVALID_ARGUMENT);
  const bool gated = activation == MOE_ACT_SWIGLU || activation == MOE_ACT_GEGLU;
  MOE_CHECK(!gated || N % 2 == 0, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(K % kBlock == 0 && K <= 65536, MOE_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return MOE_OK;
  const bool fp8 = x_scale_mode != MOE_FP8_NONE;
  MOE_CHECK(x && w && w_sf && alpha && out && fp8 == (x_scale != nullptr), MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(aligned16(x) && aligned16(x_scale) && aligned16(w) && aligned16(w_sf) && aligned16(alpha) &&
                aligned16(out) && ld_x % (fp8 ? 16 : 8) == 0,
            MOE_ERR_MISALIGNED);
  LinArgs a = {x, x_scale, w, w_sf, alpha, out, ld_x, x_scale_mode, M, K, N, gated ? N / 2 : N, activation,
               x_scale_mode == MOE_FP8_PER_GROUP ? (K + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP : 1, gated};
  const size_t ob = static_cast<size_t>(M) * a.n_out * 2;
  MOE_CHECK(!overlaps(out, ob, x, (static_cast<size_t>(M - 1) * ld_x + K) * (fp8 ? 1 : 2)) &&
                !overlaps(out, ob, w, static_cast<size_t>(N) * K / 2) &&
                !overlaps(out, ob, w_sf, static_cast<size_t>(N) * K / kBlock) && !overlaps(out, ob, alpha, 4) &&
                !overlaps(out, ob, x_scale, static_cast<size_t>(M) * a.x_groups * 4),
            MOE_ERR_OVERLAP);
  const unsigned warps = kLinThreads / 32;
  return launch_pdl(linear_kernel, dim3((a.n_out + warps - 1) / warps, M), dim3(kLinThreads), 0, as_stream(stream), a);
}
