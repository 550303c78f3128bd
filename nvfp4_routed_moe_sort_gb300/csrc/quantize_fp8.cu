// BF16 rows to E4M3 with FP32 scales: one per row and 128 columns (activations), or one per 128 x 128
// block (weights).
//
// Per scale group scale = amax|x| / 448 (1 when amax is 0), y = e4m3(x * (448 / amax)): the rule of the
// norm's E4M3 output.
//
// Bound by HBM (3 bytes a value): a group stays in the registers of its half warp between its one read and its one
// write, four groups' loads a thread in flight where rows are many (one where they are few; eight: no faster), their
// maxima folded together. Measured, one call after another (in parentheses by itself, after a flush of L2): 8 x 2048 1.3 us (a
// launch), 16384 x 7160 55 us (60; 6.4 TB/s, 95 % of the copy rate; 70 with each lane making every group's divisions),
// 7168 x 16384 in blocks 52 us (58).
//
// Rows of odd lengths or at odd addresses go by the value, two bytes in and one out: a row's 16-byte pieces do not lie at
// multiples of 16. That is bound by the number of loads and stores: 16384 x 7161 145 us, 7168 x 16383 in blocks 412 us,
// 8 x 2047 1.5 us.
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
  uint32_t M, K, groups;
};

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// the largest magnitude of eight BF16 values, NaN if there is one
__device__ __forceinline__ float most8(const uint4& u) {
  const uint32_t mask = 0x7FFF7FFFu;
  uint32_t m, n;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(u.x & mask), "r"(u.y & mask));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(u.z & mask), "r"(u.w & mask));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
  return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
template <bool TINY>
__device__ __forceinline__ uint2 encode8(const uint4& u, Inverse k) {
  float v[8], t[8];
  unpack8(u, v);
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = __fmul_rn(TINY ? v[e] * k.up : v[e], k.inv);
  return make_uint2(e4m3x2(t[0], t[1]) | e4m3x2(t[2], t[3]) << 16, e4m3x2(t[4], t[5]) | e4m3x2(t[6], t[7]) << 16);
}

// Rows of whole 16-byte pieces: half a warp to a scale group, eight neighbouring values a lane, ITEMS groups' loads
// in flight together. The groups' maxima are folded together (each exchange halves the groups that a lane still
// holds), so that a lane ends with one group's maximum and makes that group's two divisions alone.
template <int ITEMS>
__global__ void __launch_bounds__(256) quantize_fp8_rows_kernel(QuantArgs a, FastDiv groups) {
  static_assert(ITEMS <= 16 && (ITEMS & (ITEMS - 1)) == 0, "the groups fold over the 16 lanes of a half warp");
  constexpr uint32_t all_lanes = 0xffffffffu;
  pdl_wait();
  pdl_trigger();
  const uint32_t half = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const uint32_t all = static_cast<uint32_t>(a.M) * groups.d, first = blockIdx.x * 16 * ITEMS + half;
  uint4 u[ITEMS];
  int64_t at[ITEMS];  // where the eight values go, -1 for nowhere
  float top[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t g = first + 16 * i, row = groups(g), col = (g - row * groups.d) * kGroup + 8 * lane;
    const bool in = g < all && col < a.K;
    at[i] = in ? row * static_cast<int64_t>(a.K) + col : -1;
    u[i] = in ? __ldcs(reinterpret_cast<const uint4*>(a.x + row * a.ld_x + col)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) top[i] = most8(u[i]);
  uint32_t mine = 0;  // the group that this lane ends with
#pragma unroll
  for (int keep = ITEMS / 2, bit = 1; bit < 16; keep /= 2, bit *= 2) {
    const bool upper = keep > 0 && (lane & bit);
    if (upper) mine += keep;
#pragma unroll
    for (int i = 0; i < (keep > 0 ? keep : 1); ++i) {
      const float theirs = keep > 0 && !upper ? top[i + keep] : top[i], ours = upper ? top[i + keep] : top[i];
      top[i] = max_nan(ours, __shfl_xor_sync(all_lanes, theirs, bit));
    }
  }
  const Inverse inv = inverse_of(top[0]);
  if (lane < ITEMS && first + 16 * mine < all) a.scale[first + 16 * mine] = scale_of(top[0]);
  const bool tiny = __any_sync(all_lanes, inv.up != 1.0f);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    int from = 0;  // the lane whose group this is: the group's bits in reverse
#pragma unroll
    for (int keep = ITEMS / 2, bit = 1; keep > 0; keep /= 2, bit *= 2) from |= (i & keep) ? bit : 0;
    Inverse k = {1.0f, __shfl_sync(all_lanes, inv.inv, from, 16)};
    uint2 y;
    if (tiny) {
      k.up = __shfl_sync(all_lanes, inv.up, from, 16);
      y = encode8<true>(u[i], k);
    } else {
      y = encode8<false>(u[i], k);
    }
    if (at[i] >= 0) *reinterpret_cast<uint2*>(a.y + at[i]) = y;
  }
}

// Rows of any length and place: one warp per scale group, four values a lane, each by itself.
__global__ void __launch_bounds__(256) quantize_fp8_odd_rows_kernel(QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(a.M) * a.groups) return;
  const int64_t m = item / a.groups;
  const uint32_t col = static_cast<uint32_t>(item - m * a.groups) * kGroup;
  float v[4], top = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = col + lane + 32 * i;
    v[i] = c < a.K ? bf16_at(a.x + m * a.ld_x + c) : 0.0f;
    top = max_nan(top, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) a.scale[item] = scale_of(top);
  const Inverse inv = inverse_of(top);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = col + lane + 32 * i;
    if (c < a.K) a.y[m * a.K + c] = static_cast<uint8_t>(f32_to_e4m3(__fmul_rn(v[i] * inv.up, inv.inv)));
  }
}

__device__ __forceinline__ float block_max(float top, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = max_nan(top, red[w]);
  return top;
}

// One block of 8 warps per 128 x 128 values. V = 8: rows of whole 16-byte pieces, 16 lanes to a row; V = 1: any rows,
// 16 rows a warp, four values a lane.
template <int V>
__global__ void __launch_bounds__(256) quantize_fp8_blocks_kernel(QuantArgs a) {
  __shared__ float red[8];
  pdl_wait();
  pdl_trigger();
  const int64_t row = static_cast<int64_t>(blockIdx.y) * kGroup;
  float top = 0.0f;
  if constexpr (V == 8) {
    const uint32_t col = blockIdx.x * kGroup + 8 * (threadIdx.x & 15), first = threadIdx.x >> 4;
    uint4 u[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t m = row + first + 16 * r;
      u[r] = make_uint4(0, 0, 0, 0);
      if (m < a.M && col < a.K) u[r] = __ldcs(reinterpret_cast<const uint4*>(a.x + m * a.ld_x + col));
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) top = max_nan(top, most8(u[r]));
    top = block_max(top, red);
    const Inverse inv = inverse_of(top);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t m = row + first + 16 * r;
      if (m < a.M && col < a.K) *reinterpret_cast<uint2*>(a.y + m * a.K + col) = encode8<true>(u[r], inv);
    }
  } else {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * kGroup;
    float v[16][4];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t m = row + warp + 8 * r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = col + lane + 32 * i;
        v[r][i] = m < a.M && c < a.K ? bf16_at(a.x + m * a.ld_x + c) : 0.0f;
        top = max_nan(top, fabsf(v[r][i]));
      }
    }
    top = block_max(top, red);
    const Inverse inv = inverse_of(top);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int64_t m = row + warp + 8 * r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = col + lane + 32 * i;
        if (m < a.M && c < a.K) a.y[m * a.K + c] = static_cast<uint8_t>(f32_to_e4m3(__fmul_rn(v[r][i] * inv.up, inv.inv)));
      }
    }
  }
  if (threadIdx.x == 0) a.scale[static_cast<int64_t>(blockIdx.y) * a.groups + blockIdx.x] = scale_of(top);
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
  const QuantArgs a = {x, y, y_scale, ld_x, static_cast<uint32_t>(M), static_cast<uint32_t>(K), static_cast<uint32_t>(groups)};
  const bool whole = ((K | ld_x) & 7) == 0 && aligned16(x) && (reinterpret_cast<uintptr_t>(y) & 7) == 0;
  cudaStream_t s = as_stream(stream);
  if (block_rows == 1) {
    const int64_t items = strips * groups;
    if (!whole || items >= INT32_MAX - 64) return launch_pdl(quantize_fp8_odd_rows_kernel, dim3(static_cast<unsigned>((items + 7) / 8)), dim3(256), 0, s, a);
    if (items < static_cast<int64_t>(num_sms()) * 16 * 8 * 4)
      return launch_pdl(quantize_fp8_rows_kernel<1>, dim3(static_cast<unsigned>((items + 15) / 16)), dim3(256), 0, s, a, FastDiv(groups));
    return launch_pdl(quantize_fp8_rows_kernel<4>, dim3(static_cast<unsigned>((items + 63) / 64)), dim3(256), 0, s, a, FastDiv(groups));
  }
  const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>(strips));
  return launch_pdl(whole ? quantize_fp8_blocks_kernel<8> : quantize_fp8_blocks_kernel<1>, grid, dim3(256), 0, s, a);
}
