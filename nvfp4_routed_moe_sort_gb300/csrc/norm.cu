// Root-mean-square norm with the residual's addition, and its scaled E4M3 output.
//
// Per row: h = x + r, f = h * rsqrt(sum(h^2) / H + eps) * w; bf16(h), bf16(f), and per scale
// group scale = amax|f| / 448, e4m3(f * (448 / amax)).
//
// Bound by HBM (9 bytes per value with every output); few rows by the chain load - sum - store. A
// row stays in the registers of its warps between its one read and its one write. An item of a
// warp is 256 columns, eight neighbouring ones a lane, so that 16 lanes hold a scale group. Rows that are
// not whole 16-byte pieces are read and written by the value (or by pairs) side by side and change
// hands in shared memory, so that every alignment adds in the same order. Sums and scales meet
// in shared memory only where a row has several warps. Measured: 16384 x 4096 with residual and
// grouped E4M3 90.7 us (6.7 TB/s), 1 x 2048 2.1 us, 777 x 1536 3.8 us and 777 x 1531 5.0 us.
#include <math.h>

#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kNormMaxCols = 32768;

// maximum that lets a NaN through (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* r;
  const uint16_t* w;
  uint16_t* y;
  uint16_t* r_out;
  uint8_t* y8;
  float* scale;
  int64_t ld_x, ld_r;
  int M, H, fp8, groups, warps;  // warps: of one row
  float eps;
};

constexpr int kItem = 256;
constexpr int kNormWarps = 32;

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack8(float* v, uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}

template <int V> struct Piece;  // V values of BF16, and of E4M3
template <> struct Piece<2> { using Bf16 = uint32_t; using Fp8 = uint16_t; };
template <> struct Piece<1> { using Bf16 = uint16_t; using Fp8 = uint8_t; };

// One item as a lane reads it: its eight values (V == 8), or pieces of V values 32 pieces apart
template <int V>
struct Raw {
  using T = typename Piece<V>::Bf16;
  T v[8 / V];
  __device__ __forceinline__ void load(const uint16_t* p, int lane, int left) {
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      v[i] = 0;
      if ((i * 32 + lane) * V < left) v[i] = *reinterpret_cast<const T*>(p + (i * 32 + lane) * V);
    }
  }
  __device__ __forceinline__ uint4 mine(uint8_t* turn, int lane) const {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) reinterpret_cast<T*>(turn)[i * 32 + lane] = v[i];
    __syncwarp();
    return reinterpret_cast<const uint4*>(turn)[lane];
  }
};
template <>
struct Raw<8> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p, int lane, int left) {
    v = make_uint4(0, 0, 0, 0);
    if (8 * lane < left) v = *reinterpret_cast<const uint4*>(p + 8 * lane);
  }
  __device__ __forceinline__ uint4 mine(uint8_t*, int) const { return v; }
};

// An item's `left` first values, eight to a lane in u, to memory
template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, uint4 u, uint8_t* turn, int lane, int left) {
  if constexpr (V == 8) {
    if (8 * lane < left) *reinterpret_cast<uint4*>(p + 8 * lane) = u;
  } else {
    using T = typename Piece<V>::Bf16;
    __syncwarp();
    reinterpret_cast<uint4*>(turn)[lane] = u;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8 / V; ++i)
      if ((i * 32 + lane) * V < left) *reinterpret_cast<T*>(p + (i * 32 + lane) * V) = reinterpret_cast<const T*>(turn)[i * 32 + lane];
  }
}
template <int V>
__device__ __forceinline__ void store_fp8(uint8_t* p, uint2 u, uint8_t* turn, int lane, int left) {
  if constexpr (V == 8) {
    if (8 * lane < left) *reinterpret_cast<uint2*>(p + 8 * lane) = u;
  } else {
    using T = typename Piece<V>::Fp8;
    __syncwarp();
    reinterpret_cast<uint2*>(turn)[lane] = u;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8 / V; ++i)
      if ((i * 32 + lane) * V < left) *reinterpret_cast<T*>(p + (i * 32 + lane) * V) = reinterpret_cast<const T*>(turn)[i * 32 + lane];
  }
}

// The sum (or NaN-keeping maximum) of v over a row: its warp's lanes, then its warps in order.
template <bool MAX>
__device__ __forceinline__ float over_row(float v, float* red, int warps, int lane, int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  if (warps == 1) return v;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < warps; ++i) v = MAX ? max_nan(v, red[i]) : v + red[i];
  return v;
}

// V: values read at once (8, 2 or 1, by the rows' alignment); ITEMS: items of a warp
template <int V, int ITEMS>
__global__ void __launch_bounds__(ITEMS > 2 ? 512 : 1024) norm_kernel(NormArgs a) {
  __shared__ float red[2][32];
  __shared__ __align__(16) uint8_t turns[V == 8 ? 1 : (ITEMS > 2 ? 16 : 32)][V == 8 ? 16 : 2 * kItem];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, in_block = threadIdx.x >> 5;
  // several rows to a block only where a row is one warp's
  const int row = a.warps == 1 ? in_block : 0, warp = a.warps == 1 ? 0 : in_block;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * (a.warps == 1 ? blockDim.x >> 5 : 1) + row;
  if (m >= a.M) return;
  uint8_t* const turn = turns[V == 8 ? 0 : in_block];
  const int64_t out = m * a.H;
  float h[ITEMS][8];
  {
    Raw<V> x[ITEMS], r[ITEMS];  // all of the row's loads before any of them is used
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = (warp + i * a.warps) * kItem;
      x[i].load(a.x + m * a.ld_x + col, lane, a.H - col);
      if (a.r) r[i].load(a.r + m * a.ld_r + col, lane, a.H - col);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int col = (warp + i * a.warps) * kItem;
      unpack8(h[i], x[i].mine(turn, lane));
      if (a.r) {
        float t[8];
        unpack8(t, r[i].mine(turn, lane));
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = __fadd_rn(h[i][e], t[e]);
        if (a.r_out)
          store_bf16<V>(a.r_out + out + col, make_uint4(bf16x2(h[i][0], h[i][1]), bf16x2(h[i][2], h[i][3]),
                                                        bf16x2(h[i][4], h[i][5]), bf16x2(h[i][6], h[i][7])),
                        turn, lane, a.H - col);
      }
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += h[i][e] * h[i][e];
  sum = over_row<false>(sum, red[0], a.warps, lane, warp);
  const float rstd = rsqrtf(sum / static_cast<float>(a.H) + a.eps);

  float amax[ITEMS], most = 0.0f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = (warp + i * a.warps) * kItem;
    float w[8];
    Raw<8> raw;  // the weight itself is aligned; its last piece may be short
    if (V == 8 || col + 8 * lane + 8 <= a.H) {
      raw.load(a.w + col, lane, a.H - col);
      unpack8(w, raw.v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        w[e] = 0.0f;
        if (col + 8 * lane + e < a.H) w[e] = __uint_as_float(static_cast<uint32_t>(a.w[col + 8 * lane + e]) << 16);
      }
    }
    amax[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] = __fmul_rn(__fmul_rn(h[i][e], rstd), w[e]);
      if (V == 8 ? col + 8 * lane < a.H : col + 8 * lane + e < a.H) amax[i] = max_nan(amax[i], fabsf(h[i][e]));
    }
    if (a.y)
      store_bf16<V>(a.y + out + col, make_uint4(bf16x2(h[i][0], h[i][1]), bf16x2(h[i][2], h[i][3]),
                                                bf16x2(h[i][4], h[i][5]), bf16x2(h[i][6], h[i][7])),
                    turn, lane, a.H - col);
    most = max_nan(most, amax[i]);
  }
  if (a.fp8 == MOE_FP8_NONE) return;
  if (a.fp8 == MOE_FP8_PER_TOKEN) {
    most = over_row<true>(most, red[1], a.warps, lane, warp);
    if (lane == 0 && warp == 0) a.scale[m] = most == 0.0f ? 1.0f : __fdiv_rn(most, 448.0f);
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int col = (warp + i * a.warps) * kItem;
    float top = most;
    if (a.fp8 == MOE_FP8_PER_GROUP) {
      top = amax[i];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      if ((lane & 15) == 0 && col + 8 * lane < a.H)
        a.scale[m * a.groups + (col + 8 * lane) / MOE_FP8_GROUP] = top == 0.0f ? 1.0f : __fdiv_rn(top, 448.0f);
    }
    const float up = top < 0x1p-64f ? 0x1p64f : 1.0f;  // exact, and keeps 448 / amax finite
    const float inv = top == 0.0f ? 1.0f : __fdiv_rn(448.0f, top * up);
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = __fmul_rn(h[i][e] * up, inv);
    store_fp8<V>(a.y8 + out + col, make_uint2(e4m3x2(t[0], t[1]) | e4m3x2(t[2], t[3]) << 16,
                                              e4m3x2(t[4], t[5]) | e4m3x2(t[6], t[7]) << 16),
                 turn, lane, a.H - col);
  }
}

template <int V>
moe_status_t launch_norm(NormArgs a, cudaStream_t s) {
  const int items = (a.H + kItem - 1) / kItem;
  // A warp's items: up to four, its loads in flight together, while that leaves kNormWarps warps to every
  // SM; fewer, so that a row's chain gets shorter, for fewer rows (kNormWarps 16, 32, 64: 2000 x 1001 7.1, 6.05, 6.03
  // us; 777 x 1531 in ones 5.0, in fours 6.8). A block has at most 32 warps, or 16 of over two items.
  int per = 4;
  while (per > 1 && a.M * static_cast<int64_t>((items + per - 1) / per) < kNormWarps * num_sms()) per /= 2;
  while ((items + per - 1) / per > (per > 2 ? 16 : 32)) per *= 2;
  while (per > 1 && items <= per / 2) per /= 2;
  a.warps = (items + per - 1) / per;
  const int rows = a.warps == 1 ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.M) + rows - 1) / rows)), block(32 * a.warps * rows);
  switch (per) {
    case 1: return launch_pdl(norm_kernel<V, 1>, grid, block, 0, s, a);
    case 2: return launch_pdl(norm_kernel<V, 2>, grid, block, 0, s, a);
    case 4: return launch_pdl(norm_kernel<V, 4>, grid, block, 0, s, a);
    default: return launch_pdl(norm_kernel<V, 8>, grid, block, 0, s, a);
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
  const NormArgs a = {x, residual, weight, y, residual_out, y8, y8_scale, ld_x, ld_r, M, H, fp8_scale, groups, 1, eps};
  cudaStream_t s = as_stream(stream);
  if (((H | ld_x | (residual ? ld_r : 0)) & 7) == 0) return launch_norm<8>(a, s);
  if (((H | ld_x | (residual ? ld_r : 0)) & 1) == 0) return launch_norm<2>(a, s);
  return launch_norm<1>(a, s);
}
