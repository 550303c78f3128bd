// Rotary positions of queries and keys, with one or several position axes.
//
// Pair i of a head is turned by the angle positions[axes[i], n] * inv_freq[i]:
//   (a, b) -> (a cos - b sin, a sin + b cos),
// the pair being values (i, i + rotary_dim / 2) of a head or (2 i, 2 i + 1). The other values of a
// head stay as they are.
//
// The angle. A position times a frequency in 32 bits is off by a tenth of a radian from a million tokens
// on. Only the angle's fraction of a full turn counts, so the frequency becomes a 64-bit fixed-point
// fraction of a turn, inv_freq / (2 pi) * 2^64, and the integer product with the position drops whole
// turns by overflowing: what is left is exact but for the frequency's rounding to 2^-64 of a turn. Sine and
// cosine are those of a float32 in [-1, 1) times pi.
//
// Bound by HBM (4 bytes a turned value): a piece of 16 bytes is read once and written once, each thread fetching its
// next one before it writes; what is not turned is copied while the phases are made. Measured: 8 tokens of 20 heads of
// 128 2.7 us (a launch), 4099 tokens of 32 heads, three quarters of each turned, 14 us (4.7 TB/s with what is copied),
// 16384 tokens of 72 heads 93 us (6.5 TB/s, 95 % of the copy rate; 109 with phases that met in shared memory's banks).
//
// Where rotary_dim is not of 16, head_dim or a stride not of 8, or an address not of 16 bytes, pairs go by the value (two loads and
// stores of two bytes, a division for the pair's head): of those 16384 tokens with 124 of 128 values turned 178 us, with 62
// 234 (64: 97), with 62 of heads of 127 186; 8 tokens of 20 heads 3.6 us (1.9 aligned, one call after another).
#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kMaxAxes = 4;
constexpr int kMaxHeadDim = 1024;

struct RotaryArgs {
  const uint16_t* in[2];  // queries, keys
  uint16_t* out[2];
  int64_t ld_in[2], ld_out[2];
  int heads[2];
  const void* pos;
  const double* inv_freq;
  const uint8_t* axes;
  int32_t* status;
  int64_t ld_pos, N;
  int dim, half, num_axes, pos64, adjacent;
  int copy[2];  // the values that are not turned go to `out` too (it is not `in`)
};

// A frequency in turns, as a fraction of 2^64: m 2^(e - 1075) / (2 pi) with the 53-bit m of a float64, in whole numbers
// (2 / pi in 64 bits), as the card has few units for float64. Whole turns per position fall away at the top.
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(inv_freq));
  const int e = static_cast<int>(b >> 52) & 0x7FF;
  const uint64_t m = (b & 0xFFFFFFFFFFFFFull) | (e ? 1ull << 52 : 0);
  constexpr uint64_t k2OverPi = 0xA2F9836E4E441529ull;
  const uint64_t hi = __umul64hi(m, k2OverPi), lo = m * k2OverPi;
  const int down = 1077 - (e ? e : 1);
  uint64_t t;
  if (down >= 64) t = down < 128 ? hi >> (down - 64) : 0;
  else if (down > 0) t = hi << (64 - down) | lo >> down;
  else t = down > -64 ? lo << -down : 0;
  return b >> 63 ? 0 - t : t;
}

__device__ __forceinline__ int64_t position_of(const RotaryArgs& a, int64_t n, int axis) {
  const int64_t at = axis * a.ld_pos + n;
  return a.pos64 ? static_cast<const int64_t*>(a.pos)[at] : static_cast<const int32_t*>(a.pos)[at];
}

// cosine and sine of `turns` times a position
__device__ __forceinline__ float2 phase_of(int64_t position, uint64_t turns) {
  const uint64_t turn = static_cast<uint64_t>(position) * turns;
  float s, c;
  sincospif(__ll2float_rn(static_cast<int64_t>(turn)) * 0x1p-63f, &s, &c);
  return make_float2(c, s);
}

// the axis of pair i; a pair of an axis that is none is not turned: axis 0, and its frequency counts as 0
__device__ __forceinline__ int axis_of(const RotaryArgs& a, int i, uint64_t& turns) {
  const int axis = a.axes ? a.axes[i] : 0;
  if (axis < a.num_axes) return axis;
  if (a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
  turns = 0;
  return 0;
}

__device__ __forceinline__ float value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Any sizes and places, at two to two and a half times the aligned ones' time: one block per token, its phases first, then its
// heads pair by pair.
__global__ void __launch_bounds__(256) rotary_odd_kernel(RotaryArgs a) {
  __shared__ float2 phase[kMaxHeadDim / 2];
  pdl_wait();
  pdl_trigger();
  const int64_t n = blockIdx.x;
  for (int i = threadIdx.x; i < a.half; i += blockDim.x) {
    uint64_t turns = turns_of(a.inv_freq[i]);
    const int axis = axis_of(a, i, turns);
    phase[i] = phase_of(position_of(a, n, axis), turns);
  }
  __syncthreads();
  for (int t = 0; t < 2; ++t) {
    const uint16_t* in = a.in[t] + n * a.ld_in[t];
    uint16_t* out = a.out[t] + n * a.ld_out[t];
    for (int j = threadIdx.x; j < a.heads[t] * a.half; j += blockDim.x) {
      const int h = j / a.half, i = j - h * a.half;
      const int at = h * a.dim + (a.adjacent ? 2 * i : i), to = at + (a.adjacent ? 1 : a.half);
      const float x = value(in[at]), y = value(in[to]);
      const float2 p = phase[i];
      out[at] = bits(x * p.x - y * p.y);
      out[to] = bits(x * p.y + y * p.x);
    }
    const int rest = a.dim - 2 * a.half;
    if (a.copy[t])
      for (int j = threadIdx.x; j < a.heads[t] * rest; j += blockDim.x) {
        const int at = j / rest * a.dim + 2 * a.half + j % rest;
        out[at] = in[at];
      }
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// eight pairs (x[i], y[i]) of two 16-byte pieces, or (x[0], x[1]), (x[2], x[3]) ... of both where neighbours pair
template <bool ADJACENT>
__device__ __forceinline__ void turn8(uint4& u, uint4& v, const float2* p) {
  uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (ADJACENT) {
      const float a = low(x[i]), b = high(x[i]), c = low(y[i]), d = high(y[i]);
      const float2 s = p[i], t = p[4 + i];
      x[i] = bf16x2(a * s.x - b * s.y, a * s.y + b * s.x);
      y[i] = bf16x2(c * t.x - d * t.y, c * t.y + d * t.x);
    } else {
      const float a = low(x[i]), b = high(x[i]), c = low(y[i]), d = high(y[i]);
      const float2 s = p[2 * i], t = p[2 * i + 1];
      x[i] = bf16x2(a * s.x - c * s.y, b * t.x - d * t.y);
      y[i] = bf16x2(a * s.y + c * s.x, b * t.y + d * t.x);
    }
  }
  u = make_uint4(x[0], x[1], x[2], x[3]);
  v = make_uint4(y[0], y[1], y[2], y[3]);
}

// Heads of whole 16-byte pieces at 16-byte addresses. A block has a run of `tokens` tokens: their phases go to shared
// memory, and each thread takes eight pairs of a head at a time, the first ones fetched before the phases are computed.
// What is not turned is copied where `out` is not `in`. More pieces in flight a thread cost more in resident warps than
// they gain (4: 110 -> 115 us for the long prompt, 16 -> 20 for the images).
template <bool ADJACENT>
__global__ void __launch_bounds__(256, 8) rotary_kernel(RotaryArgs a, int tokens, FastDiv per_token, FastDiv per_head, FastDiv halves,
                                                        FastDiv rest_token, FastDiv rest_head) {
  extern __shared__ __align__(16) uint8_t raw[];
  uint64_t* const turns = reinterpret_cast<uint64_t*>(raw);                    // [half]
  // [tokens][half], two neighbouring pairs of each eight after the other: threads side by side read side by side (eight
  // pairs in a row cost four times the shared memory's turns, and 2 us of 10)
  float2* const phase = reinterpret_cast<float2*>(turns + a.half);
  uint8_t* const axis = reinterpret_cast<uint8_t*>(phase + tokens * a.half);   // [half]
  pdl_wait();
  pdl_trigger();
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int here = static_cast<int>(min(static_cast<int64_t>(tokens), a.N - n0));
  const int all = here * per_token.d, step = 256 * gridDim.y, apart = ADJACENT ? 8 : a.half;
  int j = threadIdx.x + blockIdx.y * 256;
  uint4 u, v;
  // piece j: its place in the queries (0) or keys (1), and its first phase
  const auto place = [&](int& t, int64_t& n, int& at) {
    const int token = per_token(j), r = j - token * per_token.d, head = per_head(r), c = r - head * per_head.d;
    t = head >= a.heads[0];
    n = n0 + token;
    at = token * a.half + 2 * c;
    return (t ? head - a.heads[0] : head) * a.dim + c * (ADJACENT ? 16 : 8);
  };
  const auto fetch = [&] {
    int t, at;
    int64_t n;
    const int in = place(t, n, at);
    const uint16_t* const from = (t ? a.in[1] : a.in[0]) + n * (t ? a.ld_in[1] : a.ld_in[0]) + in;
    u = __ldcs(reinterpret_cast<const uint4*>(from));
    v = __ldcs(reinterpret_cast<const uint4*>(from + apart));
  };
  if (j < all) fetch();
  // what is not turned, while the phases wait for their inputs
  const int rest = rest_head.d;
  if (a.copy[0] || a.copy[1]) {
    for (int i = threadIdx.x + blockIdx.y * 256; i < here * rest_token.d; i += step) {
      const int n = rest_token(i), r = i - n * rest_token.d, head = rest_head(r);
      const int t = head >= a.heads[0];
      const int64_t place = (t ? head - a.heads[0] : head) * a.dim + 2 * a.half + (r - head * rest) * 8;
      if (t ? a.copy[1] : a.copy[0])
        *reinterpret_cast<uint4*>((t ? a.out[1] : a.out[0]) + (n0 + n) * (t ? a.ld_out[1] : a.ld_out[0]) + place) =
            __ldcs(reinterpret_cast<const uint4*>((t ? a.in[1] : a.in[0]) + (n0 + n) * (t ? a.ld_in[1] : a.ld_in[0]) + place));
    }
  }
  for (int i = threadIdx.x; i < a.half; i += 256) {
    uint64_t t = turns_of(a.inv_freq[i]);
    axis[i] = static_cast<uint8_t>(axis_of(a, i, t));
    turns[i] = t;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < here * a.half; i += 256) {
    const int n = halves(i), f = i - n * a.half;
    phase[n * a.half + ((f >> 1 & 3) * per_head.d + (f >> 3)) * 2 + (f & 1)] = phase_of(position_of(a, n0 + n, axis[f]), turns[f]);
  }
  __syncthreads();
  while (j < all) {
    int t, at;
    int64_t n;
    const int in = place(t, n, at);
    uint16_t* const to = (t ? a.out[1] : a.out[0]) + n * (t ? a.ld_out[1] : a.ld_out[0]) + in;
    float2 p[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = *reinterpret_cast<const float4*>(phase + at + i * 2 * per_head.d);
    turn8<ADJACENT>(u, v, p);
    *reinterpret_cast<uint4*>(to) = u;
    *reinterpret_cast<uint4*>(to + apart) = v;
    j += step;
    if (j < all) fetch();
  }
}

template <bool ADJACENT>
moe_status_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  const int chunks = a.half / 8, per = (a.heads[0] + a.heads[1]) * chunks;  // a token's work, in eight pairs
  const int64_t sms = num_sms();
  // many tokens: several to a block, while it has less than one and a half pieces a thread (30000 tokens of five heads of
  // 64: 34 us with one, 10 with eight); few tokens: their heads over several blocks
  int tokens = 1;
  while (tokens < 32 && tokens * 2 * a.half <= 2048 && tokens * per < 384 && a.N >= sms * 4 * tokens) tokens *= 2;
  const int64_t blocks = (a.N + tokens - 1) / tokens;
  int split = 1;
  while (split < 16 && blocks * split * 2 <= sms * 2 && per * tokens > 256 * split) split *= 2;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(split));
  const size_t smem = static_cast<size_t>(a.half) * (sizeof(uint64_t) + tokens * sizeof(float2) + 1);
  RotaryArgs b = a;
  const int rest = (a.dim - 2 * a.half) / 8, left = rest > 0 ? rest : 1;
  if (rest == 0) b.copy[0] = b.copy[1] = 0;
  return launch_pdl(rotary_kernel<ADJACENT>, grid, dim3(256), smem, s, b, tokens, FastDiv(per), FastDiv(chunks), FastDiv(a.half),
                    FastDiv((a.heads[0] + a.heads[1]) * left), FastDiv(left));
}

// rows of `width` values every `ld` values; whether two of them share memory. Slices of one wider row do not.
bool rows_overlap(const uint16_t* a, int64_t lda, int64_t wa, const uint16_t* b, int64_t ldb, int64_t wb, int64_t rows) {
  if (wa == 0 || wb == 0) return false;
  if (!overlaps(a, (static_cast<size_t>(rows - 1) * lda + wa) * 2, b, (static_cast<size_t>(rows - 1) * ldb + wb) * 2)) return false;
  if (lda != ldb) return true;
  int64_t apart = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(b)) - static_cast<int64_t>(reinterpret_cast<uintptr_t>(a))) / 2 % lda;
  if (apart < 0) apart += lda;
  return apart < wa || apart + wb > lda;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_rotary(const uint16_t* q, int64_t ld_q, int32_t num_q_heads, const uint16_t* k, int64_t ld_k,
                                   int32_t num_k_heads, int32_t head_dim, int32_t rotary_dim, int32_t adjacent,
                                   const void* positions, int32_t position_bytes, int64_t ld_positions, int32_t num_axes,
                                   const double* inv_freq, const uint8_t* axes, int32_t N, uint16_t* q_out, int64_t ld_q_out,
                                   uint16_t* k_out, int64_t ld_k_out, int32_t* dev_status, moe_stream_t stream) {
  MOE_CHECK(N >= 0 && num_q_heads > 0 && num_k_heads >= 0 && head_dim > 0 && rotary_dim > 0 && rotary_dim % 2 == 0 &&
                rotary_dim <= head_dim && num_axes >= 1,
            MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(position_bytes == 4 || position_bytes == 8, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(head_dim <= kMaxHeadDim && num_axes <= kMaxAxes && num_q_heads <= 1024 && num_k_heads <= 1024, MOE_ERR_UNSUPPORTED_SHAPE);
  MOE_CHECK(num_axes == 1 || ld_positions >= N || ld_positions == 0, MOE_ERR_INVALID_ARGUMENT);  // 0: one row for every axis
  const int64_t wq = static_cast<int64_t>(num_q_heads) * head_dim, wk = static_cast<int64_t>(num_k_heads) * head_dim;
  MOE_CHECK(ld_q >= wq && ld_q_out >= wq && (num_k_heads == 0 || (ld_k >= wk && ld_k_out >= wk)), MOE_ERR_INVALID_ARGUMENT);
  if (N == 0) return MOE_OK;
  MOE_CHECK(q && q_out && positions && inv_freq && (num_k_heads == 0 || (k && k_out)), MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(num_axes == 1 || axes, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(q_out) |
              reinterpret_cast<uintptr_t>(k_out)) & 1) == 0 &&
                reinterpret_cast<uintptr_t>(positions) % position_bytes == 0 && reinterpret_cast<uintptr_t>(inv_freq) % 8 == 0,
            MOE_ERR_MISALIGNED);
  const uint16_t* in[2] = {q, k};
  uint16_t* out[2] = {q_out, k_out};
  const int64_t ld_in[2] = {ld_q, ld_k}, ld_out[2] = {ld_q_out, ld_k_out}, width[2] = {wq, wk};
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 2; ++j) {
      if (i == j && in[i] == out[i] && (ld_in[i] == ld_out[i] || N == 1)) continue;  // in place
      MOE_CHECK(!rows_overlap(out[i], ld_out[i], width[i], in[j], ld_in[j], width[j], N), MOE_ERR_OVERLAP);
    }
    const size_t bytes = width[i] ? (static_cast<size_t>(N - 1) * ld_out[i] + width[i]) * 2 : 0;
    const size_t pos_bytes = (static_cast<size_t>(num_axes - 1) * ld_positions + N) * position_bytes;
    MOE_CHECK(!overlaps(out[i], bytes, positions, pos_bytes) && !overlaps(out[i], bytes, inv_freq, rotary_dim / 2 * sizeof(double)) &&
                  !overlaps(out[i], bytes, axes, rotary_dim / 2),
              MOE_ERR_OVERLAP);
  }
  MOE_CHECK(!rows_overlap(q_out, ld_q_out, wq, k_out, ld_k_out, wk, N), MOE_ERR_OVERLAP);
  RotaryArgs a = {};
  for (int i = 0; i < 2; ++i) {
    a.in[i] = in[i], a.out[i] = out[i], a.ld_in[i] = ld_in[i], a.ld_out[i] = ld_out[i];
    a.copy[i] = in[i] != out[i];
  }
  a.heads[0] = num_q_heads, a.heads[1] = num_k_heads;
  a.pos = positions, a.inv_freq = inv_freq, a.axes = axes, a.status = dev_status;
  a.ld_pos = ld_positions, a.N = N, a.dim = head_dim, a.half = rotary_dim / 2, a.num_axes = num_axes;
  a.pos64 = position_bytes == 8, a.adjacent = adjacent != 0;
  cudaStream_t s = as_stream(stream);
  const bool whole = rotary_dim % 16 == 0 && head_dim % 8 == 0 && ((ld_q | ld_q_out | ld_k | ld_k_out) & 7) == 0 &&
                     aligned16(q) && aligned16(k) && aligned16(q_out) && aligned16(k_out);
  if (!whole) return launch_pdl(rotary_odd_kernel, dim3(static_cast<unsigned>(N)), dim3(256), 0, s, a);
  return adjacent ? launch_rotary<true>(a, s) : launch_rotary<false>(a, s);
}
