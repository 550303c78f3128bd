// Products of E4M3 activations with an E4M3 matrix that has one FP32 scale per 128 x 128 block.
//
//   y[m, n] = act(sum_b xs[m, b] * ws[n / 128, b] * sum_{k in block b} x[m, k] * w[n, k])
//
// The products of a block b of K run on tcgen05 (kind::f8f6f4, FP32 sums in TMEM). Its scales are any FP32
// numbers whose product is a normal one or 0 (to carry those where it is not costs 2 to 6 % of every call's time), so that its
// sums leave TMEM every 128 of K: warps of sums read them into registers, free the accumulator at
// once, and add them times their scale to the tile's sums there, while the tensor core makes the next blocks'.
//
// What bounds it. Few tokens: the bytes of w, and a chain of launch, first load, sums and the slices' meeting of about
// 4 us. Many: the way of an accumulator from MMA to MMA. All of TMEM is accumulators, 512 columns; from a block's MMAs over
// commit, wait, read-out and release to the next ones into the same columns takes 1200 to 1500 cycles where 1024 would
// keep the tensor core busy. What shortened that way, 8192 x 7168 x 7168: a relaxed arrival where a releasing one waited
// for the scales' loads (780 -> 460 us); halves of the columns as accumulators of their own and a warp of MMAs for each of
// the four (-> 440); scales through shared memory by a warp of their own, read before the wait; copies by three warps; the
// loads' barrier waited for before the accumulator's, whole warps that elect a lane for the MMAs (-> 332); packed
// FP32 multiply-adds (-> 314); the last 64 columns' reads under the first ones' additions (-> 307); results stored by
// whole 32-byte sectors (-> 290), packed before any of them is (-> 282).
//
// Measured (us, in a graph): 4 x 2048 x 512 3.3, 16 x 4096 x 4096 6.7, 48 x 4096 x 7168 with SwiGLU 9.0, 256 x 4096 x 4096
// 12.3, 333 x 7001 x 2000 13.4, 512 x 4096 x 4096 14.8, 1024 x 4096 x 4096 20 (1.7 PFLOP/s), 4096 x 4096 x 7168 with SwiGLU
// 94 (2.55), 8192 x 7168 x 7168 282 (3.0; one after another for seconds the card's power limit lowers the clock to 1.7 GHz,
// and it takes 320 to 330). With nothing read out, loaded or varied (a timing copy), the
// MMAs alone reach 3.8 PFLOP/s at 4096 x 4096 x 16384, whose tiles fill 84 % of the pairs' turns.
#include <math.h>

#include <atomic>

#include "cluster.cuh"
#include "common.cuh"
#include "host_util.h"
#include "layout.h"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kGroup = MOE_FP8_GROUP;
// 2^x to 2^-22 of itself, 0 where that is no normal number; 1 / x to 2^-23 for 1 <= x <= 2
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two values an instruction
struct Two {
  float x, y;
};
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// g / (1 + e^-g) by e = e^-|g|, which cannot overflow: the square of a power of two, whose exponent's rounding is made good, so
// that e is right where it is no normal number any more. Within 2^-19 of itself down to g = -87, and to 2^-148 |g| below, far
// under the rounding to BF16 that follows. 4096 x 4096 x 1024 with SwiGLU: 24.2 us; with expf and an IEEE quotient 35, one value an
// instruction 24.9.
__device__ __forceinline__ Two silu(Two g) {
  constexpr float kHigh = 0.5f * 1.44269502f, kLow = 0.5f * 1.92596299e-8f;  // log2(e) / 2 as two floats
  const Two a = {fminf(fabsf(g.x), 256.0f), fminf(fabsf(g.y), 256.0f)};      // an infinity would leave no rest of its own
  const Two p = mul2(a, {-kHigh, -kHigh}), rest = fma2(a, {kLow, kLow}, fma2(a, {kHigh, kHigh}, p));
  Two h = {exp2_approx(p.x), exp2_approx(p.y)};
  h = fma2(h, mul2(rest, {-0.693147181f, -0.693147181f}), h);
  const Two ge = mul2(g, mul2(h, h)), d = fma2(h, h, {1.0f, 1.0f});
  return mul2({g.x < 0.0f ? ge.x : g.x, g.y < 0.0f ? ge.y : g.y}, {rcp_approx(d.x), rcp_approx(d.y)});
}
__device__ __forceinline__ float silu(float g) { return silu(Two{g, g}).x; }
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

// mbar_wait that looks at the clock and the flag once in a while only: they cost more than the wait
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status, uint64_t limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, status, limit_ns);
}

// whether the phase is over, without waiting: the answer's latency is covered by what is done before it is used
__device__ __forceinline__ uint32_t mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok;
}

// wait of a block that ends: short, and it gives up without a word
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > 200000000ull) return;
}

// Instruction descriptor of tcgen05.mma.kind::f8f6f4: E4M3 A and B, K-major both, FP32 accumulation, M x N (x K = 32).
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4)                        // D format: FP32
         | ((uint32_t)(N >> 3) << 17)     // N / 8
         | ((uint32_t)(M >> 4) << 24);    // M / 16
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void store_cluster4(uint32_t at, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

__host__ __device__ constexpr bool is_gated(int act) { return act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU; }

// a thread's N results from its sums; of the gated kinds from N of gate and, behind them, N of up
template <int ACT, int N>
__device__ __forceinline__ void activate_all(float* v) {
  if constexpr (ACT == MOE_ACT_SWIGLU || ACT == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      Two y = silu(Two{v[i], v[i + 1]});
      if constexpr (ACT == MOE_ACT_SWIGLU) y = mul2(y, {v[N + i], v[N + i + 1]});
      v[i] = y.x, v[i + 1] = y.y;
    }
  } else if constexpr (ACT != MOE_ACT_IDENTITY) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate(ACT, v[i], is_gated(ACT) ? v[N + i] : 0.0f);
  }
}

struct Fp8Args {
  CUtensorMap tmap_x, tmap_w;
  const float* xs;
  const float* ws;
  uint16_t* out;
  int32_t* status;
  uint64_t wait_ns;
  int M, N, K, groups;
  int xs_step, xs_ld;  // per 128 columns and per row: 1 and groups, or 0 and 1
  int cols;            // of out: N, or N / 2
  int slices, m_tiles, x_rows, wide, stages, stage_bytes;
  int withhold;        // test build: the first block of K of a tile's first copies never comes
};

// a += t * s for two values at once
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t t0, uint32_t t1, float s) {
  asm("{\n .reg .b64 a, t, f;\n mov.b64 a, {%0, %1};\n mov.b64 t, {%2, %3};\n mov.b64 f, {%4, %4};\n"
      " fma.rn.f32x2 a, t, f, a;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "r"(t0), "r"(t1), "f"(s));
}

// one lane of a whole warp
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(yes));
  return yes != 0;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// 32 bytes at a multiple of 32
__device__ __forceinline__ void store_sector(uint16_t* to, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// as arrive_cluster() does, in this block
__device__ __forceinline__ void arrive_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

constexpr int kRows = 128, kCols = 128;   // of a block's tile
constexpr int kMaxStages = 8, kBufs = 4;
constexpr int kOperand = 128 * 128;       // bytes of a stage's w (and of its x, where rows are 128)
constexpr int kMaxSlices = 8;
constexpr int kSumLd = kCols + 4;         // of a row of sums in shared memory: no bank conflicts
constexpr int kThreads = 384;             // warps: copies, two of MMAs, scales, eight of sums
constexpr int kScaleRun = 8;              // blocks of K whose scales are fetched together: a sector of x_scale
constexpr int kScaleBytes = 2 * kScaleRun * (128 + 2) * 4;
constexpr int kBarBytes = 256;
constexpr int kTileSmem = 227 * 1024;     // at most

// The scales of kScaleRun blocks of K at a time, turned so that the threads of a row's sums read them side by
// side (read from global memory by those threads, one value a block of K, they cost half of the kernel's time):
// x_ring [2][kScaleRun][128 rows], w_ring [2][kScaleRun][2]. One whole warp; `rows` of the tile's rows from m0 on.
__device__ __forceinline__ void fetch_scales(const Fp8Args& a, int run, int kb, int64_t m0, int rows, const float* ws, const float* ws2,
                                             float* x_ring, float* w_ring, int lane) {
  float* const x_to = x_ring + (run & 1) * kScaleRun * 128;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (32 * j >= rows) break;
    const float* const xs = a.xs + (m0 + min(32 * j + lane, rows - 1)) * a.xs_ld;
    float v[kScaleRun];
#pragma unroll
    for (int i = 0; i < kScaleRun; ++i) v[i] = __ldg(xs + min(kb + i, a.groups - 1) * a.xs_step);
#pragma unroll
    for (int i = 0; i < kScaleRun; ++i) x_to[i * 128 + 32 * j + lane] = v[i];
  }
  if (lane < 2 * kScaleRun)
    w_ring[(run & 1) * 2 * kScaleRun + lane] = __ldg((lane & 1 ? ws2 : ws) + min(kb + (lane >> 1), a.groups - 1));
}

// N neighbouring values, a pair to a word, to any place in a row: `some` of them, the others lie behind the row. The ones
// before the first whole sector go in pieces of 1, 2, 4 and 8 values, each at a multiple of its size, and what follows
// moves up by as many; so do the ones behind the last. (Through shared memory, value by value in row order, 2048 x 129021 x
// 512 took twice the time of 2048 x 129024 x 512.)
template <int N>
__device__ __forceinline__ void store_odd(uint32_t (&w)[N / 2], uint16_t* to, int some) {
  if (some < 16) {
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < some) to[i] = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    return;
  }
  const uint32_t head = (0 - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to) >> 1)) & 15;
  const auto up = [&](int words) {  // moves all of them by `words`
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = i + words < N / 2 ? w[i + words] : 0;
  };
  if (head & 1) *to = static_cast<uint16_t>(w[0]);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = __funnelshift_r(w[i], i + 1 < N / 2 ? w[i + 1] : 0, (head & 1) * 16);
  to += head & 1;
  if (head & 2) {
    *reinterpret_cast<uint32_t*>(to) = w[0];
    up(1);
  }
  to += head & 2;
  if (head & 4) {
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    up(2);
  }
  to += head & 4;
  if (head & 8) {
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    up(4);
  }
  to += head & 8;
  const int left = some - static_cast<int>(head), whole = left >> 4;
  uint32_t z[8];  // what is behind the whole sectors
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = 0;
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    if (i < whole) store_sector(to + 16 * i, w + 8 * i);
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = i == whole ? w[8 * i + e] : z[e];
  }
  to += 16 * whole;
  if (left & 8) {
    *reinterpret_cast<uint4*>(to) = make_uint4(z[0], z[1], z[2], z[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = z[e + 4];
  }
  to += left & 8;
  if (left & 4) {
    *reinterpret_cast<uint2*>(to) = make_uint2(z[0], z[1]);
    z[0] = z[2], z[1] = z[3];
  }
  to += left & 4;
  if (left & 2) {
    *reinterpret_cast<uint32_t*>(to) = z[0];
    z[0] = z[1];
  }
  to += left & 2;
  if (left & 1) *to = static_cast<uint16_t>(z[0]);
}

// N values of a thread's row, from column c0 on, to out
template <int N, bool GATED>
__device__ __forceinline__ void store_row(const Fp8Args& a, const float* v, int64_t row, int c0) {
  if (row >= a.M || c0 >= a.cols) return;
  uint16_t* const to = a.out + row * a.cols + c0;
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = bf16x2(v[2 * i], v[2 * i + 1]);
  if (a.wide == 2) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
      if (c0 + 16 * i < a.cols) store_sector(to + 16 * i, w + 8 * i);
  } else if (GATED || a.wide) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      if (c0 + 8 * i < a.cols) *reinterpret_cast<uint4*>(to + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  } else {
    store_odd<N>(w, to, min(N, a.cols - c0));
  }
}

// One 128 x 128 tile of the product, or one slice of its K. The blocks of a cluster are a tile's slices: their sums meet in
// distributed shared memory in the slices' order, so that results repeat.
template <int ACT>
__global__ void __launch_bounds__(kThreads, 1) linear_fp8_kernel(const __grid_constant__ Fp8Args a) {
  constexpr bool GATED = is_gated(ACT);
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  float* const x_ring = reinterpret_cast<float*>(smem + a.stages * a.stage_bytes);
  float* const w_ring = x_ring + 2 * kScaleRun * 128;
  uint64_t* const full = reinterpret_cast<uint64_t*>(w_ring + 2 * kScaleRun * 2);
  uint64_t* const done = full + kMaxStages;    // a stage's products are summed
  uint64_t* const taken = done + kMaxStages;   // ... and read
  uint64_t* const scales = taken + kBufs;      // a run of scales is there
  uint64_t* const scales_free = scales + 2;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(scales_free + 2);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* const sums = reinterpret_cast<float*>(smem + a.stages * a.stage_bytes + kScaleBytes + kBarBytes);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int slice = blockIdx.x % a.slices, tile = blockIdx.x / a.slices;
  const int m0 = tile % a.m_tiles * kRows;
  constexpr int kOut = GATED ? kCols / 2 : kCols;  // columns of out
  const int n0 = tile / a.m_tiles * kOut;
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.groups) * slice / a.slices);
  const int n = static_cast<int>(static_cast<int64_t>(a.groups) * (slice + 1) / a.slices) - kb0;  // blocks of K
  const int rows = min(kRows, a.M - m0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1), mbar_init(&done[i], 1);
    for (int i = 0; i < kBufs; ++i) mbar_init(&taken[i], 8);
    for (int i = 0; i < 2; ++i) mbar_init(&scales[i], 1), mbar_init(&scales_free[i], 8);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&a.tmap_x);
    prefetch_tensormap(&a.tmap_w);
  }
  __syncwarp();
  if (warp == 2) {
    tmem_alloc(tmem_slot, kBufs * kCols);
    tmem_relinquish();
  }
  __syncwarp();
  if (a.slices > 1) cluster_arrive();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (lane == 0) {  // (the whole warp waiting, one of its lanes issuing, takes 5 to 10 % longer)
      const uint32_t bytes = a.x_rows * 128 + kOperand;
      int stage = 0, phase = 0, issued = 0;
      for (int i = 0; i < n; ++i) {
        if (!wait_for(&done[stage], phase ^ 1, abort_flag, a.status, a.wait_ns)) break;
        if (!(a.withhold && i == 0)) {
          uint8_t* const st = smem + stage * a.stage_bytes;
          const int k = (kb0 + i) * 128;
          mbar_arrive_expect_tx(&full[stage], bytes);
          tma_load_2d(st, &a.tmap_w, k, n0, &full[stage]);
          if (GATED) tma_load_2d(st + kOperand / 2, &a.tmap_w, k, a.cols + n0, &full[stage]);
          tma_load_2d(st + kOperand, &a.tmap_x, k, m0, &full[stage]);
        }
        ++issued;
        if (++stage == a.stages) stage = 0, phase ^= 1;
      }
      // what was issued lands before the block ends, even if nothing waited for it
      for (int i = max(a.withhold ? 1 : 0, issued - a.stages); i < issued; ++i) mbar_drain(&full[i % a.stages], i / a.stages & 1);
    }
  } else if (warp < 3) {
    // two warps take the blocks of K by turns: what one costs them in waits is more than it costs the tensor core
    const uint64_t w_desc = sdesc_kmajor_sw128(smem_u32(smem)), x_desc = sdesc_kmajor_sw128(smem_u32(smem) + kOperand);
    uint64_t* last = nullptr;
    int last_phase = 0, stage = warp - 1, phase = 0;
    for (int i = warp - 1; i < n; i += 2) {
      const int buf = i % kBufs;
      const bool ok = wait_for(&full[stage], phase, abort_flag, a.status, a.wait_ns) &&
                      wait_for(&taken[buf], (i / kBufs & 1) ^ 1, abort_flag, a.status, a.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      last = &done[stage], last_phase = phase;
      if (elect_one()) {
        const uint64_t at = static_cast<uint64_t>(stage * (a.stage_bytes >> 4));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_e4m3(tmem + buf * kCols, x_desc + at + 2 * k, w_desc + at + 2 * k, idesc_e4m3(kRows, kCols), k != 0);
        tc_commit(last);
      }
      __syncwarp();
      stage += 2;
      if (stage >= a.stages) stage -= a.stages, phase ^= 1;
    }
    if (last) mbar_drain(last, last_phase);  // no MMA runs when TMEM is released
  } else if (warp == 3) {
    const float* const ws = a.ws + static_cast<int64_t>(n0 / kGroup) * a.groups;
    const float* const ws2 = GATED ? a.ws + static_cast<int64_t>((a.cols + n0) / kGroup) * a.groups : ws;
    for (int i = 0, run = 0; i < n; i += kScaleRun, ++run) {
      if (!__all_sync(0xffffffffu, wait_for(&scales_free[run & 1], ((run >> 1) & 1) ^ 1, abort_flag, a.status, a.wait_ns))) break;
      fetch_scales(a, run, kb0 + i, m0, rows, ws, ws2, x_ring, w_ring, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&scales[run & 1]);
    }
  } else {
    const int quarter = warp & 3, half = (warp - 4) >> 2;  // of the tile's rows and columns
    const int r = quarter * 32 + lane;
    const bool some = quarter * 32 < rows;                 // of the warp's rows there are any
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * (GATED ? 32 : 64);
    float acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
    int stage = 0, phase = 0, run = 0;
    for (int i = 0; i < n; ++i) {
      bool ok = true;
      if (i % kScaleRun == 0) ok = wait_for(&scales[run & 1], (run >> 1) & 1, abort_flag, a.status, a.wait_ns);
      const int in = (run & 1) * kScaleRun + i % kScaleRun, buf = i % kBufs;
      const float x = x_ring[in * 128 + r];
      const float s0 = x * w_ring[2 * in], s1 = GATED ? x * w_ring[2 * in + 1] : s0;
      ok = ok && wait_for(&done[stage], phase, abort_flag, a.status, a.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint32_t t[64];
      if (some) {
        tc_fence_after();
        tmem_ld32_issue(at + buf * kCols, t);
        tmem_ld32_issue(at + buf * kCols + (GATED ? 64 : 32), t + 32);
        tmem_wait_ld<64>(t);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        arrive_relaxed(&taken[buf]);
        if (i % kScaleRun == kScaleRun - 1) mbar_arrive(&scales_free[run & 1]);
      }
      if (some) {
#pragma unroll
        for (int c = 0; c < 64; c += 2) fma2(acc[c], acc[c + 1], t[c], t[c + 1], c < 32 ? s0 : s1);
      }
      if (i % kScaleRun == kScaleRun - 1) ++run;
      if (++stage == a.stages) stage = 0, phase ^= 1;
    }
    if (a.slices == 1) {
      activate_all<ACT, GATED ? 32 : 64>(acc);
      store_row<GATED ? 32 : 64, GATED>(a, acc, static_cast<int64_t>(m0) + r, n0 + half * (GATED ? 32 : 64));
    } else {
      cluster_wait();  // every block of the cluster runs
      // The rows of the tile are dealt out to its slices, which add up their rows' sums: row r to block r / per.
      const int per = (rows + a.slices - 1) / a.slices;
      if (r < rows) {
        const uint32_t there = cluster_address(sums + (slice * per + r % per) * kSumLd + half * (GATED ? 32 : 64), r / per);
#pragma unroll
        for (int i = 0; i < 64; i += 4)
          store_cluster4(there + (GATED && i >= 32 ? i + 32 : i) * 4, acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      }
    }
  }
  __syncwarp();
  if (a.slices > 1) {
    if (warp < 4) cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, kBufs * kCols);
  }
  if (a.slices == 1) return;
  const int per = (rows + a.slices - 1) / a.slices, first = slice * per, mine = min(per, rows - first);
  if (!GATED && !a.wide) {  // columns side by side to threads side by side
    for (int i = threadIdx.x; i < mine * kOut; i += kThreads) {
      const int r = i / kOut, c = i % kOut;
      if (n0 + c >= a.cols) continue;
      float v = 0.0f;
      for (int s = 0; s < a.slices; ++s) v += sums[(s * per + r) * kSumLd + c];
      a.out[static_cast<int64_t>(m0 + first + r) * a.cols + n0 + c] = __bfloat16_as_ushort(__float2bfloat16_rn(activate(ACT, v, 0.0f)));
    }
    return;
  }
  for (int i = threadIdx.x; i < mine * (kOut / 4); i += kThreads) {  // four columns each
    const int r = i / (kOut / 4), c = i % (kOut / 4) * 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < a.slices; ++s) {
      const float* const from = sums + (s * per + r) * kSumLd + c;
      const float4 p = *reinterpret_cast<const float4*>(from);
      v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
      if (GATED) {
        const float4 q = *reinterpret_cast<const float4*>(from + kOut);
        u[0] += q.x, u[1] += q.y, u[2] += q.z, u[3] += q.w;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = activate(ACT, v[e], u[e]);
    uint16_t* const to = a.out + static_cast<int64_t>(m0 + first + r) * a.cols + n0 + c;
    if (n0 + c < a.cols) *reinterpret_cast<uint2*>(to) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
  }
}

// rows of out: 2 whole 32-byte sectors, 1 whole 16-byte pieces, 0 neither
int row_pieces(const Fp8Args& a) {
  return a.cols % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 32 == 0 ? 2 : a.cols % 8 == 0;
}

// How many clusters of `size` blocks of a kernel run at once on the current device: looked up once for each size.
moe_status_t resident(const void* kern, int size, int threads, int smem, std::atomic<int>* known, int& clusters) {
  int dev = 0;
  MOE_CUDA(cudaGetDevice(&dev));
  std::atomic<int>& here = known[(dev & 63) * kMaxSlices + size - 1];
  clusters = here.load(std::memory_order_relaxed);
  if (clusters > 0) return MOE_OK;
  MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size * num_sms());
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MOE_CUDA(cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg));
  if (clusters < 1) return MOE_ERR_CUDA;
  here.store(clusters, std::memory_order_relaxed);
  return MOE_OK;
}

// Single blocks: in how many slices K is cut, by the least estimated time. A wave of blocks takes 3 us and 0.26 us a block of
// K, up to 0.10 more where all SMs load 128 rows of x; the slices' meeting 0.4 us and 3 more for 128 rows. The clusters
// that run at once are fewer than their blocks would let one think (of eight blocks 15 on 152 SMs, not 19).
moe_status_t cut_tiles(int M, int groups, int64_t tiles, int& slices, double& time) {
  static std::atomic<int> known[64 * kMaxSlices];
  const double rows = (M < kRows ? M : kRows) / static_cast<double>(kRows);
  time = -1.0;
  for (int n = 1; n <= kMaxSlices && (n == 1 || groups >= 2 * n); ++n) {
    int clusters = 0;
    const moe_status_t st = resident(reinterpret_cast<const void*>(linear_fp8_kernel<MOE_ACT_IDENTITY>), n, kThreads, kTileSmem, known, clusters);
    if (st != MOE_OK) return st;
    const double waves = ceil(static_cast<double>(tiles) / clusters), busy = fmin(1.0, static_cast<double>(tiles) / clusters);
    const double t = waves * (3.0 + ceil(static_cast<double>(groups) / n) * (0.26 + 0.10 * busy * rows)) + (n > 1 ? 0.4 + 3.0 * rows : 0.0);
    if (time < 0.0 || t < time) time = t, slices = n;
  }
  return MOE_OK;
}

template <int ACT>
moe_status_t launch_tiles(Fp8Args a, const void* x, int64_t ld_x, const void* w, cudaStream_t s) {
  constexpr int kOut = is_gated(ACT) ? kCols / 2 : kCols;
  a.m_tiles = (a.M - 1) / kRows + 1;
  a.x_rows = a.M < kRows ? (a.M + 7) / 8 * 8 : kRows;
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * ((a.cols - 1) / kOut + 1);
  double time = 0.0;
  const moe_status_t cut = cut_tiles(a.M, a.groups, tiles, a.slices, time);
  if (cut != MOE_OK) return cut;
  MOE_CHECK(tiles * a.slices <= INT32_MAX, MOE_ERR_UNSUPPORTED_SHAPE);
  a.wide = row_pieces(a);
  const int held = a.M < kRows ? a.M : kRows;
  int sums = a.slices > 1 ? (held + a.slices - 1) / a.slices * a.slices * kSumLd * 4 : 0;
  // The MMA reads 128 rows of x where fewer were loaded (what it makes of the others is not used): they lie in the
  // following stages, and after the last one in what follows the stages.
  if (sums < kOperand - kScaleBytes - kBarBytes) sums = kOperand - kScaleBytes - kBarBytes;
  a.stage_bytes = kOperand + (a.x_rows * 128 + 1023) / 1024 * 1024;
  const int rest = 1024 + kScaleBytes + kBarBytes + sums;
  a.stages = (kTileSmem - rest) / a.stage_bytes / 2 * 2;  // even: two warps take them by turns
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const int smem = rest + a.stages * a.stage_bytes;
  if (!encode_rows(&a.tmap_x, x, a.K, a.M, ld_x, a.x_rows) || !encode_rows(&a.tmap_w, w, a.K, a.N, a.K, kOut)) return MOE_ERR_CUDA;
  const auto kern = linear_fp8_kernel<ACT>;
  MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem));
  return launch_clusters(kern, a.slices, dim3(static_cast<unsigned>(tiles * a.slices)), dim3(kThreads), smem, s, a);
}

// ---------------------------------------------------------------------------------------------------
// Large products: a pair of blocks (two SMs) to a tile of 256 x 256, the pairs staying for tile after tile.
// ---------------------------------------------------------------------------------------------------
__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on both blocks' `bar` once every MMA issued so far by this thread has completed
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// a load into this block's shared memory that completes on a barrier of the pair's first block
__device__ __forceinline__ void tma_load_pair(void* smem_dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(smem_dst)), "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Sums were read (tcgen05.wait::ld came before) and nothing else is told: with a release the arrival would wait for every
// load of the thread that is under way.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 256 x 256 columns to two SMs, since each then loads 32 KB a block of K and not 48: at the tensor core's rate one SM's tiles
// of 128 x 256 would want 27 TB/s from L2.
constexpr int kPairStages = 6;
static_assert(kPairStages % 6 == 0, "three warps of copies and two buffers of sums take the stages by turns");
constexpr int kPairCols = 256;         // of a tile, and of one accumulator
constexpr int kPairThreads = 512;      // warps: three of copies, four of MMAs, scales, eight of sums
constexpr int kPairRegs = 208, kPairRegsOther = 48, kPairRegsAtLaunch = 128;
static_assert(256 * kPairRegs + 256 * kPairRegsOther <= kPairThreads * kPairRegsAtLaunch, "the raise draws on the launch's registers");
constexpr int kPairSmem = 1024 + kPairStages * 2 * kOperand + kScaleBytes + kBarBytes;
constexpr int kPairGroup = 8;          // row tiles that follow one another before the next column tile

template <int ACT>
__global__ void __launch_bounds__(kPairThreads, 1) linear_fp8_pair_kernel(const __grid_constant__ Fp8Args a) {
  constexpr bool GATED = is_gated(ACT);
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  float* const x_ring = reinterpret_cast<float*>(smem + kPairStages * 2 * kOperand);  // [2][kScaleRun][128 rows]
  float* const w_ring = x_ring + 2 * kScaleRun * 128;                        // [2][kScaleRun][halves, or gate and up]
  uint64_t* const full = reinterpret_cast<uint64_t*>(w_ring + 2 * kScaleRun * 2);
  uint64_t* const done = full + kPairStages;   // a stage's products are summed, one for each half of its columns
  uint64_t* const taken = done + 2 * kPairStages;  // ... and read
  uint64_t* const scales = taken + 4;              // a run of scales is there
  uint64_t* const scales_free = scales + 2;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(scales_free + 2);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;  // in the pair: rows 0-127 and columns 0-127 of w, or the others
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  constexpr int kOut = GATED ? kPairCols / 2 : kPairCols;
  const int n_tiles = (a.cols - 1) / kOut + 1, tiles = a.m_tiles * n_tiles;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) mbar_init(&full[i], 1), mbar_init(&done[2 * i], 1), mbar_init(&done[2 * i + 1], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&taken[i], 8);
    for (int i = 0; i < 2; ++i) mbar_init(&scales[i], 1), mbar_init(&scales_free[i], 8);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&a.tmap_x);
    prefetch_tensormap(&a.tmap_w);
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // both blocks' barriers and TMEM are there
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  // tile t: groups of kPairGroup row tiles, column by column
  const auto place = [&](int t, int& m0, int& n0) {
    const int group = t / (kPairGroup * n_tiles), first = group * kPairGroup, in = t - group * kPairGroup * n_tiles;
    const int high = min(kPairGroup, a.m_tiles - first);
    m0 = (first + in % high) * 256;
    n0 = in / high * kOut;
  };

  if (warp < 8) {
    setmaxnreg_dec<kPairRegsOther>();
    if (warp == 0 || warp > 5) {
      // Three warps take the blocks of K by turns: the wait for a stage and its three copies cost one more time
      // than the MMAs leave it.
      const int all = (tiles - pair + pairs - 1) / pairs * a.groups;  // blocks of K of this pair's tiles
      int t = pair, kb = warp == 0 ? 0 : warp - 5, stage = kb, phase = 0, last = -1, m0 = 0, n0 = 0;
      bool ok = true;
      for (int i = kb; i < all; i += 3) {
        while (kb >= a.groups) kb -= a.groups, t += pairs;
        if (kb < 3) place(t, m0, n0);
        const int y_x = m0 + rank * 128, y_w = n0 + rank * (GATED ? a.cols : 64);
        ok = wait_for(&done[2 * stage], phase ^ 1, abort_flag, a.status, a.wait_ns) &&
             wait_for(&done[2 * stage + 1], phase ^ 1, abort_flag, a.status, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (!(a.withhold && i == 0) && elect_one()) {
          uint8_t* const st = smem + stage * 2 * kOperand;
          const uint32_t bar = cluster_address(&full[stage], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 4 * kOperand);  // both blocks' loads
          tma_load_pair(st, &a.tmap_x, kb * 128, y_x, bar);
          tma_load_pair(st + kOperand, &a.tmap_w, kb * 128, y_w, bar);
          tma_load_pair(st + kOperand + kOperand / 2, &a.tmap_w, kb * 128, y_w + (GATED ? 64 : 128), bar);
        }
        __syncwarp();
        last = i;
        kb += 3, stage += 3;
        if (stage >= kPairStages) stage -= kPairStages, phase ^= 1;
      }
      // loads land before the pair ends, even if nothing waited for them
      if (rank == 0) {
        for (int i = last >= 3 ? last - 3 : last; i >= 0 && i <= last; i += 3)
          if (!(a.withhold && i == 0)) mbar_drain(&full[i % kPairStages], i / kPairStages & 1);
      } else if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
      }
    } else if (warp <= 4) {
      if (rank == 0) {
        // One warp for each of the four accumulators, so that their waits and commits, which take longer than the MMAs
        // take the tensor core, go on side by side.
        const int buf = (warp - 1) & 1, half = (warp - 1) >> 1;
        const int all = (tiles - pair + pairs - 1) / pairs * a.groups;  // blocks of K of this pair's tiles
        const uint32_t to = tmem + buf * kPairCols + half * 128;
        const uint64_t x_desc = sdesc_kmajor_sw128(smem_u32(smem));
        const uint64_t w_desc = sdesc_kmajor_sw128(smem_u32(smem) + kOperand + half * (kOperand / 2));
        uint64_t* last = nullptr;
        int last_phase = 0, stage = buf, phase = 0;
        for (int i = buf; i < all; i += 2) {
          // the loads are ahead of the sums: their wait comes first, off the way from sums read to MMAs issued
          const bool ok = wait_for(&full[stage], phase, abort_flag, a.status, a.wait_ns) &&
                          wait_for(&taken[2 * buf + half], ((i >> 1) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          last = &done[2 * stage + half], last_phase = phase;
          if (elect_one()) {
            const uint64_t at = static_cast<uint64_t>(stage * (2 * kOperand >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_e4m3_pair(to, x_desc + at + 2 * k, w_desc + at + 2 * k, idesc_e4m3(256, 128), k != 0);
            tc_commit_pair(last);
          }
          __syncwarp();
          stage += 2;
          if (stage >= kPairStages) stage -= kPairStages, phase ^= 1;
        }
        if (last) mbar_drain(last, last_phase);
      }
    } else if (warp == 5) {
      int run = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs) {
        int m0, n0;
        place(t, m0, n0);
        const int row0 = min(m0 + rank * 128, a.M - 1);
        const int blocks = (a.N - 1) / kGroup;  // a tile's second half may lie behind the matrix: its sums are not stored
        const float* const ws = a.ws + static_cast<int64_t>(n0 / kGroup) * a.groups;
        const float* const ws2 = a.ws + static_cast<int64_t>(min((GATED ? a.cols + n0 : n0 + 128) / kGroup, blocks)) * a.groups;
        for (int kb = 0; kb < a.groups; kb += kScaleRun, ++run) {
          ok = __all_sync(0xffffffffu, wait_for(&scales_free[run & 1], ((run >> 1) & 1) ^ 1, abort_flag, a.status, a.wait_ns));
          if (!ok) break;
          fetch_scales(a, run, kb, row0, max(1, min(128, a.M - row0)), ws, ws2, x_ring, w_ring, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&scales[run & 1]);
        }
      }
    }
  } else {
    setmaxnreg_inc<kPairRegs>();
    // a warp has 32 rows and a half's 128 columns; gated: 64 of gate and the same 64 of up
    const int quarter = warp & 3, half = (warp - 8) >> 2;
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    const uint32_t free_bar = cluster_address(&taken[half], 0);
    int buf = 0, stage = 0, phase = 0, run = 0;
    uint32_t here = 0;  // the next sums were seen done
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
      for (int kb = 0; kb < a.groups; ++kb) {
        if (kb % kScaleRun == 0)
          ok = __all_sync(0xffffffffu, wait_for(&scales[run & 1], (run >> 1) & 1, abort_flag, a.status, a.wait_ns));
        const int in = (run & 1) * kScaleRun + kb % kScaleRun;
        const float x = x_ring[in * 128 + quarter * 32 + lane];
        const float s0 = x * w_ring[2 * in + (GATED ? 0 : half)], s1 = GATED ? x * w_ring[2 * in + 1] : s0;
        if (!__all_sync(0xffffffffu, here))
          ok = ok && __all_sync(0xffffffffu, wait_for(&done[2 * stage + half], phase, abort_flag, a.status, a.wait_ns));
        if (!ok) break;
        tc_fence_after();
        const uint32_t from = at + buf * kPairCols;
        uint32_t v[2][32];
        const auto add = [&](int c) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) fma2(acc[32 * c + i], acc[32 * c + i + 1], v[c & 1][i], v[c & 1][i + 1], c < 2 ? s0 : s1);
        };
        tmem_ld32_issue(from, v[0]);
        tmem_ld32_issue(from + 32, v[1]);
        if (kb % kScaleRun == kScaleRun - 1 || kb == a.groups - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&scales_free[run & 1]);
          ++run;
        }
        tmem_wait_ld<64>(&v[0][0]);
        add(0);
        tmem_ld32_issue(from + 64, v[0]);
        add(1);
        tmem_ld32_issue(from + 96, v[1]);
        tmem_wait_ld<64>(&v[0][0]);  // all of it is in registers
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(free_bar + 2 * buf * 8);
        if (++stage == kPairStages) stage = 0, phase ^= 1;
        here = mbar_test(&done[2 * stage + half], phase);
        add(2);
        add(3);
        buf ^= 1;
      }
      if (!ok) break;
      int m0, n0;
      place(t, m0, n0);
      constexpr int kMine = GATED ? 64 : 128;            // columns of out
      const int c0 = n0 + half * kMine;
      activate_all<ACT, kMine>(acc);
      store_row<kMine, GATED>(a, acc, static_cast<int64_t>(m0) + rank * 128 + quarter * 32 + lane, c0);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // neither block goes while the other may still reach into it
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// How many pairs run at once on the current device.
template <int ACT>
moe_status_t resident_pairs(int& pairs) {
  static std::atomic<int> known[64 * kMaxSlices];
  static std::atomic<bool> checked;
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa;
    MOE_CUDA(cudaFuncGetAttributes(&fa, linear_fp8_pair_kernel<ACT>));
    if (fa.numRegs < kPairRegsAtLaunch) return MOE_ERR_CUDA;  // the raise of the registers would wait forever
    checked.store(true, std::memory_order_relaxed);
  }
  return resident(reinterpret_cast<const void*>(linear_fp8_pair_kernel<ACT>), 2, kPairThreads, kPairSmem, known, pairs);
}

// Pairs, or single blocks: the one of less estimated time. A wave of pairs takes 0.46 us a block of K (for four times the
// rows and columns of a single block), 1.3 around it, and all of them 4 once.
moe_status_t use_pairs(int M, int cols, int groups, bool gated, bool& pairs) {
  const int out = gated ? 2 : 1;
  const auto tiles = [&](int side) { return (M + side - 1ll) / side * ((static_cast<int64_t>(cols) * out + side - 1) / side); };
  int slices = 1, at_once = 0;
  double one = 0.0;
  moe_status_t st = cut_tiles(M, groups, tiles(128), slices, one);
  if (st != MOE_OK) return st;
  st = resident_pairs<MOE_ACT_IDENTITY>(at_once);
  if (st != MOE_OK) return st;
  pairs = ceil(static_cast<double>(tiles(256)) / at_once) * (groups * 0.46 + 1.3) + 4.0 < one;
  return MOE_OK;
}

template <int ACT>
moe_status_t launch_pairs(Fp8Args a, const void* x, int64_t ld_x, const void* w, cudaStream_t s) {
  constexpr int kOut = is_gated(ACT) ? kPairCols / 2 : kPairCols;
  a.m_tiles = (a.M - 1) / 256 + 1;
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * ((a.cols - 1) / kOut + 1);
  MOE_CHECK(tiles <= INT32_MAX / 2, MOE_ERR_UNSUPPORTED_SHAPE);
  a.wide = row_pieces(a);
  if (!encode_rows(&a.tmap_x, x, a.K, a.M, ld_x, 128) || !encode_rows(&a.tmap_w, w, a.K, a.N, a.K, 64)) return MOE_ERR_CUDA;
  const auto kern = linear_fp8_pair_kernel<ACT>;
  MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem));
  int pairs = 0;
  const moe_status_t known = resident_pairs<ACT>(pairs);
  if (known != MOE_OK) return known;
  const unsigned grid = static_cast<unsigned>(tiles < pairs ? tiles : pairs);
  return launch_clusters(kern, 2, dim3(2 * grid), dim3(kPairThreads), kPairSmem, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

namespace moe {

moe_status_t linear_fp8(const uint8_t* x, int64_t ld_x, const float* x_scale, int32_t x_scale_mode, int32_t M, int32_t K,
                        const uint8_t* w, const float* w_scale, int32_t N, int32_t activation, uint16_t* out,
                        int32_t* dev_status, const TestOptions& topt, moe_stream_t stream) {
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
  Fp8Args a = {};
  a.xs = x_scale, a.ws = w_scale, a.out = out, a.status = dev_status, a.wait_ns = topt.wait_limit_ns;
  a.withhold = topt.withhold_release;
  a.M = M, a.N = N, a.K = K, a.groups = groups, a.cols = cols;
  a.xs_step = per_token ? 0 : 1, a.xs_ld = per_token ? 1 : groups;
  bool pairs = false;
  const moe_status_t st = use_pairs(M, cols, groups, gated, pairs);
  if (st != MOE_OK) return st;
  cudaStream_t s = as_stream(stream);
#define MOE_FP8_CASE(ACT) \
  case ACT: return pairs ? launch_pairs<ACT>(a, x, ld_x, w, s) : launch_tiles<ACT>(a, x, ld_x, w, s)
  switch (activation) {
    MOE_FP8_CASE(MOE_ACT_SWIGLU);
    MOE_FP8_CASE(MOE_ACT_RELU2);
    MOE_FP8_CASE(MOE_ACT_GEGLU);
    MOE_FP8_CASE(MOE_ACT_GELU);
    MOE_FP8_CASE(MOE_ACT_RELU);
    MOE_FP8_CASE(MOE_ACT_SILU);
    MOE_FP8_CASE(MOE_ACT_IDENTITY);
  }
#undef MOE_FP8_CASE
  return MOE_ERR_INVALID_ARGUMENT;
}

}  // namespace moe

extern "C" moe_status_t moe_linear_fp8(const uint8_t* x, int64_t ld_x, const float* x_scale, int32_t x_scale_mode,
                                       int32_t M, int32_t K, const uint8_t* w, const float* w_scale, int32_t N,
                                       int32_t activation, uint16_t* out, int32_t* dev_status, moe_stream_t stream) {
  return linear_fp8(x, ld_x, x_scale, x_scale_mode, M, K, w, w_scale, N, activation, out, dev_status, TestOptions(), stream);
}
