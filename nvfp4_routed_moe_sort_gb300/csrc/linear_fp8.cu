// Products of E4M3 activations with an E4M3 matrix that has one FP32 scale per 128 x 128 block.
//
//   y[m, n] = act(sum_b xs[m, b] * ws[n / 128, b] * sum_{k in block b} x[m, k] * w[n, k])
#include <math.h>

#include "cluster.cuh"
#include "common.cuh"
#include "host_util.h"
#include "tensor_map.h"

namespace moe {
namespace {

constexpr int kGroup = MOE_FP8_GROUP;
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

struct Fp8Args {
  CUtensorMap tmap_x, tmap_w;
  const float* xs;
  const float* ws;
  uint16_t* out;
  int32_t* status;
  uint64_t wait_ns;
  int M, N, K, groups, act;
  int xs_step, xs_ld;  // per 128 columns and per row: 1 and groups, or 0 and 1
  int cols;            // of out: N, or N / 2
  int slices, m_tiles, x_rows;
};

constexpr int kRows = 128, kCols = 128;   // of a block's tile
constexpr int kStages = 4, kBufs = 4;
constexpr int kOperand = 128 * 128;       // bytes of a stage's x, and of its w
constexpr int kMaxSlices = 8;
constexpr int kSumLd = kCols + 4;         // of a row of sums in shared memory: no bank conflicts
constexpr int kSumRows = kRows + kMaxSlices;
constexpr int kThreads = 320;             // warps: copies, MMA, eight of sums
constexpr int kTileSmem = 1024 + kStages * 2 * kOperand + kSumRows * kSumLd * 4 + 256;

// One 128 x 128 tile of the product, or one slice of its K. The blocks of a cluster are a tile's slices.
template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1) linear_fp8_kernel(const __grid_constant__ Fp8Args a) {
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  float* const sums = reinterpret_cast<float*>(smem + kStages * 2 * kOperand);
  uint64_t* const full = reinterpret_cast<uint64_t*>(sums + kSumRows * kSumLd);
  uint64_t* const empty = full + kStages;
  uint64_t* const done = empty + kStages;   // a buffer's block of K is summed
  uint64_t* const taken = done + kBufs;     // ... and read
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(taken + kBufs);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slice = blockIdx.x % a.slices, tile = blockIdx.x / a.slices;
  const int m0 = tile % a.m_tiles * kRows;
  constexpr int kOut = GATED ? kCols / 2 : kCols;  // columns of out
  const int n0 = tile / a.m_tiles * kOut;
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.groups) * slice / a.slices);
  const int kb1 = static_cast<int>(static_cast<int64_t>(a.groups) * (slice + 1) / a.slices);
  const int rows = min(kRows, a.M - m0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < kBufs; ++i) mbar_init(&done[i], 1), mbar_init(&taken[i], 8);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&a.tmap_x);
    prefetch_tensormap(&a.tmap_w);
  }
  if (warp == 1) {
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
    if (lane == 0) {
      const uint32_t bytes = a.x_rows * 128 + kOperand;
      int stage = 0, phase = 0, issued = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, a.status, a.wait_ns)) break;
        uint8_t* const st = smem + stage * 2 * kOperand;
        mbar_arrive_expect_tx(&full[stage], bytes);
        tma_load_2d(st, &a.tmap_x, kb * 128, m0, &full[stage]);
        tma_load_2d(st + kOperand, &a.tmap_w, kb * 128, n0, &full[stage]);
        if (GATED) tma_load_2d(st + kOperand + kOperand / 2, &a.tmap_w, kb * 128, a.cols + n0, &full[stage]);
        ++issued;
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
      // what was issued lands before the block ends, even if nothing waited for it
      for (int i = max(0, issued - kStages); i < issued; ++i) mbar_drain(&full[i % kStages], i / kStages & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0, phase = 0, buf = 0, buf_phase = 0, last = -1, last_phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&taken[buf], buf_phase ^ 1, abort_flag, a.status, a.wait_ns)) break;
        if (!mbar_wait(&full[stage], phase, abort_flag, a.status, a.wait_ns)) break;
        tc_fence_after();
        const uint32_t st = smem_u32(smem + stage * 2 * kOperand);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_e4m3(tmem + buf * kCols, sdesc_kmajor_sw128(st + 32 * k), sdesc_kmajor_sw128(st + kOperand + 32 * k),
                   idesc_e4m3(kRows, kCols), k != 0);
        tc_commit(&empty[stage]);
        tc_commit(&done[buf]);
        last = buf, last_phase = buf_phase;
        if (++stage == kStages) stage = 0, phase ^= 1;
        if (++buf == kBufs) buf = 0, buf_phase ^= 1;
      }
      if (last >= 0) mbar_drain(&done[last], last_phase);  // no MMA runs when TMEM is released
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;  // of the tile's rows and columns
    const int r = quarter * 32 + lane;
    const bool some = quarter * 32 < rows;                 // of the warp's rows there are any
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * (GATED ? 32 : 64);
    const float* const xs = a.xs + static_cast<int64_t>(m0 + min(r, rows - 1)) * a.xs_ld;
    const float* const ws = a.ws + static_cast<int64_t>(n0 / kGroup) * a.groups;
    const float* const ws_up = GATED ? a.ws + static_cast<int64_t>((a.cols + n0) / kGroup) * a.groups : ws;
    float acc[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0.0f;
    int buf = 0, buf_phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      const float x = some ? __ldg(xs + static_cast<int64_t>(kb) * a.xs_step) : 0.0f;
      const float s0 = x * __ldg(ws + kb), s1 = GATED ? x * __ldg(ws_up + kb) : s0;
      ok = __all_sync(0xffffffffu, mbar_wait(&done[buf], buf_phase, abort_flag, a.status, a.wait_ns));
      if (!ok) break;
      if (some) {
        uint32_t t[64];
        tc_fence_after();
        tmem_ld32_issue(at + buf * kCols, t);
        tmem_ld32_issue(at + buf * kCols + (GATED ? 64 : 32), t + 32);
        tmem_wait_ld<64>(t);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken[buf]);
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = fmaf(__uint_as_float(t[i]), i < 32 ? s0 : s1, acc[i]);
      } else if (lane == 0) {
        mbar_arrive(&taken[buf]);
      }
      if (++buf == kBufs) buf = 0, buf_phase ^= 1;
    }
    if (a.slices > 1) cluster_wait();  // every block of the cluster runs
    // The rows of the tile are dealt out to its slices, which add up their rows' sums: row r to block r / per.
    const int per = (rows + a.slices - 1) / a.slices;
    if (r < rows) {
      float* const to = sums + (slice * per + r % per) * kSumLd + half * (GATED ? 32 : 64);
      const uint32_t there = a.slices > 1 ? cluster_address(to, r / per) : smem_u32(to);
#pragma unroll
      for (int i = 0; i < 64; i += 4)
        store_cluster4(there + (GATED && i >= 32 ? i + 32 : i) * 4, acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    }
  }
  __syncwarp();
  if (a.slices > 1) {
    if (warp < 2) cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kBufs * kCols);
  }
  const int per = (rows + a.slices - 1) / a.slices, first = slice * per, mine = min(per, rows - first);
  for (int i = threadIdx.x; i < mine * kOut; i += kThreads) {
    const int r = i / kOut, c = i % kOut;
    if (n0 + c >= a.cols) continue;
    float g = 0.0f, u = 0.0f;
    for (int s = 0; s < a.slices; ++s) {
      g += sums[(s * per + r) * kSumLd + c];
      if (GATED) u += sums[(s * per + r) * kSumLd + kOut + c];
    }
    a.out[static_cast<int64_t>(m0 + first + r) * a.cols + n0 + c] = __bfloat16_as_ushort(__float2bfloat16_rn(activate(a.act, g, u)));
  }
}

template <bool GATED>
moe_status_t launch_tiles(Fp8Args a, const void* x, int64_t ld_x, const void* w, cudaStream_t s) {
  constexpr int kOut = GATED ? kCols / 2 : kCols;
  a.m_tiles = (a.M - 1) / kRows + 1;
  a.x_rows = a.M < kRows ? (a.M + 7) / 8 * 8 : kRows;
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * ((a.cols - 1) / kOut + 1);
  a.slices = 1;
  while (a.slices < kMaxSlices && tiles * a.slices * 2 <= num_sms() && a.groups >= 4 * a.slices) a.slices *= 2;
  MOE_CHECK(tiles * a.slices <= INT32_MAX, MOE_ERR_UNSUPPORTED_SHAPE);
  if (!encode_rows(&a.tmap_x, x, a.K, a.M, ld_x, a.x_rows) || !encode_rows(&a.tmap_w, w, a.K, a.N, a.K, kOut)) return MOE_ERR_CUDA;
  const auto kern = linear_fp8_kernel<GATED>;
  MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem));
  return launch_clusters(kern, a.slices, dim3(static_cast<unsigned>(tiles * a.slices)), dim3(kThreads), kTileSmem, s, a);
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
  Fp8Args a = {};
  a.xs = x_scale, a.ws = w_scale, a.out = out, a.status = dev_status, a.wait_ns = kWaitLimitNs;
  a.M = M, a.N = N, a.K = K, a.groups = groups, a.act = activation, a.cols = cols;
  a.xs_step = per_token ? 0 : 1, a.xs_ld = per_token ? 1 : groups;
  return gated ? launch_tiles<true>(a, x, ld_x, w, as_stream(stream)) : launch_tiles<false>(a, x, ld_x, w, as_stream(stream));
}
