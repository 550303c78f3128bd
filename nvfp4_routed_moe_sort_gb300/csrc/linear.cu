// A few tokens times one dense NVFP4 matrix: y[m, n] = act(alpha * sum_k x[m, k] * w[n, k]).
//
// Bound by HBM: 9/16 byte per weight, read once per 16 tokens. A block of warps takes 16 rows
// of w each and a slice of K: mma.m16n8k16 with the 16 weight rows as one operand
// and eight tokens as the other. Per 128 values of K (a chunk) lane (r, c) = (lane / 4, lane % 4)
// reads bytes [16c, 16c + 16) of rows r and r + 8 and their two scales each, kLinAhead chunks
// ahead in registers; MMA step j of the chunk takes its values 32c + 4j to 32c + 4j + 3.
//
// The block first lays its slice of x out in shared memory as FP16 in fragment order. Each
// (token, chunk) has an FP32 factor: the tokens' own scales for E4M3 (exact in FP16), a power of two
// that brings the chunk's values into FP16's range for BF16. A chunk is summed on its own and
// enters the FP32 sum times its factor.
//
// Blocks that share rows (slices of K) form a cluster. A row belongs to one of them: the others
// store their sums into its shared memory, and after one cluster barrier it adds them in rank
// order, so results do not depend on timing. alpha, the activation and the BF16 rounding come
// once at the end. A block goes on to further rows while there are any, its first chunks of them
// already in flight.
#include "common.cuh"
#include "fp4_mma.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kLinWarps = 8;              // most warps of a block, 16 rows of w each
constexpr int kLinTokens = 16;
constexpr int kLinChunk = 128;            // = MOE_FP8_GROUP
constexpr int kLinAhead = 4;
static_assert(kLinChunk == MOE_FP8_GROUP, "one E4M3 scale per chunk");

struct LinArgs {
  const void* x;
  const float* x_scale;
  const uint8_t* w;
  const uint8_t* sf;
  const float* alpha;
  uint16_t* out;
  int64_t ld_x;
  int x_mode, M, K, n_out, act, x_groups;  // n_out: columns of out
  int slices, slice;                       // blocks of a cluster, chunks of each
  int tokens;                              // tokens of a block
  int warps;                               // of a block; gated: half gate, half up rows
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

__device__ __forceinline__ void store_cluster_f32(float* p, uint32_t rank, float v) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 32 codes (16 bytes) of a row at byte `at`, and their two scales
struct Codes {
  uint32_t w[4], sf;
};

// One chunk's share of a lane: w and sf point at it. WIDE: rows are multiples of 16 bytes, otherwise
// of 8 (a lane's two blocks are loaded one by one).
template <bool WIDE>
__device__ __forceinline__ void load_codes(Codes& d, const uint8_t* w, const uint8_t* sf) {
  if constexpr (WIDE) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(d.w[0]), "=r"(d.w[1]), "=r"(d.w[2]), "=r"(d.w[3]) : "l"(w));
    d.sf = *reinterpret_cast<const uint16_t*>(sf);
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(w), b = *reinterpret_cast<const uint2*>(w + 8);
    d.w[0] = a.x, d.w[1] = a.y, d.w[2] = b.x, d.w[3] = b.y;
    d.sf = sf[0] | static_cast<uint32_t>(sf[1]) << 8;
  }
}
// A chunk that K ends in: a block past the end repeats the row's last one. Those meet zeros of x, but
// have to be numbers where the row holds numbers.
template <bool WIDE>
__device__ __forceinline__ void load_last_codes(Codes& d, const uint8_t* w, const uint8_t* sf, int k, int K) {
  if constexpr (WIDE) {
    k = min(k, K - 32);
    load_codes<true>(d, w + k / 2, sf + k / kBlock);
  } else {
    const int k0 = min(k, K - kBlock), k1 = min(k + kBlock, K - kBlock);
    const uint2 a = *reinterpret_cast<const uint2*>(w + k0 / 2), b = *reinterpret_cast<const uint2*>(w + k1 / 2);
    d.w[0] = a.x, d.w[1] = a.y, d.w[2] = b.x, d.w[3] = b.y;
    d.sf = sf[k0 / kBlock] | static_cast<uint32_t>(sf[k1 / kBlock]) << 8;
  }
}

// NT: groups of eight tokens
template <int NT, bool WIDE>
__global__ void __launch_bounds__(kLinWarps * 32, 2) linear_kernel(LinArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, threads = 32 * a.warps, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  const int rank = blockIdx.x % a.slices;
  if (a.slices > 1) cluster_arrive();  // this block has started: its shared memory may be written
  const int m0 = blockIdx.y * a.tokens, M = min(a.M - m0, a.tokens);
  const int chunk0 = rank * a.slice;
  const int chunks = max(0, min(a.slice, (a.K + kLinChunk - 1) / kLinChunk - chunk0));
  // shared memory: x [M][slice * 256 + 64 bytes], factors [slice][8 * NT], sums (twice) [16 * warps][8 * NT + 1]
  const int x_row = a.slice * (kLinChunk * 2) + 64;
  float* const factor = reinterpret_cast<float*>(smem + M * x_row);
  constexpr int kSumRow = 8 * NT + 1;
  float* sums = factor + a.slice * 8 * NT;
  float* sums_next = sums + 16 * a.warps * kSumRow;

  // A row block is n_per output columns: their rows of w, or for the gated kinds their gate rows
  // (first half of the warps) and up rows (second half)
  const int n_per = a.gated ? 8 * a.warps : 16 * a.warps;
  const bool up = a.gated && warp >= a.warps / 2;
  const int i0 = (up ? warp - a.warps / 2 : warp) * 16 + r;
  const int blocks = (a.n_out + n_per - 1) / n_per, stride = gridDim.x / a.slices;
  int block = blockIdx.x / a.slices;
  const uint8_t *w[2], *sf[2];
  auto rows_of = [&](int b) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int64_t n = min(static_cast<int64_t>(b) * n_per + i0 + 8 * h, static_cast<int64_t>(a.n_out) - 1);  // spare rows are dropped
      if (up) n += a.n_out;
      w[h] = a.w + n * (a.K / 2);
      sf[h] = a.sf + n * (a.K / kBlock);
    }
  };
  Codes buf[kLinAhead][2];
  // chunks ch to ch + kLinAhead - 1 of the slice; those past its end stay what they were
  auto load_step = [&](int u, int ch) {
    const int k = (chunk0 + ch) * kLinChunk + 32 * c;
    if ((chunk0 + ch + u + 1) * kLinChunk <= a.K && ch + u < chunks) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        load_codes<WIDE>(buf[u][h], w[h] + k / 2 + u * (kLinChunk / 2), sf[h] + k / kBlock + u * (kLinChunk / kBlock));
    } else if (ch + u < chunks) {
#pragma unroll
      for (int h = 0; h < 2; ++h) load_last_codes<WIDE>(buf[u][h], w[h], sf[h], k + u * kLinChunk, a.K);
    }
  };
  rows_of(block);
#pragma unroll
  for (int u = 0; u < kLinAhead; ++u) load_step(u, 0);

  // x: half a warp per (token, chunk), eight values a lane, four loads in flight
  const int pairs = threads / 16;
  for (int i = tid >> 4; i < M * chunks; i += 4 * pairs) {
    const int piece = tid & 15;
    uint4 raw[4];
    float scale[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int m = (i + u * pairs) / chunks, ch = i + u * pairs - m * chunks;
      const int64_t k = static_cast<int64_t>(chunk0 + ch) * kLinChunk + 8 * piece;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (m >= M) continue;
      if (a.x_mode == MOE_FP8_NONE) {
        if (k < a.K) raw[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + (m0 + m) * a.ld_x + k);
      } else {
        if (k < a.K) {
          const uint2 e = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + (m0 + m) * a.ld_x + k);
          raw[u].x = e.x, raw[u].y = e.y;
        }
        scale[u] = a.x_scale[static_cast<int64_t>(m0 + m) * a.x_groups + (a.x_mode == MOE_FP8_PER_GROUP ? chunk0 + ch : 0)];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int m = (i + u * pairs) / chunks, ch = i + u * pairs - m * chunks;
      if (m >= M) break;
      const uint32_t v[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      uint4 f;
      if (a.x_mode == MOE_FP8_NONE) {
        float amax = 0.0f, grow;
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(v[j])), fabsf(bf16_hi(v[j]))));
        const uint32_t half_warp = 0xFFFFu << (lane & 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(half_warp, amax, o));
        f16_range(amax, &grow, &scale[u]);
        f = make_uint4(pack_f16x2(bf16_lo(v[0]) * grow, bf16_hi(v[0]) * grow),
                       pack_f16x2(bf16_lo(v[1]) * grow, bf16_hi(v[1]) * grow),
                       pack_f16x2(bf16_lo(v[2]) * grow, bf16_hi(v[2]) * grow),
                       pack_f16x2(bf16_lo(v[3]) * grow, bf16_hi(v[3]) * grow));
      } else {
        f = make_uint4(e4m3x2_to_f16x2(v[0] & 0xFFFF), e4m3x2_to_f16x2(v[0] >> 16), e4m3x2_to_f16x2(v[1] & 0xFFFF),
                       e4m3x2_to_f16x2(v[1] >> 16));
      }
      // piece p is half of lane column p / 4's share: its steps 2 * (p % 4) and the next
      *reinterpret_cast<uint4*>(smem + m * x_row + ch * 256 + ((piece & 3) * 4 + (piece >> 2)) * 16) = f;
      if (piece == 0) factor[ch * 8 * NT + m] = scale[u];
    }
  }
  __syncthreads();

  const int share = n_per / a.slices, kinds = a.gated ? 2 : 1;
  const float alpha = *a.alpha;
  if (a.slices > 1) cluster_wait();
  const uint8_t* x_lane[NT];  // columns of no token repeat the last one and are dropped
#pragma unroll
  for (int t = 0; t < NT; ++t) x_lane[t] = smem + min(8 * t + r, M - 1) * x_row + c * 16;
  for (; block < blocks; block += stride) {
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
    for (int ch0 = 0; ch0 < chunks; ch0 += kLinAhead) {
      // what is loaded while this step's chunks are computed: the row block's next, or the next block's first
      const bool last = ch0 + kLinAhead >= chunks;
      const bool more = !last || block + stride < blocks;
      const int next = last ? 0 : ch0 + kLinAhead;
      if (last) rows_of(block + stride);
#pragma unroll
      for (int u = 0; u < kLinAhead; ++u) {
        const int ch = ch0 + u;
        if (ch < chunks) {
          float part[NT][4];
          const uint32_t two[2] = {e4m3x2_to_f16x2(buf[u][0].sf), e4m3x2_to_f16x2(buf[u][1].sf)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // a word of either row: two MMA steps
            uint32_t f[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t s = __byte_perm(two[h], two[h], j < 2 ? 0x1010 : 0x3232);
              e2m1x8_to_f16x2(buf[u][h].w[j], f[h]);
#pragma unroll
              for (int i = 0; i < 4; ++i) f[h][i] = mul_f16x2(f[h][i], s);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint4 x = *reinterpret_cast<const uint4*>(x_lane[t] + ch * 256 + j * 64);
              const uint32_t b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t A[4] = {f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1]};
                if (j == 0 && i == 0) mma_f16_first(part[t], A, b);
                else mma_f16(part[t], A, b + 2 * i);
              }
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float2 s = *reinterpret_cast<const float2*>(factor + (ch * NT + t) * 8 + 2 * c);
            acc[t][0] += part[t][0] * s.x, acc[t][1] += part[t][1] * s.y;
            acc[t][2] += part[t][2] * s.x, acc[t][3] += part[t][3] * s.y;
          }
        }
        if (more) load_step(u, next);
      }
    }

    // sums [rank][kind][column of the owner's share][token], in the owner's shared memory
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int owner = (i0 + 8 * h) / share;
      float* const to = sums + ((rank * kinds + (up ? 1 : 0)) * share + i0 + 8 * h - owner * share) * kSumRow + 2 * c;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (a.slices > 1) store_cluster_f32(to + 8 * t + i, owner, acc[t][2 * h + i]);
          else to[8 * t + i] = acc[t][2 * h + i];
        }
    }
    if (a.slices > 1) cluster_arrive(), cluster_wait();
    else __syncthreads();
    for (int i = tid; i < share * M; i += threads) {
      const int m = i / share, col = i - m * share;
      const int64_t n = static_cast<int64_t>(block) * n_per + rank * share + col;
      if (n >= a.n_out) continue;
      float y[2] = {0.0f, 0.0f};
      for (int s = 0; s < a.slices; ++s) {
        y[0] += sums[(s * kinds * share + col) * kSumRow + m];
        if (a.gated) y[1] += sums[((s * 2 + 1) * share + col) * kSumRow + m];
      }
      a.out[static_cast<int64_t>(m0 + m) * a.n_out + n] =
          __bfloat16_as_ushort(__float2bfloat16_rn(activate(a.act, y[0] * alpha, y[1] * alpha)));
    }
    // The other buffer is free: what it held was added before the barrier above.
    float* const t = sums;
    sums = sums_next;
    sums_next = t;
  }
}

template <int NT, bool WIDE>
moe_status_t launch_linear(const LinArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * a.warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.slices;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (smem > 48 * 1024)
    MOE_CUDA(cudaFuncSetAttribute(linear_kernel<NT, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
  return cudaLaunchKernelEx(&cfg, linear_kernel<NT, WIDE>, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

constexpr size_t kLinSmem = 100 * 1024, kLinSmemMost = 227 * 1024;  // two blocks per SM; the most of one

size_t linear_smem(int tokens, int slice, int warps) {
  const int columns = tokens > 8 ? 16 : 8;
  return static_cast<size_t>(tokens) * (slice * kLinChunk * 2 + 64) + static_cast<size_t>(slice) * columns * 4 +
         2 * static_cast<size_t>(16 * warps) * (columns + 1) * 4;
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
  const int chunks = (K + kLinChunk - 1) / kLinChunk;
  LinArgs a = {x, x_scale, w, w_sf, alpha, out, ld_x, x_scale_mode, M, K, gated ? N / 2 : N, activation,
               x_scale_mode == MOE_FP8_PER_GROUP ? chunks : 1, 1, chunks, kLinTokens, kLinWarps, gated};
  const size_t ob = static_cast<size_t>(M) * a.n_out * 2;
  MOE_CHECK(!overlaps(out, ob, x, (static_cast<size_t>(M - 1) * ld_x + K) * (fp8 ? 1 : 2)) &&
                !overlaps(out, ob, w, static_cast<size_t>(N) * K / 2) &&
                !overlaps(out, ob, w_sf, static_cast<size_t>(N) * K / kBlock) && !overlaps(out, ob, alpha, 4) &&
                !overlaps(out, ob, x_scale, static_cast<size_t>(M) * a.x_groups * 4),
            MOE_ERR_OVERLAP);
  // Slices of K (a cluster barrier each row block) while a warp keeps the chunks that it has in flight
  // anyway and all blocks run at once, two to an SM; more where x's share of shared memory asks for it.
  auto blocks = [&] {
    const int64_t n_per = gated ? 8 * a.warps : 16 * a.warps;
    return (a.n_out + n_per - 1) / n_per;
  };
  auto cut = [&](int most) {  // for blocks of at most `most` tokens
    a.tokens = M < most ? M : most;
    a.slices = 1, a.slice = chunks;
    const int64_t groups = (static_cast<int64_t>(M) + a.tokens - 1) / a.tokens;
    while (a.slices < 8 && a.slices < chunks &&
           ((a.slice > kLinAhead && blocks() * groups * a.slices <= num_sms()) ||
            linear_smem(a.tokens, a.slice, a.warps) > kLinSmem)) {
      a.slices *= 2;
      a.slice = (chunks + a.slices - 1) / a.slices;
    }
    return groups;
  };
  int64_t groups = cut(kLinTokens);
  if (linear_smem(a.tokens, a.slice, a.warps) > kLinSmemMost) groups = cut(8);  // the longest K
  // smaller blocks where whole ones leave SMs idle
  while (a.warps > 2 && blocks() * groups * a.slices < num_sms()) a.warps /= 2;
  const size_t smem = linear_smem(a.tokens, a.slice, a.warps);
  MOE_CHECK(groups <= 65535, MOE_ERR_UNSUPPORTED_SHAPE);
  // two blocks per SM; they take row blocks in turn
  const int64_t at_once = 2 * num_sms() / a.slices;
  const dim3 grid(static_cast<unsigned>((blocks() < at_once ? blocks() : at_once) * a.slices), static_cast<unsigned>(groups));
  const bool wide = K % 32 == 0;
  cudaStream_t s = as_stream(stream);
  if (a.tokens <= 8) return wide ? launch_linear<1, true>(a, grid, smem, s) : launch_linear<1, false>(a, grid, smem, s);
  return wide ? launch_linear<2, true>(a, grid, smem, s) : launch_linear<2, false>(a, grid, smem, s);
}
