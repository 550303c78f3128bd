// A few tokens times one dense NVFP4 matrix: y[m, n] = act(alpha * sum_k x[m, k] * w[n, k]).
//
// Bound by HBM: 9/16 byte per weight, read once per 16 tokens. A warp takes 16 rows of w and a run
// of K: mma.m16n8k16 with the 16 weight rows as one operand and eight tokens as the other. K
// goes by chunks of 128 values. In a chunk lane (r, c) = (lane / 4, lane % 4) holds the values 32c
// to 32c + 31 of rows r and r + 8, and MMA step j takes its values 32c + 4j to 32c + 4j + 3.
//
// The codes come through a ring in shared memory that belongs to the warp (cp.async; two chunks a
// stage, kLinStages of them): copied as 128 contiguous bytes per row, a quarter of the L1 lines
// that fetching them in fragment order would touch, and swizzled so that reading them in that
// order meets no bank twice.
//
// The block first lays its slice of x out in shared memory as FP16 in fragment order. Each
// (token, chunk) has an FP32 factor: the tokens' own scales for E4M3 (exact in FP16), a power of two
// that brings the chunk's values into FP16's range for BF16. A chunk is summed on its own and
// enters the FP32 sum times its factor.
//
// Two ways of sharing K. Warps of one block (`across` of them) take neighbouring runs of the same
// rows, so that a block reads whole rows: DRAM gives 128 rows at a time read along K 4.8 TB/s, whole
// rows 5.9 (302 MB, read alone). Blocks of a cluster take slices of K where there are too few
// rows for the SMs, or too much x for shared memory. A row's sums belong to one block: the
// others store theirs into its shared memory, and after one barrier it adds all in a fixed order, so
// results do not depend on timing. alpha, the activation and the BF16 rounding come once at the
// end. A block goes on to further rows while there are any, their first chunks already in flight.
#include "cluster.cuh"
#include "common.cuh"
#include "fp4_mma.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kLinWarps = 16;             // most warps of a block, 16 rows of w each
constexpr int kLinTokens = 16;
constexpr int kLinChunk = 128;            // = MOE_FP8_GROUP
constexpr int kLinStages = 3, kLinStage = 16 * 128 + 16 * 20;  // of two chunks: codes, scales
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
  int warps, across;                       // warps of a block, and how many of them share rows
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

// N bytes of global memory into shared memory, asynchronously; fewer `bytes` leave zeros behind them
template <int N>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, uint32_t bytes = N) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How rows of codes and of scales are aligned: K % 256 == 0, K % 32 == 0, or only K % 16 == 0
enum Align : int { kAlign256, kAlign32, kAlign16 };

// NT: groups of eight tokens
template <int NT, int ALIGN>
__global__ void __launch_bounds__(kLinWarps * 32, 1) linear_kernel(LinArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, threads = 32 * a.warps, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
  const int rank = blockIdx.x % a.slices;
  if (a.slices > 1) cluster_arrive();  // this block has started: its shared memory may be written
  const int m0 = blockIdx.y * a.tokens, M = min(a.M - m0, a.tokens);
  const int chunk0 = rank * a.slice;
  const int chunks = max(0, min(a.slice, (a.K + kLinChunk - 1) / kLinChunk - chunk0));
  // shared memory: rings [warps][kLinStages * kLinStage], x [M][slice * 256 + 64 bytes],
  // factors [slice][8 * NT], sums (twice) [16 * warps][8 * NT + 1]
  uint8_t* const xs = smem + a.warps * (kLinStages * kLinStage);
  const int x_row = a.slice * (kLinChunk * 2) + 64;
  float* const factor = reinterpret_cast<float*>(xs + M * x_row);
  constexpr int kSumRow = 8 * NT + 1;
  float* sums = factor + a.slice * 8 * NT;
  float* sums_next = sums + 16 * a.warps * kSumRow;

  // A row block is n_per output columns: their rows of w, or for the gated kinds their gate rows
  // (first half of the row tiles) and up rows (second half). Warp (tile, part) takes 16 of the rows
  // and the chunks [first, last) of the slice.
  const int tiles = a.warps / a.across, tile = warp / a.across, part = warp - tile * a.across;
  const int n_per = a.gated ? 8 * tiles : 16 * tiles;
  const bool up = a.gated && tile >= tiles / 2;
  const int i0 = (up ? tile - tiles / 2 : tile) * 16;
  const int blocks = (a.n_out + n_per - 1) / n_per, stride = gridDim.x / a.slices;
  const int run = ((chunks + a.across - 1) / a.across + 1) & ~1;  // whole stages
  const int first = min(part * run, chunks), last = min(first + run, chunks);

  // ---- the ring. Lane (q, p) = (lane / 8, lane % 8) copies piece p (16 bytes) of rows q, q + 4, ...
  const uint32_t ring = smem_u32(smem) + warp * (kLinStages * kLinStage);
  const uint8_t* const ring_at = smem + warp * (kLinStages * kLinStage);
  const int q = lane >> 3, p = lane & 7;
  const uint32_t to = q * 128 + ((p ^ (q & 1) << 2) << 4);
  const int sf_ld = a.K / kBlock;
  const uint8_t *w_from, *sf_from;  // this lane's first piece of codes, and of scales, of the next stage
  int load_block = blockIdx.x / a.slices, load_ch = first, load_rows;
  auto rows_of = [&] {
    const int64_t n = static_cast<int64_t>(load_block) * n_per + i0;
    load_rows = load_block < blocks ? static_cast<int>(min(static_cast<int64_t>(a.n_out) - n, int64_t(16))) : 0;
    const int64_t row = n + (up ? a.n_out : 0);
    w_from = a.w + (row + q) * (a.K / 2) + (chunk0 + first) * (kLinChunk / 2) + 16 * p;
    sf_from = a.sf + (row + (ALIGN == kAlign256 ? lane : q)) * sf_ld + (chunk0 + first) * (kLinChunk / kBlock);
  };
  const uint8_t* const sf_end = a.sf + static_cast<int64_t>(a.gated ? 2 : 1) * a.n_out * sf_ld;
  auto load_stage = [&](int stage) {
    const uint32_t at = ring + stage * kLinStage;
    if (load_ch < last && load_rows > 0) {
      const int k = (chunk0 + load_ch) * kLinChunk;
      const bool whole = load_rows == 16 && load_ch + 2 <= last && k + 2 * kLinChunk <= a.K;
      if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (ALIGN != kAlign16) {
            copy_async<16>(at + to + i * 512, w_from + i * 2 * a.K);
          } else {
            copy_async<8>(at + to + i * 512, w_from + i * 2 * a.K);
            copy_async<8>(at + to + i * 512 + 8, w_from + i * 2 * a.K + 8);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // rows past the matrix, pieces past K: zeros
          const bool row = q + 4 * i < load_rows && (p < 4 || load_ch + 1 < last);
          const bool in0 = row && k + 32 * p < a.K, in1 = row && k + 32 * p + kBlock < a.K;
          const uint8_t* const from = w_from + i * 2 * static_cast<int64_t>(a.K);
          if constexpr (ALIGN != kAlign16) {
            copy_async<16>(at + to + i * 512, in0 ? from : a.w, in0 ? 16 : 0);
          } else {
            copy_async<8>(at + to + i * 512, in0 ? from : a.w, in0 ? 8 : 0);
            copy_async<8>(at + to + i * 512 + 8, in1 ? from + 8 : a.w, in1 ? 8 : 0);
          }
        }
      }
      if constexpr (ALIGN == kAlign256) {  // one row's 16 scales a lane
        if (lane < 16) copy_async<16>(at + 2048 + lane * 16, lane < load_rows ? sf_from : a.sf, lane < load_rows ? 16 : 0);
      } else {  // the (up to five) words that hold a row's 16 scales, four rows at a time
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* const s = sf_from + 4 * i * static_cast<int64_t>(sf_ld);
          const uint8_t* const from = s - (reinterpret_cast<uintptr_t>(s) & 3) + 4 * p;
          const bool in = q + 4 * i < load_rows && from < sf_end;
          const int left = in ? static_cast<int>(min(sf_end - from, static_cast<ptrdiff_t>(4))) : 0;
          if (p < 5) copy_async<4>(at + 2048 + (q + 4 * i) * 20 + 4 * p, in ? from : a.sf, left);
        }
      }
    }
    copies_commit();
    load_ch += 2;
    w_from += kLinChunk, sf_from += 2 * kLinChunk / kBlock;
    if (load_ch >= last) {
      load_ch = first, load_block += stride;
      rows_of();
    }
  };
  rows_of();
#pragma unroll
  for (int u = 0; u < kLinStages - 1; ++u) load_stage(u);

  // x: half a warp per (token, chunk), eight values a lane, eight loads in flight
  const int pairs = threads / 16;
  for (int i = tid >> 4; i < M * chunks; i += 8 * pairs) {
    const int piece = tid & 15;
    uint4 raw[8];
    float scale[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
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
    for (int u = 0; u < 8; ++u) {
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
      *reinterpret_cast<uint4*>(xs + m * x_row + ch * 256 + ((piece & 3) * 4 + (piece >> 2)) * 16) = f;
      if (piece == 0) factor[ch * 8 * NT + m] = scale[u];
    }
  }
  __syncthreads();

  const int share = n_per / a.slices, kinds = a.gated ? 2 : 1, parts = a.slices * a.across;
  const float alpha = *a.alpha;
  if (a.slices > 1) cluster_wait();
  const uint8_t* x_lane[NT];  // columns of no token repeat the last one and are dropped
#pragma unroll
  for (int t = 0; t < NT; ++t) x_lane[t] = xs + min(8 * t + r, M - 1) * x_row + c * 16;
  int stage = 0;
  for (int block = blockIdx.x / a.slices; block < blocks; block += stride) {
    float acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
    uint32_t shift[2] = {0, 0};  // of a row's scales in their first word
    if constexpr (ALIGN != kAlign256) {
      const int64_t row = static_cast<int64_t>(block) * n_per + i0 + (up ? a.n_out : 0) + r;
      shift[0] = (row * sf_ld) & 3, shift[1] = ((row + 8) * sf_ld) & 3;
    }
    for (int ch0 = first; ch0 < last; ch0 += 2) {
      copies_wait<kLinStages - 2>();
      __syncwarp();  // every lane's copies of this stage are there, and the stage before it has been read
      load_stage(stage == 0 ? kLinStages - 1 : stage - 1);
      const uint8_t* const at = ring_at + stage * kLinStage;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int ch = ch0 + u;
        if (u == 1 && ch >= last) break;
        uint32_t codes[2][4], two[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = r + 8 * h;
          const uint4 x = *reinterpret_cast<const uint4*>(at + row * 128 + ((4 * u + c) ^ (r & 1) << 2) * 16);
          codes[h][0] = x.x, codes[h][1] = x.y, codes[h][2] = x.z, codes[h][3] = x.w;
          if constexpr (ALIGN == kAlign256) {
            two[h] = *reinterpret_cast<const uint16_t*>(at + 2048 + row * 16 + 8 * u + 2 * c);
          } else {
            const uint8_t* const s = at + 2048 + row * 20 + shift[h] + 8 * u + 2 * c;
            two[h] = s[0] | static_cast<uint32_t>(s[1]) << 8;
            // past K lie the next row's scales, which may be no numbers
            const int k = (chunk0 + ch) * kLinChunk + 32 * c;
            if (k + 32 > a.K) two[h] = k < a.K ? two[h] & 0xFF : 0;
          }
          two[h] = e4m3x2_to_f16x2(two[h]);
        }
        float sum[NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // a word of either row: two MMA steps
          uint32_t f[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t s = __byte_perm(two[h], two[h], j < 2 ? 0x1010 : 0x3232);
            e2m1x8_to_f16x2(codes[h][j], f[h]);
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
              if (j == 0 && i == 0) mma_f16_first(sum[t], A, b);
              else mma_f16(sum[t], A, b + 2 * i);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 s = *reinterpret_cast<const float2*>(factor + (ch * NT + t) * 8 + 2 * c);
          acc[t][0] += sum[t][0] * s.x, acc[t][1] += sum[t][1] * s.y;
          acc[t][2] += sum[t][2] * s.x, acc[t][3] += sum[t][3] * s.y;
        }
      }
      if (++stage == kLinStages) stage = 0;
    }

    // sums [part of K][kind][column of the owner's share][token], in the owner's shared memory
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = i0 + r + 8 * h, owner = col / share;
      float* const to_sum =
          sums + (((rank * a.across + part) * kinds + (up ? 1 : 0)) * share + col - owner * share) * kSumRow + 2 * c;
      const uint32_t to_cluster = a.slices > 1 ? cluster_address(to_sum, owner) : 0;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (a.slices > 1) store_cluster(to_cluster + 4 * (8 * t + i), acc[t][2 * h + i]);
          else to_sum[8 * t + i] = acc[t][2 * h + i];
        }
    }
    // What meets at the barrier: the cluster, or the warps of one tile (and of its up rows), which then
    // add the tile's columns
    int at_col = 0, cols = share, member = tid, members = threads;
    if (a.slices > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      const int own = tiles / kinds, group = tile % own;
      at_col = group * 16, cols = 16;
      member = ((tile / own) * a.across + part) * 32 + lane, members = a.across * kinds * 32;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(members) : "memory");
    }
    for (int i = member; i < cols * M; i += members) {
      const int m = i / cols, col = at_col + i - m * cols;
      const int64_t n = static_cast<int64_t>(block) * n_per + rank * share + col;
      if (n >= a.n_out) continue;
      float y[2] = {0.0f, 0.0f};
      for (int s = 0; s < parts; ++s) {
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

template <int NT, int ALIGN>
moe_status_t launch_linear(const LinArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
  if (smem > 48 * 1024)
    MOE_CUDA(cudaFuncSetAttribute(linear_kernel<NT, ALIGN>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
  return launch_clusters(linear_kernel<NT, ALIGN>, a.slices, grid, dim3(32 * a.warps), smem, s, a);
}

// shared memory of a block: two to an SM; the most of one; an SM's, 1 KB of it taken by each block
constexpr size_t kLinSmem = 113 * 1024, kLinSmemMost = 227 * 1024, kLinSmemSm = 228 * 1024;

size_t linear_smem(int tokens, int slice, int warps) {
  const int columns = tokens > 8 ? 16 : 8;
  return static_cast<size_t>(tokens) * (slice * kLinChunk * 2 + 64) + static_cast<size_t>(slice) * columns * 4 +
         2 * static_cast<size_t>(16 * warps) * (columns + 1) * 4 + static_cast<size_t>(warps) * kLinStages * kLinStage;
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
               x_scale_mode == MOE_FP8_PER_GROUP ? chunks : 1, 1, chunks, kLinTokens, 8, 1, gated};
  const size_t ob = static_cast<size_t>(M) * a.n_out * 2;
  MOE_CHECK(!overlaps(out, ob, x, (static_cast<size_t>(M - 1) * ld_x + K) * (fp8 ? 1 : 2)) &&
                !overlaps(out, ob, w, static_cast<size_t>(N) * K / 2) &&
                !overlaps(out, ob, w_sf, static_cast<size_t>(N) * K / kBlock) && !overlaps(out, ob, alpha, 4) &&
                !overlaps(out, ob, x_scale, static_cast<size_t>(M) * a.x_groups * 4),
            MOE_ERR_OVERLAP);
  auto blocks = [&] {
    const int64_t n_per = (gated ? 8 : 16) * (a.warps / a.across);
    return (a.n_out + n_per - 1) / n_per;
  };
  const int64_t sms = num_sms();
  a.tokens = M < kLinTokens ? M : kLinTokens;
  int64_t groups = (static_cast<int64_t>(M) + a.tokens - 1) / a.tokens;
  auto slice = [&](int n) { a.slices = n, a.slice = ((chunks + n - 1) / n + 1) & ~1; };  // whole stages
  auto smem_of = [&] { return linear_smem(a.tokens, a.slice, a.warps); };
  slice(1);
  if (blocks() * groups >= 2 * sms) {
    // Rows for many turns of every SM: one block of 16 warps to an SM, so that it lays x out once, four warps
    // to whole rows. Where x does not fit beside their rings, slices of K, and more rows to each of the
    // cluster's barriers as long as every cluster has four turns.
    a.warps = 16;
    while (a.slices < 8 && smem_of() > kLinSmemMost) slice(2 * a.slices);
    if (smem_of() > kLinSmemMost) {  // the longest K
      a.tokens = 8, groups = (static_cast<int64_t>(M) + 7) / 8;
    }
    a.across = a.slice >= 8 ? 4 : 1;
    if (a.slices > 1)
      while (a.across > 1 && blocks() / 2 * a.slices >= 4 * sms) a.across /= 2;
  } else {
    // Fewer rows: slices of K while a warp keeps two stages to itself and all blocks run at once, two to an SM,
    // and as x asks for; then smaller blocks where whole ones leave SMs idle.
    while (a.slices < 8 && a.slices < chunks &&
           ((a.slice > 4 && blocks() * groups * a.slices <= sms) || smem_of() > kLinSmem))
      slice(2 * a.slices);
    if (smem_of() > kLinSmemMost) {
      a.tokens = 8, groups = (static_cast<int64_t>(M) + 7) / 8;
    }
    while (a.warps > 2 && blocks() * groups * a.slices < sms) a.warps /= 2;
  }
  const size_t smem = smem_of();
  MOE_CHECK(groups <= 65535, MOE_ERR_UNSUPPORTED_SHAPE);
  // as many blocks as run at once; they take row blocks in turn
  const int64_t at_once = (a.warps > 8 || kLinSmemSm / (smem + 1024) < 2 ? 1 : 2) * sms / a.slices;
  const dim3 grid(static_cast<unsigned>((blocks() < at_once ? blocks() : at_once) * a.slices), static_cast<unsigned>(groups));
  cudaStream_t s = as_stream(stream);
  const int align = K % 256 == 0 ? kAlign256 : K % 32 == 0 ? kAlign32 : kAlign16;
  if (a.tokens <= 8)
    return align == kAlign256  ? launch_linear<1, kAlign256>(a, grid, smem, s)
           : align == kAlign32 ? launch_linear<1, kAlign32>(a, grid, smem, s)
                               : launch_linear<1, kAlign16>(a, grid, smem, s);
  return align == kAlign256  ? launch_linear<2, kAlign256>(a, grid, smem, s)
         : align == kAlign32 ? launch_linear<2, kAlign32>(a, grid, smem, s)
                             : launch_linear<2, kAlign16>(a, grid, smem, s);
}
