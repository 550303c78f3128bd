// A few tokens times one dense NVFP4 matrix: y[m, n] = act(alpha * sum_k x[m, k] * w[n, k]).
//
// 9/16 byte per weight, read once per 16 tokens: bound by latency at four warps a scheduler (issue slots 62 %,
// the ALU pipe, which converts, 47 %) and by HBM (76 % of the copy rate). A warp takes 16 rows of w and a run
// of K: mma.m16n8k16 with the 16 weight rows as one operand and eight tokens as the other. K goes by chunks
// of 128 values. In a chunk lane (r, c) = (lane / 4, lane % 4) holds the values 32c to 32c + 31 of rows r and
// r + 8, and MMA step j takes its values 32c + 4j to 32c + 4j + 3.
//
// The codes come through a ring in shared memory that belongs to the warp (cp.async; two chunks a
// stage, two or three of them): copied as 128 contiguous bytes per row, a quarter of the L1 lines
// that fetching them in fragment order would touch, and swizzled so that reading them in that
// order meets no bank twice.
//
// The block first lays its slice of x out in shared memory as FP16 in fragment order. Each
// (token, chunk) has an FP32 factor: the tokens' own scales for E4M3 (exact in FP16), a power of two
// that brings the chunk's values into FP16's range for BF16. A chunk is summed on its own and
// enters the FP32 sum times its factor. Where a chunk's BF16 values span more than FP16 holds exactly (2^31;
// rare), the block lays x out again as it is and runs on BF16 MMAs, for which the weights take a
// second conversion: where the largest value's weight is zero, the small ones are all of the sum.
//
// Two ways of sharing K. Warps of one block (`across` of them) take neighbouring runs of the same
// rows, so that a block reads whole rows: DRAM gives 128 rows at a time read along K 4.8 TB/s, whole
// rows 5.9 (264 MB, read alone). Blocks of a cluster take slices of K where there are too few
// rows for the SMs, or too much x for shared memory. A row's sums belong to one block: the
// others store theirs into its shared memory, and after one barrier it adds all in a fixed order, so
// results do not depend on timing. alpha, the activation and the BF16 rounding come once at the
// end. A block goes on to further rows while there are any, their first chunks already in flight.
//
// Measured: 4 tokens x 129021 x 4096 57.6 us (5.2 TB/s; 159 instructions per 16 rows and chunk, 64 of them
// conversions at half rate; on BF16 MMAs 85 us); 8 x 4096 x 7168 with SwiGLU, E4M3 8.1 us, 1 x 2048 x 512
// 3.4 us, both chains of launch, loads, sums and barrier. The loop over rows exists twice: with the choice of
// the MMA inside it, calls that do not run BF16 ones took 0.2 to 1.2 us more.
#include <type_traits>

#include "cluster.cuh"
#include "common.cuh"
#include "fp4_mma.cuh"
#include "host_util.h"
#include "linear_cut.h"

namespace moe {
namespace {

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
  int stages;                              // of a warp's ring, two chunks each: 3 or 2
  int buffers;                             // of sums: 2, or 1 where memory is short
  bool gated;
};

__device__ __forceinline__ float silu(float g) { return __fdiv_rn(g, __fadd_rn(1.0f, expf(-g))); }
__device__ __forceinline__ float gelu(float x) {
  return __fmul_rn(__fmul_rn(0.5f, x), __fadd_rn(1.0f, erff(__fmul_rn(x, 0.70710678118654752f))));
}

__device__ __forceinline__ float relu(float x) { return x <= 0.0f ? 0.0f : x; }  // lets a NaN through

// act(g) * u for the gated kinds, act(g) otherwise
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

// 16 bytes of global memory into shared memory, asynchronously and past L1; fewer `bytes` leave zeros
// behind them
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// NT: groups of eight tokens; FP8: x is E4M3 with scales, else BF16
template <int NT, int ALIGN, bool FP8>
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
  constexpr int kRow = code_row(ALIGN), kSfRow = scale_row(ALIGN), kStage = stage_bytes(ALIGN);
  // shared memory: rings [warps][stages][kStage], x [M][slice * 256 + 64 bytes],
  // factors [slice][8 * NT], sums [buffers][16 * warps][8 * NT + 1]
  uint8_t* const xs = smem + a.warps * a.stages * kStage;
  const int x_row = a.slice * (kLinChunk * 2) + 64;
  float* const factor = reinterpret_cast<float*>(xs + M * x_row);
  constexpr int kSumRow = 8 * NT + 1;
  float* sums = factor + a.slice * 8 * NT;
  float* sums_next = a.buffers == 2 ? sums + 16 * a.warps * kSumRow : sums;

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

  // ---- the ring. Lane (q, p) = (lane / 8, lane % 8) copies piece p (16 bytes) of the codes of rows q, q + 4,
  // ..., lane 2i + j piece j of row i's scales. Past K lies the next row, which is copied along (zeros of x
  // meet its codes, its scales are cleared when read); past the matrix nothing is read.
  const uint32_t ring = smem_u32(smem) + warp * a.stages * kStage;
  const uint8_t* const ring_at = smem + warp * a.stages * kStage;
  const int q = lane >> 3, p = lane & 7;
  const uint32_t to = q * kRow + (ALIGN == kAlign16 ? p : p ^ (q & 1) << 2) * 16;
  const uint32_t sf_to = 16 * kRow + (lane >> 1) * kSfRow + (lane & 1) * 16;
  const int row_bytes = a.K / 2, sf_bytes = a.K / kBlock;
  const int64_t rows = static_cast<int64_t>(a.gated ? 2 : 1) * a.n_out;
  const uint8_t* const w_end = a.w + rows * row_bytes;
  const uint8_t* const sf_end = a.sf + rows * sf_bytes;
  // The tile to load next: its first column, its rows, and this lane's pieces of its first stage; the pieces
  // of the stage to load next. Tiles are 16 * so many rows apart, so that where a row starts in a
  // piece is the same for all of them.
  int load_col = static_cast<int>(blockIdx.x / a.slices) * n_per + i0, load_ch = first;
  const int64_t row_first = load_col + (up ? a.n_out : 0);
  const int64_t k_at = static_cast<int64_t>(chunk0 + first) * (kLinChunk / 2);
  const int64_t w_at = (row_first + q) * row_bytes, sf_at = (row_first + (lane >> 1)) * sf_bytes;
  const int64_t w_step = static_cast<int64_t>(stride) * n_per * row_bytes, sf_step = static_cast<int64_t>(stride) * n_per * sf_bytes;
  const uint8_t* w_tile = a.w + w_at + k_at + 16 * p - (ALIGN == kAlign16 ? w_at & 8 : 0);
  const uint8_t* sf_tile = a.sf + (sf_at & ~int64_t(15)) + k_at / 8 + 16 * (lane & 1);
  const bool sf_mine = (lane & 1) == 0 || (ALIGN != kAlign256 && (sf_at & 15) != 0);
  // a ninth piece of row `lane`'s codes, where it starts inside one
  const bool ninth = ALIGN == kAlign16 && lane < 16 && (((row_first + lane) * row_bytes) & 8) != 0;
  const int64_t to_ninth = (static_cast<int64_t>(lane) * row_bytes + 120) - (w_tile - (a.w + row_first * row_bytes + k_at));
  const uint8_t *w_from = w_tile, *sf_from = sf_tile;
  // a tile is whole, 16 rows and every piece of them inside the matrix, up to this column
  const int past_rows = static_cast<int>((static_cast<int64_t>(chunk0 + last + 2) * (kLinChunk / 2) + row_bytes - 1) / row_bytes);
  const int whole_to = static_cast<int>(min(rows - (up ? a.n_out : 0) - 15 - past_rows, static_cast<int64_t>(a.n_out) - 16));
  auto left = [](const uint8_t* from, const uint8_t* end) {
    return static_cast<uint32_t>(max(min(end - from, static_cast<ptrdiff_t>(16)), static_cast<ptrdiff_t>(0)));
  };
  auto load_stage = [&](int stage) {
    const uint32_t at = ring + stage * kStage;
    if (load_ch < last && load_col < a.n_out) {
      if (load_col <= whole_to) {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy_async(at + to + i * 4 * kRow, w_from + i * 4 * row_bytes);
        if (ninth) copy_async(at + lane * kRow + 128, w_from + to_ninth);
        if (ALIGN == kAlign256) {
          if (sf_mine) copy_async(at + sf_to, sf_from);
        } else if (sf_mine) {
          copy_async(at + sf_to, sf_from, left(sf_from, sf_end));
        }
      } else {
        const int load_rows = min(a.n_out - load_col, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* const from = w_from + i * 4 * static_cast<int64_t>(row_bytes);
          const uint32_t n = q + 4 * i < load_rows ? left(from, w_end) : 0;
          copy_async(at + to + i * 4 * kRow, n ? from : a.w, n);
        }
        if (ninth) {
          const uint32_t n = lane < load_rows ? left(w_from + to_ninth, w_end) : 0;
          copy_async(at + lane * kRow + 128, n ? w_from + to_ninth : a.w, n);
        }
        if (sf_mine) {
          const uint32_t n = (lane >> 1) < load_rows ? left(sf_from, sf_end) : 0;
          copy_async(at + sf_to, n ? sf_from : a.sf, n);
        }
      }
    }
    copies_commit();
    load_ch += 2;
    w_from += kLinChunk, sf_from += 2 * kLinChunk / kBlock;
    if (load_ch >= last) {
      load_ch = first, load_col += stride * n_per;
      w_from = w_tile += w_step, sf_from = sf_tile += sf_step;
    }
  };
  load_stage(0);
  if (a.stages == 3) load_stage(1);

  // x: half a warp per (token, chunk), eight values a lane, four loads in flight
  const int pairs = threads / 16, piece = tid & 15;
  uint32_t lost = 0;  // not zero: some value of x is not exact in FP16
  int m_next = chunks ? (tid >> 4) / chunks : M, ch_next = (tid >> 4) - m_next * chunks;
  const int m_step = chunks ? pairs / chunks : 0, ch_step = pairs - m_step * chunks;
  while (m_next < M) {
    uint4 raw[4];
    float scale[4];
    int ms[4], chs[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      ms[u] = m_next, chs[u] = ch_next;
      m_next += m_step, ch_next += ch_step;
      if (ch_next >= chunks) ch_next -= chunks, ++m_next;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int m = ms[u], ch = chs[u];
      const int64_t k = static_cast<int64_t>(chunk0 + ch) * kLinChunk + 8 * piece;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (m >= M) continue;
      if constexpr (!FP8) {
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
      const int m = ms[u], ch = chs[u];
      if (m >= M) break;
      const uint32_t v[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      uint4 f;
      if constexpr (!FP8) {
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
        if (amax < INFINITY)  // a sum with an infinity in it needs no other bits
          lost |= below_f16(v[0], f.x) | below_f16(v[1], f.y) | below_f16(v[2], f.z) | below_f16(v[3], f.w);
      } else {
        f = make_uint4(e4m3x2_to_f16x2(v[0] & 0xFFFF), e4m3x2_to_f16x2(v[0] >> 16), e4m3x2_to_f16x2(v[1] & 0xFFFF),
                       e4m3x2_to_f16x2(v[1] >> 16));
      }
      // piece p is half of lane column p / 4's share: its steps 2 * (p % 4) and the next
      *reinterpret_cast<uint4*>(xs + m * x_row + ch * 256 + ((piece & 3) * 4 + (piece >> 2)) * 16) = f;
      if (piece == 0) factor[ch * 8 * NT + m] = scale[u];
    }
  }
  bool wide = false;
  if constexpr (FP8) __syncthreads();
  else wide = __syncthreads_or(lost);
  if (!FP8 && wide) {
#pragma unroll 1
    for (int ch = tid >> 4; ch < chunks; ch += pairs) {
      const int64_t k = static_cast<int64_t>(chunk0 + ch) * kLinChunk + 8 * piece;
      const uint16_t* from = static_cast<const uint16_t*>(a.x) + m0 * a.ld_x + k;
      uint8_t* to = xs + ch * 256 + ((piece & 3) * 4 + (piece >> 2)) * 16;
#pragma unroll 1
      for (int m = 0; m < M; ++m, from += a.ld_x, to += x_row) {
        *reinterpret_cast<uint4*>(to) = k < a.K ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
        if (piece == 0) factor[ch * 8 * NT + m] = 1.0f;
      }
    }
    __syncthreads();
  }

  const int share = n_per / a.slices, kinds = a.gated ? 2 : 1, parts = a.slices * a.across;
  const float alpha = *a.alpha;
  if (a.slices > 1) cluster_wait();
  const uint8_t* x_lane[NT];  // columns of no token repeat the last one and are dropped
#pragma unroll
  for (int t = 0; t < NT; ++t) x_lane[t] = xs + min(8 * t + r, M - 1) * x_row + c * 16 + first * 256;
  const float* const factor_lane = factor + first * 8 * NT + 2 * c;
  // where rows r and r + 8 start in their first piece of codes, and of scales
  int code_at = 0, scale_at[2] = {0, 0};
  if constexpr (ALIGN != kAlign256) {
    if (ALIGN == kAlign16) code_at = ((row_first + r) * row_bytes) & 8;
    scale_at[0] = ((row_first + r) * sf_bytes) & 15, scale_at[1] = ((row_first + r + 8) * sf_bytes) & 15;
  }
  // Sums [part of K][kind][column of the owner's share][token], in the owner's shared memory: where this lane's
  // go. What meets at the barrier is the cluster, or the warps of one tile (and of its up rows), which
  // then add the tile's columns.
  int sum_at[2], owner[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int col = i0 + r + 8 * h;
    owner[h] = col / share;
    sum_at[h] = (((rank * a.across + part) * kinds + (up ? 1 : 0)) * share + col - owner[h] * share) * kSumRow + 2 * c;
  }
  const int own = tiles / kinds, group = tile % own;
  const int cols = a.slices > 1 ? share : 16, at_col = a.slices > 1 ? 0 : group * 16;
  const int member = a.slices > 1 ? tid : ((tile / own) * a.across + part) * 32 + lane;
  const int members = a.slices > 1 ? threads : a.across * kinds * 32;
  const int m_member = member / cols, col_member = at_col + member - m_member * cols;
  const int m_members = members / cols, col_members = members - m_members * cols;
  int stage = 0;
  auto turns = [&](auto in_bf16) {
    constexpr bool kBf16 = decltype(in_bf16)::value;
    for (int block = blockIdx.x / a.slices; block < blocks; block += stride) {
      float acc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
      const float* scale_of = factor_lane;
      int x_at = 0;
      for (int ch0 = first; ch0 < last; ch0 += 2) {
        if (a.stages == 3) copies_wait<1>();
        else copies_wait<0>();
        __syncwarp();  // every lane's copies of this stage are there, and the stage before it has been read
        load_stage(stage == 0 ? a.stages - 1 : stage - 1);
        const uint8_t* const at = ring_at + stage * kStage;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int ch = ch0 + u;
          if (u == 1 && ch >= last) break;
          uint32_t codes[2][4], two[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = r + 8 * h;
            if constexpr (ALIGN == kAlign16) {
              const uint2* const w = reinterpret_cast<const uint2*>(at + row * kRow + code_at + (4 * u + c) * 16);
              const uint2 x = w[0], y = w[1];
              codes[h][0] = x.x, codes[h][1] = x.y, codes[h][2] = y.x, codes[h][3] = y.y;
            } else {
              const uint4 x = *reinterpret_cast<const uint4*>(at + row * kRow + ((4 * u + c) ^ (r & 1) << 2) * 16);
              codes[h][0] = x.x, codes[h][1] = x.y, codes[h][2] = x.z, codes[h][3] = x.w;
            }
            const uint8_t* const s = at + 16 * kRow + row * kSfRow + scale_at[h] + 8 * u + 2 * c;
            if constexpr (ALIGN == kAlign16) two[h] = s[0] | static_cast<uint32_t>(s[1]) << 8;
            else two[h] = *reinterpret_cast<const uint16_t*>(s);
            if (ALIGN != kAlign256 && (chunk0 + ch + 1) * kLinChunk > a.K) {  // the next row's may be no numbers
              const int k = (chunk0 + ch) * kLinChunk + 32 * c;
              two[h] = k >= a.K ? 0 : k + kBlock >= a.K ? two[h] & 0xFF : two[h];
            }
            two[h] = e4m3x2_to_f16x2(two[h]);
          }
          float sum[NT][4];
          if constexpr (kBf16) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[t][0] = sum[t][1] = sum[t][2] = sum[t][3] = 0.0f;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // a word of either row: two MMA steps
            uint32_t f[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t s = __byte_perm(two[h], two[h], j < 2 ? 0x1010 : 0x3232);
              e2m1x8_to_f16x2(codes[h][j], f[h]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f[h][i] = mul_f16x2(f[h][i], s);
                if constexpr (kBf16) f[h][i] = f16x2_to_bf16x2(f[h][i]);
              }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const uint4 x = *reinterpret_cast<const uint4*>(x_lane[t] + x_at + u * 256 + j * 64);
              const uint32_t b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t A[4] = {f[0][2 * i], f[1][2 * i], f[0][2 * i + 1], f[1][2 * i + 1]};
                if constexpr (kBf16) mma_bf16(sum[t], A, b + 2 * i);
                else if (j == 0 && i == 0) mma_f16_first(sum[t], A, b);
                else mma_f16(sum[t], A, b + 2 * i);
              }
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float2 s = *reinterpret_cast<const float2*>(scale_of + (u * NT + t) * 8);
            acc[t][0] += sum[t][0] * s.x, acc[t][1] += sum[t][1] * s.y;
            acc[t][2] += sum[t][2] * s.x, acc[t][3] += sum[t][3] * s.y;
          }
        }
        x_at += 512, scale_of += 16 * NT;
        if (++stage == a.stages) stage = 0;
      }

      // A warp that has all of K and no activation to do has the result: 16 x 60000 x 256 6.4 us against 11.8 through
      // shared memory. (With the activations here too, their code made every size 0.1 us slower.)
      if (parts == 1 && a.act == MOE_ACT_IDENTITY) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = block * n_per + i0 + r + 8 * h;
          uint16_t* const to = a.out + static_cast<int64_t>(m0 + 2 * c) * a.n_out + col;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (col < a.n_out && 8 * t + 2 * c + i < M)
                to[static_cast<int64_t>(8 * t + i) * a.n_out] =
                    __bfloat16_as_ushort(__float2bfloat16_rn(acc[t][2 * h + i] * alpha));
        }
        continue;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* const to_sum = sums + sum_at[h];
        const uint32_t to_cluster = a.slices > 1 ? cluster_address(to_sum, owner[h]) : 0;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (a.slices > 1) store_cluster(to_cluster + 4 * (8 * t + i), acc[t][2 * h + i]);
            else to_sum[8 * t + i] = acc[t][2 * h + i];
          }
      }
      if (a.slices > 1) {
        cluster_arrive();
        cluster_wait();
      } else {
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(members) : "memory");
      }
      const int left_cols = a.n_out - (block * n_per + rank * share);
      for (int i = member, m = m_member, col = col_member; i < cols * M;) {
        if (col < left_cols) {
          const float* at = sums + col * kSumRow + m;
          float y[2] = {0.0f, 0.0f};
          for (int s = 0; s < parts; ++s) {
            y[0] += *at, at += share * kSumRow;
            if (a.gated) y[1] += *at, at += share * kSumRow;
          }
          a.out[static_cast<int64_t>(m0 + m) * a.n_out + block * n_per + rank * share + col] =
              __bfloat16_as_ushort(__float2bfloat16_rn(activate(a.act, y[0] * alpha, y[1] * alpha)));
        }
        i += members, m += m_members, col += col_members;
        if (col >= at_col + cols) col -= cols, ++m;
      }
      if (a.buffers == 2) {  // the other buffer is free: what it held was added before the barrier above
        float* const t = sums;
        sums = sums_next;
        sums_next = t;
      } else {
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(members) : "memory");
      }
    }
  };
  if constexpr (FP8) turns(std::false_type{});
  else if (wide) turns(std::true_type{});
  else turns(std::false_type{});
}

template <int NT, int ALIGN>
moe_status_t launch_linear(const LinArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
  auto* const kern = a.x_mode == MOE_FP8_NONE ? linear_kernel<NT, ALIGN, false> : linear_kernel<NT, ALIGN, true>;
  if (smem > 48 * 1024) MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
  return launch_clusters(kern, a.slices, grid, dim3(32 * a.warps), smem, s, a);
}

}  // namespace

constexpr int kLinSmem = 227 * 1024, kLinSmemSm = 228 * 1024;  // of a block; of an SM, 1 KB taken by each block

static int linear_smem(const LinCut& k, int align) {
  const int columns = k.tokens > 8 ? 16 : 8;
  return k.tokens * (k.slice * kLinChunk * 2 + 64) + k.slice * columns * 4 + k.buffers * 16 * k.warps * (columns + 1) * 4 +
         k.warps * k.stages * stage_bytes(align);
}

// The cut whose estimated time is least, of blocks of 2 to 16 warps, 1 to 8 of them on the same rows, in clusters
// of 1 to 8. The estimate (in us, less the launch) adds up what a block does:
//   1.0    per round of a warp's loads of x (four for either half), 0.005 per token and chunk laid out on an SM;
//   0.47   per turn (the sums), 0.7 more where a cluster meets; shared where an SM has several blocks and turns;
//   a warp's chunks one after the other at 0.18 each, or all of an SM's at 0.024 (up to 8 tokens) or 0.038, the
//   issue slots' rate, whichever is longer; 3 % more with a ring of two stages, and over several turns 23 % more
//   where one warp takes a run of K alone and 13 % where two or three do (DRAM: whole rows 5.9 TB/s, one run 4.8).
// Of that and the weights' bytes at 6 TB/s the longer counts, and a fifth of the shorter. Constants fitted to 61 shapes from
// 1 x 200 x 8192 to 4 x 129021 x 4096 and 16 x 60000 x 7168, each timed in every cut: the cut chosen is on average 2 %
// off the best of them (worst 20 %). Before the fit, halving and doubling blocks and slices until they filled the SMs was 15 %
// off (worst 52 %): 12 x 10240 x 7168 30.2 us against 21.6, 1 x 4096 x 4096 7.2 against 5.7.
bool cut_linear(int64_t M, int K, int n_out, bool gated, int align, int sms, LinCut* cut) {
  // warps and across: all of a block's to one tile of rows for little work, whole tiles for much
  static constexpr signed char kBlocks[][2] = {{2, 2},  {3, 3},  {4, 1},  {4, 2},  {4, 4},  {5, 5},  {6, 1},  {6, 2},  {6, 3},
                                               {7, 1},  {8, 1},  {8, 2},  {8, 4},  {8, 8},  {10, 1}, {10, 2}, {12, 1}, {12, 2},
                                               {12, 3}, {12, 4}, {14, 1}, {14, 2}, {16, 1}, {16, 2}, {16, 4}, {16, 8}};
  const int chunks = (K + kLinChunk - 1) / kLinChunk, kinds = gated ? 2 : 1;
  const float copy = static_cast<float>(n_out) * kinds * K * (9.0f / 16) / 6e6f;
  LinCut k;
  k.tokens = static_cast<int>(M < kLinTokens ? M : kLinTokens);
  float best = 0.0f;
  bool found = false;
  while (true) {
    k.groups = (M + k.tokens - 1) / k.tokens;
    const float unit = k.tokens > 8 ? 0.038f : 0.024f;
    for (k.slices = 1; k.slices <= 8; k.slices *= 2) {
      k.slice = ((chunks + k.slices - 1) / k.slices + 1) & ~1;  // whole stages
      if ((k.slices - 1) * k.slice >= chunks) break;
      const int pairs = k.tokens * (k.slice < chunks ? k.slice : chunks);
      for (const auto& b : kBlocks) {
        k.warps = b[0], k.across = b[1];
        const int tiles = k.warps / k.across, n_per = (gated ? 8 : 16) * tiles;
        if (tiles % kinds != 0 || n_per % k.slices != 0 || (k.across > 1 && 2 * k.across > k.slice + 1)) continue;
        if (k.slices == 1 && tiles / kinds > 15) continue;  // a barrier for each, and one for all
        k.stages = 3, k.buffers = 2;
        int smem = linear_smem(k, align);
        if (smem > kLinSmem) k.stages = 2, smem = linear_smem(k, align);
        if (smem > kLinSmem && k.slices == 1) k.buffers = 1, smem = linear_smem(k, align);  // a cluster needs both
        if (smem > kLinSmem) continue;
        const int fit = kLinSmemSm / (smem + 1024), most = kLinWarps / k.warps, per_sm = fit < most ? fit : most;
        // SMs that clusters of 4 and 8 leave over (the occupancy query's answer for 152): 8 and 32 at one block to an
        // SM, half and a quarter of that otherwise; the same share of fewer
        const int alone_over = k.slices == 8 ? sms * 4 / 19 : k.slices == 4 ? sms / 19 : 0;
        const int over = per_sm == 1 ? alone_over : k.slices == 8 ? sms / 19 : k.slices == 4 ? sms / 38 : 0;
        k.at_once = (sms - over) * per_sm / k.slices;
        if (k.at_once < 1) continue;
        const int64_t blocks = (static_cast<int64_t>(n_out) + n_per - 1) / n_per * k.groups;
        const int first = static_cast<int>(blocks < k.at_once ? blocks : k.at_once) * k.slices;
        const int spread = sms - alone_over;
        const int on_sm = (first + spread - 1) / spread < per_sm ? (first + spread - 1) / spread : per_sm;
        const float turns = static_cast<float>((blocks + k.at_once - 1) / k.at_once);
        int run = ((k.slice + k.across - 1) / k.across + 1) & ~1;
        run = run < chunks ? run : chunks;
        const float ends = turns * (k.slices > 1 ? 1.17f : 0.47f);
        const float alone = turns * 0.18f * run + ends;
        const float shared = turns * unit * (on_sm * k.warps * run) * (k.stages == 2 ? 1.03f : 1.0f) +
                             (turns > 1.0f ? ends / on_sm : ends);
        const float rows = turns == 1.0f || k.across >= 4 ? 1.0f : k.across > 1 ? 1.13f : 1.23f;
        const float work = (pairs + 8 * k.warps - 1) / (8 * k.warps) + 0.005f * (on_sm * pairs) + (alone > shared ? alone : shared) * rows;
        const float time = work > copy ? work + 0.2f * copy : copy + 0.2f * work;
        if (!found || time < best) found = true, best = time, *cut = k;
      }
    }
    if (found || k.tokens <= 8) return found;
    k.tokens = 8;  // the longest K: x of 16 tokens does not fit
  }
}

namespace {

// The estimates take 2 us of host time, so a thread keeps the cuts of the sizes it last asked for (a decoder's
// handful); they follow from the sizes alone.
bool cut_of(int64_t M, int K, int n_out, bool gated, int align, int sms, LinCut* cut) {
  struct Kept {
    int64_t M;
    int K, n_out, gated, sms;
    LinCut cut;
  };
  static thread_local Kept kept[64];
  const uint64_t hash = (static_cast<uint64_t>(M) * 0x9E3779B97F4A7C15ull ^ static_cast<uint64_t>(K) << 32 ^ n_out) * 0x9E3779B97F4A7C15ull;
  Kept& c = kept[hash >> 58];
  if (c.M != M || c.K != K || c.n_out != n_out || c.gated != gated || c.sms != sms) {
    if (!cut_linear(M, K, n_out, gated, align, sms, cut)) return false;
    c = {M, K, n_out, gated, sms, *cut};
  }
  *cut = c.cut;
  return true;
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
  MOE_CHECK(K % kBlock == 0 && K <= 65536 && N <= (1 << 30), MOE_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return MOE_OK;
  const bool fp8 = x_scale_mode != MOE_FP8_NONE;
  MOE_CHECK(x && w && w_sf && alpha && out && fp8 == (x_scale != nullptr), MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(aligned16(x) && reinterpret_cast<uintptr_t>(x_scale) % sizeof(float) == 0 && aligned16(w) && aligned16(w_sf) &&
                aligned16(alpha) && aligned16(out) && ld_x % (fp8 ? 16 : 8) == 0,
            MOE_ERR_MISALIGNED);
  const int chunks = (K + kLinChunk - 1) / kLinChunk, n_out = gated ? N / 2 : N, align = align_of(K);
  LinCut cut;
  MOE_CHECK(cut_of(M, K, n_out, gated, align, num_sms(), &cut) && cut.groups <= 65535, MOE_ERR_UNSUPPORTED_SHAPE);
  const LinArgs a = {x, x_scale, w, w_sf, alpha, out, ld_x, x_scale_mode, M, K, n_out, activation,
                     x_scale_mode == MOE_FP8_PER_GROUP ? chunks : 1, cut.slices, cut.slice, cut.tokens, cut.warps,
                     cut.across, cut.stages, cut.buffers, gated};
  const size_t ob = static_cast<size_t>(M) * a.n_out * 2;
  MOE_CHECK(!overlaps(out, ob, x, (static_cast<size_t>(M - 1) * ld_x + K) * (fp8 ? 1 : 2)) &&
                !overlaps(out, ob, w, static_cast<size_t>(N) * K / 2) &&
                !overlaps(out, ob, w_sf, static_cast<size_t>(N) * K / kBlock) && !overlaps(out, ob, alpha, 4) &&
                !overlaps(out, ob, x_scale, static_cast<size_t>(M) * a.x_groups * 4),
            MOE_ERR_OVERLAP);
  const size_t smem = linear_smem(cut, align);
  const int n_per = (gated ? 8 : 16) * (cut.warps / cut.across), blocks = (n_out + n_per - 1) / n_per;
  // as many clusters as run at once; they take row blocks in turn
  const dim3 grid((blocks < cut.at_once ? blocks : cut.at_once) * cut.slices, static_cast<unsigned>(cut.groups));
  cudaStream_t s = as_stream(stream);
  if (a.tokens <= 8)
    return align == kAlign256  ? launch_linear<1, kAlign256>(a, grid, smem, s)
           : align == kAlign32 ? launch_linear<1, kAlign32>(a, grid, smem, s)
                               : launch_linear<1, kAlign16>(a, grid, smem, s);
  return align == kAlign256  ? launch_linear<2, kAlign256>(a, grid, smem, s)
         : align == kAlign32 ? launch_linear<2, kAlign32>(a, grid, smem, s)
                             : launch_linear<2, kAlign16>(a, grid, smem, s);
}
