// A paged key/value cache in NVFP4: the append that encodes new tokens into it and the
// attention of a decode step that reads it.
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "fp4_mma.cuh"
#include "host_util.h"
#include "layout.h"

namespace moe {
namespace {

constexpr int kAppendThreads = 128;

struct Cache {
  uint8_t* data[2];  // keys, values
  uint8_t* sf[2];
  int64_t data_page, sf_page;
  float g[2];
  int pages, page_shift, heads, dim;
};

// One thread per 16-value block of one token's keys (blockIdx.y 0) or values (1): bound by its chain of
// load, block maximum, two divisions and stores (1 token of 8 heads of 128 1.3 us, 64 tokens 1.5, 512 tokens 1.7).
// The held value is code * (scale / g).
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(Cache c, const uint16_t* __restrict__ k_new,
                                                                   int64_t ld_k, const uint16_t* __restrict__ v_new,
                                                                   int64_t ld_v, const int64_t* __restrict__ slots,
                                                                   int N, uint16_t* k_seen, uint16_t* v_seen,
                                                                   int32_t* dev_status) {
  pdl_wait();
  pdl_trigger();
  const bool vals = blockIdx.y != 0;
  const int per_head = c.dim / kBlock, per_token = c.heads * per_head;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int64_t n = i / per_token;
  if (n >= N) return;
  const int b = static_cast<int>(i - n * per_token);
  const int head = b / per_head, blk = b - head * per_head;
  const int64_t slot = slots[n];
  float v[16];
  load_block16((vals ? v_new + n * ld_v : k_new + n * ld_k) + b * kBlock, v);
  uint32_t codes[2];
  const float g = vals ? c.g[1] : c.g[0];
  const uint32_t q = quantize_block16(v, g, codes);
  const int64_t page = slot >> c.page_shift;
  if (slot >= 0 && page < c.pages) {
    const int64_t row = (static_cast<int64_t>(head) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
    uint8_t* const data = (vals ? c.data[1] : c.data[0]) + page * c.data_page + row * (c.dim / 2) + blk * 8;
    uint8_t* const sf = (vals ? c.sf[1] : c.sf[0]) + page * c.sf_page + row * per_head + blk;
    *reinterpret_cast<uint2*>(data) = make_uint2(codes[0], codes[1]);
    *sf = static_cast<uint8_t>(q);
  } else if (slot >= 0 && dev_status && b == 0 && !vals) {
    atomicOr(dev_status, MOE_DEV_BAD_INDEX);
  }
  uint16_t* const seen = vals ? v_seen : k_seen;
  if (seen) {
    const float s = __fdiv_rn(e4m3_to_f32(q), g);
    uint32_t o[8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t f[4];
      e2m1x8_to_f16x2(codes[w], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
        const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * s, x.y * s);
        o[4 * w + j] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    uint4* const dst = reinterpret_cast<uint4*>(seen + (n * per_token + b) * kBlock);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---------------------------------------------------------------------------
// attention of a decode step
// ---------------------------------------------------------------------------
// One block per (share of a sequence's steps, kv head and up to 8 * NT of its query rows,
// sequence); each of `splits` blocks takes every splits-th run of `run` steps, so that they share what a sequence
// has whatever the table's width. Query rows are q_len * group many per kv head, row = t * group + g. Both
// products run transposed on mma.m16n8k16 (FP16 in, FP32 sums), so that the cached side is
// the 16-row operand and eight query rows fill its 8 columns:
//   S^T[token, row] = K[token, :] . Q[row, :]     per 16 tokens, D / 16 steps
//   O^T[dim, row]  += V^T[dim, token] . P^T       per 16 tokens, D / 16 tiles
// A cached value is code * scale with 6 significant bits, exact in FP16. The dimensions of an
// MMA step and the rows of an MMA tile are numbered so that a lane's operand bytes lie side
// by side in the cache: with r = lane / 4 and c = lane % 4, lane (r, c) reads bytes
// [c * D/8, +D/8) of the keys of tokens r and r + 8 (step j uses its dimensions c * D/4 + 4j to
// 4j + 3), and bytes [r * D/16, +D/16) of the values of tokens 2c, 2c+1, 2c+8 and 2c+9 (tile i
// has dimension r * D/8 + 2i as its row r and the next as its row r + 8). P^T's fragment is
// S^T's, transposed in 8 x 8 pieces (movmatrix).
//
// Each warp takes every kAttWarps-th group of 16 * U tokens and feeds itself through a ring of
// kAttStages groups in shared memory (bulk copies of 16 tokens, or of the group where one page holds
// it, one mbarrier per stage), so the warps of a block never wait for one another before the end.
//
// Softmax in base 2. A row's weights are p = 2^(s f - c), s a raw sum, f the row's factor from raw sums to scores and c
// the running reference fl(max f - 15), so that p is at most 2^15 but for c's rounding; they are
// rounded to FP16 for the second product (11 significant bits down to 2^-29 of the largest weight), their sum is
// FP32. Nothing but c's own rounding is between s f and c (one FMA), and c is what sums of different steps
// are brought together by. That holds while c is exact to a part of 1: query rows are scaled by a power
// of two to a largest value in [2^14, 2^15), so no score is above f 2^15 2688 D, and rows for which that is
// below 2^22 are the plain case. BF16 values so scaled fit FP16 down to 2^-31 of the largest.
//
// A block with a row of larger possible scores or of smaller values starts again with its queries in BF16, on BF16
// MMAs for the scores (the keys take a second conversion), with p = 2^((s - max) f + 15), which is right for
// scores of any size.
//
// Bound by latency at three warps a scheduler: no pipe is full (ALU, which converts, 54 %; issue slots 61 %; HMMA
// 27 %; 18.0 instructions per token and kv head), nor is HBM: 64 sequences of 4000 to 8191 tokens, 8 kv heads, 88 us
// (5.0 TB/s; the copies alone 73 us), one of 131071 tokens 35 us. Short ones by the chain of length, pages, first
// copies, steps and the join. Blocks that start again: those 64 sequences 125 us, the one 45.
constexpr int kAttWarps = 4;
constexpr int kAttStages = 2;
constexpr float kPShift = 15.0f;
constexpr float kMostScore = 0x1p22f;  // of the plain case, in base 2
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttendArgs {
  const uint16_t* q;
  const int32_t* table;
  const int32_t* lens;
  uint16_t* out;
  float* lse;
  float* part_o;   // [rows, splits, D]
  float2* part_ml; // [rows, splits]: reference of the weights and their sum
  float* row_f;    // [rows]: factor from references to base 2
  int32_t* dev_status;
  int64_t ld_q, ld_table;
  int q_len, q_heads, group, row_blocks, max_pages, splits, run;
  float scale;
  uint32_t wait_us;  // limit of every bounded wait (kWaitLimitNs unless a test build shortens it); 64 bits cost 2 %
  int withhold;      // test build only: the first of the tokens that are never copied, else -1
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// first token position that query row `row` of a sequence of `len` tokens does not see
__device__ __forceinline__ int row_limit(const AttendArgs& a, int len, int row) {
  return len - (a.q_len - 1) + row / a.group;
}

// four dimensions of a finished row (zeros when it saw nothing), and its log sum
__device__ __forceinline__ void store_row(const AttendArgs& a, int64_t at, float4 v, float total, float g) {
  const float f = total == 0.0f ? 0.0f : 1.0f / (total * g);
  ushort4 h;
  h.x = __bfloat16_as_ushort(__float2bfloat16_rn(v.x * f));
  h.y = __bfloat16_as_ushort(__float2bfloat16_rn(v.y * f));
  h.z = __bfloat16_as_ushort(__float2bfloat16_rn(v.z * f));
  h.w = __bfloat16_as_ushort(__float2bfloat16_rn(v.w * f));
  *reinterpret_cast<ushort4*>(a.out + at) = h;
}
__device__ __forceinline__ float row_lse(float top, float f, float total) {
  return total == 0.0f ? -INFINITY : (top * f + log2f(total)) * kLn2;
}

// A block's shared memory beside the ring; the plain case, which comes first, initialises it for both
template <int NT>
struct AttendShared {
  uint64_t full[2][kAttWarps][kAttStages];  // copies' barriers of the plain and the rare case
  float m[kAttWarps][8 * NT], l[kAttWarps][8 * NT], f[8 * NT];
  int abort_flag;
};

// The work of a block. False: its rows are not the plain case; nothing has been written and no copy is in flight.
template <int D, int NT, int U, bool RARE>
__device__ __forceinline__ bool attend_block(const Cache& c, const AttendArgs& a, uint8_t* ring, AttendShared<NT>& sh) {
  constexpr int kGroup = 16 * U, kStep = kAttWarps * kGroup;  // tokens of a step of a warp, of the block
  constexpr int KS = D / 16;       // MMA steps of S, MMA tiles of O
  constexpr int KW = D / 32;       // words of one token's keys per lane
  constexpr int VW = D / 64;       // words of one token's values per lane
  constexpr int R = 8 * NT;        // query rows of the block
  // a stage: keys and values of kGroup tokens, then their scales
  constexpr int kData = kGroup * D / 2, kSf = kGroup * D / 16, kStage = 2 * (kData + kSf);
  // ring: [warp][stage][kStage]; the warps' sums at the end
  uint64_t(&full)[kAttWarps][kAttStages] = sh.full[RARE];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, cc = lane & 3;
  if constexpr (!RARE) {
    if (lane < 2 * kAttStages) mbar_init(&sh.full[lane / kAttStages][warp][lane % kAttStages], 1);
    if (tid == 0) sh.abort_flag = 0;
    fence_mbar_init();
    __syncthreads();
    pdl_wait();
    pdl_trigger();
  }
  const int split = blockIdx.x, kvh = blockIdx.y / a.row_blocks, b = blockIdx.z;
  const int row0 = (blockIdx.y - kvh * a.row_blocks) * R;
  const int rows_here = min(R, a.q_len * a.group - row0);
  // Everything the block's first copies and its queries wait for is fetched at once; pages past the
  // sequence's end are fetched too and not used.
  const int32_t* table = a.table + b * a.ld_table;
  const int half = (lane >> 2) & (U - 1), first = split * a.run * kStep;
  // this warp's tokens of its present step, of the steps in flight, and of the one whose page is looked up
  int toks[kAttStages + 2], left = a.run;
  auto after = [&](int tok) {
    if (--left > 0) return tok + kStep;
    left = a.run;
    return tok + ((a.splits - 1) * a.run + 1) * kStep;
  };
  toks[0] = first + warp * kGroup;
#pragma unroll
  for (int i = 1; i <= kAttStages; ++i) toks[i] = after(toks[i - 1]);
  int len = a.lens[b], pages[kAttStages + 1];
#pragma unroll
  for (int i = 0; i <= kAttStages; ++i) {
    const int at = (toks[i] + 16 * half) >> c.page_shift;
    pages[i] = at < a.max_pages ? table[at] : -1;
  }
  uint32_t raw[NT][D / 8];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + 8 * t + r, at = row / a.group, g = row - at * a.group;
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q + (static_cast<int64_t>(b) * a.q_len + at) * a.ld_q + (kvh * a.group + g) * D + cc * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (8 * t + r < rows_here) u = src[i];
      raw[t][4 * i] = u.x, raw[t][4 * i + 1] = u.y, raw[t][4 * i + 2] = u.z, raw[t][4 * i + 3] = u.w;
    }
  }
  len = max(len, 0);
  const int64_t most = static_cast<int64_t>(a.max_pages) << c.page_shift;
  if (len > most) {
    len = static_cast<int>(most);
    if (a.dev_status && tid == 0) atomicOr(a.dev_status, MOE_DEV_BAD_INDEX);
  }
  const int seen = max(row_limit(a, len, row0 + rows_here - 1), 0);  // by the block's last row
  if (split > 0 && first >= seen) {  // nothing to see here: the join skips parts of sum 0
    if (tid < rows_here) {
      const int row = row0 + tid, t = row / a.group, g = row - t * a.group;
      const int64_t at = (static_cast<int64_t>(b) * a.q_len + t) * a.q_heads + kvh * a.group + g;
      a.part_ml[at * a.splits + split] = make_float2(-INFINITY, 0.0f);
    }
    return true;
  }
  const int end = seen, all_see = row_limit(a, len, row0);                       // every row sees the tokens before it

  // Lane 4u + w copies array w (keys, values, their scales) of the stage's u-th 16 tokens, or (u = 0) of
  // all of them where a page holds them. Copies stay inside a page whatever the sequence's length.
  uint8_t* const my_ring = ring + warp * (kAttStages * kStage);
  const bool wide = (1 << c.page_shift) >= kGroup;
  const int arr = lane & 3;
  const uint32_t row_bytes = arr < 2 ? D / 2 : D / 16;
  const uint8_t* const from = (arr == 0 ? c.data[0] : arr == 1 ? c.data[1] : arr == 2 ? c.sf[0] : c.sf[1]) +
                              (static_cast<int64_t>(kvh) << c.page_shift) * row_bytes;
  const int64_t from_page = arr < 2 ? c.data_page : c.sf_page;
  const uint32_t to = (arr < 2 ? arr * kData : 2 * kData + (arr - 2) * kSf) + half * 16 * row_bytes;
  auto page_of = [&](int tok) { return tok + 16 * half < end ? table[(tok + 16 * half) >> c.page_shift] : -1; };
  constexpr uint32_t kAll = 0x1111u & ((1u << (4 * U)) - 1);  // the lanes of array 0
  uint32_t held_next = 0;  // which 16-token runs of the stages in flight were copied, the oldest stage's in the low half
  auto issue = [&](int stage, int tok, int page) {
    const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(c.pages);
    const uint32_t held = __ballot_sync(0xffffffffu, ok) & kAll;
    held_next = kAttStages == 1 ? held : held_next >> 16 | held << (16 * (kAttStages - 1));
    if (lane == 0) mbar_arrive_expect_tx(&full[warp][stage], __popc(held) * (kStage / U));
    __syncwarp();
    const bool all = wide && held == kAll;
    if (lane < 4 * U && ok && (half == 0 || !all) && tok != a.withhold)
      bulk_load(my_ring + stage * kStage + to, from + page * from_page + ((tok + 16 * half) & ((1 << c.page_shift) - 1)) * row_bytes,
                (all ? kGroup : 16) * row_bytes, &full[warp][stage]);
  };
#pragma unroll
  for (int i = 0; i < kAttStages; ++i)
    if (toks[i] < end) issue(i, toks[i], toks[i] + 16 * half < end ? pages[i] : -1);
    else held_next >>= 16;
  int page = toks[kAttStages] + 16 * half < end ? pages[kAttStages] : -1;

  // Q^T fragments and each row's factor from raw sums to base-2 scores
  uint32_t q[NT][KS][2];
  float to_log2[NT][2];
  bool plain = true;
  // above 0, so that -inf stays -inf; finite, so that no difference stays 0
  auto factor = [&](float down) { return fminf(fmaxf(fabsf(a.scale) * kLog2e / c.g[0] * down, FLT_MIN), FLT_MAX); };
  if constexpr (RARE) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) q[t][i >> 1][i & 1] = raw[t][i] ^ (a.scale < 0.0f ? 0x80008000u : 0u);
      to_log2[t][0] = to_log2[t][1] = factor(1.0f);
    }
  } else {
    uint32_t not_plain = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(raw[t][i])), fabsf(bf16_hi(raw[t][i]))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float up, down;
      f16_range(amax, &up, &down);
      if (a.scale < 0.0f) up = -up;  // the factor is never negative
      uint32_t below = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        q[t][i >> 1][i & 1] = pack_f16x2(bf16_lo(raw[t][i]) * up, bf16_hi(raw[t][i]) * up);
        below |= below_f16(raw[t][i], q[t][i >> 1][i & 1]);
      }
      if (amax < INFINITY) not_plain |= below;  // a score with an infinity in it needs no other bits
      const float f = factor(down);
      not_plain |= f >= kMostScore / (0x1p15f * 2688.0f * D);
      to_log2[t][0] = __shfl_sync(0xffffffffu, f, 8 * cc);
      to_log2[t][1] = __shfl_sync(0xffffffffu, f, 8 * cc + 4);
    }
    plain = !__any_sync(0xffffffffu, not_plain != 0);  // the same for every warp of the block, by the same rows
  }

  float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int i = 0; i < KS; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.0f;
  }

  int stage = 0, no_number = INT_MAX;  // the first token after all_see whose values this lane keeps out
  uint32_t parity = 0;
  auto advance = [&] {
#pragma unroll
    for (int i = 0; i < kAttStages; ++i) toks[i] = toks[i + 1];
  };
  while (toks[0] < end && (RARE || plain)) {
    const int tok = toks[0];
    if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][stage], parity, &sh.abort_flag, a.dev_status, a.wait_us * uint64_t(1000)))) break;
    const uint8_t* const st = my_ring + stage * kStage;
    const uint32_t held = held_next & 0xFFFF;
    // ---- scores
    float s[U][NT][4];
    if constexpr (RARE) {
#pragma unroll
      for (int i = 0; i < U * NT * 4; ++i) s[i / (NT * 4)][i / 4 % NT][i % 4] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t kw[2][KW], sc[2][2];  // [token r or r + 8][...]; a block's scale in both halves
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * u + 8 * h + r;
        load_words<KW>(kw[h], st + row * (D / 2) + cc * (D / 8));
        const uint8_t* f = st + 2 * kData + row * (D / 16) + cc * (D / 64);
        const uint32_t two = e4m3x2_to_f16x2(D == 128 ? *reinterpret_cast<const uint16_t*>(f) : *f);
        sc[h][0] = __byte_perm(two, two, 0x1010);
        sc[h][1] = D == 128 ? __byte_perm(two, two, 0x3232) : sc[h][0];
      }
#pragma unroll
      for (int w = 0; w < KW; ++w) {  // a word is two steps
        uint32_t f[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) e2m1x8_to_f16x2(kw[h][w], f[h]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t x[4] = {mul_f16x2(f[0][2 * j], sc[0][w / 2]), mul_f16x2(f[1][2 * j], sc[1][w / 2]),
                                 mul_f16x2(f[0][2 * j + 1], sc[0][w / 2]), mul_f16x2(f[1][2 * j + 1], sc[1][w / 2])};
          if constexpr (RARE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f16x2_to_bf16x2(x[i]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if constexpr (RARE) mma_bf16(s[u][t], x, q[t][2 * w + j]);
            else if (w == 0 && j == 0) mma_f16_first(s[u][t], x, q[t][0]);
            else mma_f16(s[u][t], x, q[t][2 * w + j]);
          }
        }
      }
    }
    // ---- running maximum, weights
    uint32_t vsf[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        vsf[u][h] = st[2 * kData + kSf + (16 * u + 2 * cc + (h & 1) + 8 * (h >> 1)) * (D / 16) + r * (D / 16) / 8];
    if (tok + kGroup > min(all_see, end) || held != kAll) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool here = held >> (4 * u) & 1;
        if (!here && tok + 16 * u < end && a.dev_status && lane == 0) atomicOr(a.dev_status, MOE_DEV_BAD_INDEX);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = tok + 16 * u + r + 8 * (i >> 1);
            const int lim = min(end, row_limit(a, len, row0 + 8 * t + 2 * cc + (i & 1)));
            if (!here || at >= lim) s[u][t][i] = -INFINITY;
          }
        // values past the sequence's end may be anything: a zero scale keeps them out
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (!here || tok + 16 * u + 2 * cc + (h & 1) + 8 * (h >> 1) >= end) vsf[u][h] = 0;
      }
      // Of tokens that only some rows see, a scale that is no number is kept from the others too (the MMA
      // would give them 0 * NaN): the rows that see the first such token get their NaN after the last step.
      if (all_see < end) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int at = tok + 16 * u + 2 * cc + (h & 1) + 8 * (h >> 1);
            if (at >= all_see && (vsf[u][h] & 0x7F) == 0x7F) no_number = min(no_number, at), vsf[u][h] = 0;
          }
      }
    }
    uint32_t p[U][NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top[2], keep[2];
      bool grew = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = fmaxf(s[0][t][i], s[0][t][i + 2]);
#pragma unroll
        for (int u = 1; u < U; ++u) x = fmaxf(x, fmaxf(s[u][t][i], s[u][t][i + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        if constexpr (!RARE) x = fmaf(x, to_log2[t][i], -kPShift);
        top[i] = fmaxf(m[t][i], x);
        grew |= top[i] > m[t][i];
        keep[i] = top[i] == -INFINITY ? 0.0f : top[i];
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = ex2(RARE ? (m[t][i] - keep[i]) * to_log2[t][i] : m[t][i] - keep[i]);
          l[t][i] *= f;
#pragma unroll
          for (int j = 0; j < KS; ++j) o[t][j][i] *= f, o[t][j][i + 2] *= f;
          m[t][i] = top[i];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[u][t][i] = ex2(RARE ? fmaf(s[u][t][i] - keep[i & 1], to_log2[t][i & 1], kPShift)
                                 : fmaf(s[u][t][i], to_log2[t][i & 1], -keep[i & 1]));
          l[t][i & 1] += s[u][t][i];
        }
        p[u][t][0] = transpose8x8(pack_f16x2(s[u][t][0], s[u][t][1]));
        p[u][t][1] = transpose8x8(pack_f16x2(s[u][t][2], s[u][t][3]));
      }
    }

    // ---- weighted values
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t s01 = e4m3x2_to_f16x2(__byte_perm(vsf[u][0], vsf[u][1], 0x0040));
      const uint32_t s89 = e4m3x2_to_f16x2(__byte_perm(vsf[u][2], vsf[u][3], 0x0040));
      uint32_t vw[4][VW];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        load_words<VW>(vw[h], st + kData + (16 * u + 2 * cc + (h & 1) + 8 * (h >> 1)) * (D / 2) + r * (D / 16));
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        // bytes that pair one dimension's codes of two neighbouring tokens
        const uint32_t low = 0x0F0F0F0Fu;
        uint32_t f[4][4];
        e2m1x8_to_f16x2((vw[0][w] & low) | (vw[1][w] << 4 & ~low), f[0]);
        e2m1x8_to_f16x2((vw[0][w] >> 4 & low) | (vw[1][w] & ~low), f[1]);
        e2m1x8_to_f16x2((vw[2][w] & low) | (vw[3][w] << 4 & ~low), f[2]);
        e2m1x8_to_f16x2((vw[2][w] >> 4 & low) | (vw[3][w] & ~low), f[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x[4] = {mul_f16x2(f[0][i], s01), mul_f16x2(f[1][i], s01), mul_f16x2(f[2][i], s89),
                                 mul_f16x2(f[3][i], s89)};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_f16(o[t][4 * w + i], x, p[u][t]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    const int next = toks[kAttStages];
    if (next < end) {
      issue(stage, next, page);
      toks[kAttStages + 1] = after(next);
      page = page_of(toks[kAttStages + 1]);
    } else {
      held_next >>= 16;
      toks[kAttStages + 1] = next;
    }
    advance();
    toks[kAttStages] = toks[kAttStages + 1];
    if (++stage == kAttStages) stage = 0, parity ^= 1;
  }
  if constexpr (RARE) {  // the references are maxima here: 2^15 of the weights go
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[t][i] *= 0x1p-15f;
#pragma unroll
        for (int j = 0; j < KS; ++j) o[t][j][i] *= 0x1p-15f, o[t][j][i + 2] *= 0x1p-15f;
      }
  }
  // after a wait that gave up, or where the case is not plain: the stages in flight, before their memory is used again
  for (int i = 0; i < kAttStages && toks[0] < end; ++i) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(&full[warp][stage], parity))
      if (globaltimer_ns() - t0 > a.wait_us * uint64_t(1000)) {
        if (a.dev_status) atomicOr(a.dev_status, MOE_DEV_TIMEOUT);
        break;
      }
    if (++stage == kAttStages) stage = 0, parity ^= 1;
    advance();
  }
  __syncthreads();
  if (!plain) return false;

  if (__any_sync(0xffffffffu, no_number != INT_MAX)) {
    no_number = min(no_number, __shfl_xor_sync(0xffffffffu, no_number, 1));  // the lanes of the same dimensions
    no_number = min(no_number, __shfl_xor_sync(0xffffffffu, no_number, 2));
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (no_number < row_limit(a, len, row0 + 8 * t + 2 * cc + i))
#pragma unroll
          for (int j = 0; j < KS; ++j) o[t][j][i] = o[t][j][i + 2] = __int_as_float(0x7FC00000);
  }

  // ---- join the warps
  constexpr int ST = D + 4;
  auto so = reinterpret_cast<float(*)[R][ST]>(ring);  // [warp][row][dim]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = l[t][i];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      const int row = 8 * t + 2 * cc + i;
      if (r == 0) {
        sh.m[warp][row] = m[t][i];
        sh.l[warp][row] = x;
        if (RARE && warp == 0) sh.f[row] = to_log2[t][i];
      }
#pragma unroll
      for (int j = 0; j < KS; ++j)
        *reinterpret_cast<float2*>(&so[warp][row][r * (D / 8) + 2 * j]) = make_float2(o[t][j][i], o[t][j][i + 2]);
    }
  __syncthreads();
  for (int i = tid; i < rows_here * (D / 4); i += kAttWarps * 32) {
    const int row = i / (D / 4), d = 4 * (i - row * (D / 4));
    const float f_row = RARE ? sh.f[row] : 1.0f;
    float top = sh.m[0][row];
#pragma unroll
    for (int w = 1; w < kAttWarps; ++w) top = fmaxf(top, sh.m[w][row]);
    float total = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      if (sh.l[w][row] == 0.0f) continue;  // saw nothing (its maximum may be -inf)
      const float f = ex2((sh.m[w][row] - top) * f_row);
      total += sh.l[w][row] * f;
      const float4 x = *reinterpret_cast<const float4*>(&so[w][row][d]);
      v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
    }
    const int grow = row0 + row, t = grow / a.group, g = grow - t * a.group;
    const int64_t at = (static_cast<int64_t>(b) * a.q_len + t) * a.q_heads + kvh * a.group + g;
    if (a.splits > 1) {
      *reinterpret_cast<float4*>(a.part_o + (at * a.splits + split) * D + d) = v;
      if (d == 0) a.part_ml[at * a.splits + split] = make_float2(top, RARE ? -total : total);
      if (RARE && d == 0 && split == 0) a.row_f[at] = f_row;
    } else {
      store_row(a, at * D + d, v, total, c.g[1]);
      if (a.lse && d == 0) a.lse[at] = row_lse(top, f_row, total);
    }
  }
  return true;
}

// a function of its own: in the kernel, its code and registers cost the plain case up to 0.8 us
template <int D, int NT, int U>
__device__ __noinline__ void attend_rare(const Cache& c, const AttendArgs& a, uint8_t* ring, AttendShared<NT>& sh) {
  attend_block<D, NT, U, true>(c, a, ring, sh);
}

// U: runs of 16 tokens in a step of a warp. Two keep a short run's chain short; four spend less on the
// maximum, the barrier and the copies: 131071 tokens 35.2 us against 38.9, 64 x 4000 to 8191 91.9 against 102, 16 x
// 500 to 2000 11.9 against 14.0; 1 x 2000 7.1 either way.
template <int D, int NT, int U>
__global__ void __launch_bounds__(kAttWarps * 32, NT == 1 ? (U == 2 ? 4 : 3) : NT <= 3 ? 3 : 2)
    kv_attend_kernel(const __grid_constant__ Cache c, const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ AttendShared<NT> sh;
  if (!attend_block<D, NT, U, false>(c, a, ring, sh)) attend_rare<D, NT, U>(c, a, ring, sh);
}

// Joins the parts of query rows, W warps to a row. Every warp weighs all parts (a lane a part; those
// that saw nothing are not read, those of weight 0 are, for they may hold a NaN), then adds every so-manieth part with D / 4 lanes
// of four dimensions each; the groups of lanes are added in order.
constexpr int kJoinThreads = 256;

template <int D, int W>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(AttendArgs a, float g, int64_t rows) {
  constexpr int L = D / 4, P = 32 / L;  // lanes of a part, parts of a warp
  __shared__ float4 acc[W > 1 ? kJoinThreads / 32 : 1][L];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32 / W) + warp / W;
  const bool row = at < rows;
  const float2* ml = a.part_ml + at * a.splits;
  float top = -INFINITY, f_row = 1.0f;
  bool raw = false;  // references are raw sums, totals are stored negative
  if (row)
    for (int i = lane; i < a.splits; i += 32) {
      const float2 x = ml[i];
      top = fmaxf(top, x.x);
      raw |= signbit(x.y);
    }
  top = warp_max(top);
  if (__any_sync(0xffffffffu, raw)) f_row = a.row_f[at];
  const int part = lane / L, d = lane - part * L;
  const float4* po = reinterpret_cast<const float4*>(a.part_o + at * a.splits * D) + d;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float total = 0.0f;
  for (int i0 = 0; i0 < a.splits; i0 += 32) {
    float mine = -1.0f;
    if (row && i0 + lane < a.splits) {
      const float2 x = ml[i0 + lane];
      if (x.y != 0.0f) {
        mine = ex2((x.x - top) * f_row);
        total += mine * fabsf(x.y);
      }
    }
    const int here = min(a.splits - i0, 32);
#pragma unroll 4
    for (int j = w * P; j < here; j += W * P) {
      const float f = __shfl_sync(0xffffffffu, mine, (j + part) & 31);
      if (j + part < here && !(f < 0.0f)) {
        const float4 x = po[static_cast<int64_t>(i0 + j + part) * L];
        v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if constexpr (P == 2) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, 16), v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, 16), v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
  }
  if constexpr (W > 1) {
    if (part == 0) acc[warp][d] = v;
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int i = 1; i < W; ++i) {
      const float4 x = acc[warp + i][d];
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
  }
  if (!row || part != 0) return;
  store_row(a, at * D + 4 * d, v, total, g);
  if (a.lse && d == 0) a.lse[at] = row_lse(top, f_row, total);
}

// Steps that a block takes side by side, where several sequences share the SMs; a lone one's blocks take
// every so-manieth step. One run for each block would leave most blocks without work where the table is far wider
// than the sequences, runs of one step spread short sequences over more blocks than they are worth. One run, runs of one and
// runs of 8, with 131072 tokens' columns: 16 x 0 to 4097 tokens 34.6, 16.0 and 25.1 us, 64 x 4000 to 8191 131, 121 and 104;
// with the sequences' own: 16 x 500 to 2000 11.9, 14.1 and 11.9, 64 x 4000 to 8191 91.9, 94.1 and 91.9.
constexpr int kAttRun = 8;

// How a call is cut: rows of a block, and blocks of a sequence. A block takes as many row tiles as
// its registers hold, since all of them share one conversion of the cache.
struct Cut {
  int row_tiles, row_blocks, splits, run, halves;
};

Cut cut_attend(int batch, int kv_heads, int head_dim, int rows, int64_t most) {
  Cut k;
  const int tiles = (rows + 7) / 8, most_tiles = head_dim == 64 ? 4 : 2;
  k.row_blocks = (tiles + most_tiles - 1) / most_tiles;
  k.row_tiles = (tiles + k.row_blocks - 1) / k.row_blocks;
  // As many blocks as leave each 1 to 96 steps of the longest sequence, or twice, four times ... that, by the least
  // estimated time. The estimate (in us):
  //   a block's steps one after the other, 0.8 each (1.27 with U = 4), half as much again per further row tile, or the
  //   blocks of an SM, 0.0042 (0.006, 0.005, 0.0125 for 2 to 4 tiles, 9 % less with U = 4) per token and
  //   0.3 per tile for joining the warps, half of both where D is 64; whichever is longer;
  //   the blocks of one sequence come in whole rounds; of several, whose lengths are taken to fill 0.8 of the
  //   table, all but the last tenth of what runs at once is shared evenly where there are more than that;
  //   2.4 for the join and 1.4e-5 per row and run (half for D = 64).
  // Constants fitted to 39 shapes from 1 x 500 tokens to 64 x 8191, each timed in every cut. With three draws of the lengths
  // of the ragged ones the cut chosen is on average 6 % off the best (worst 38 %: the lengths are
  // not known here); before the fit, runs of at least two steps that filled the SMs once or twice were 11 % off (worst 42 %): 1 x 60000
  // tokens of 8 rows on one kv head 15.2 us against 10.9, 16 x 500 to 2000 of 8 x 4 heads 14.2 against 11.4; the other
  // way 3 x 10000 to 20000 of 8 x 8 heads 21.3 against 24.4.
  const int sms = num_sms();
  const int64_t blocks = static_cast<int64_t>(batch) * kv_heads * k.row_blocks;
  static constexpr float kToken[] = {0.0042f, 0.006f, 0.005f, 0.0125f};
  const float half = head_dim == 64 ? 0.5f : 1.0f, filled = batch == 1 ? 1.0f : 0.8f;
  const float of_rows = 1.4e-5f * half * batch * kv_heads * rows;
  float best = 0.0f;
  k.splits = 0;
  for (int u = 2; u <= (k.row_tiles == 1 ? 4 : 2); u += 2) {
    const int per_sm = k.row_tiles == 1 ? (u == 2 ? 4 : 3) : k.row_tiles <= 3 ? 3 : 2;
    const float token = kToken[k.row_tiles - 1] * half * (u == 4 ? 0.91f : 1.0f);
    const float step = (u == 4 ? 1.27f : 0.8f) * (1.0f + 0.52f * (k.row_tiles - 1));
    for (int64_t m = 1;; m += m < 10 ? 1 : m < 20 ? 2 : m < 32 ? 4 : m < 48 ? 8 : m < 64 ? 16 : m < 96 ? 32 : m) {
      const int64_t chunk = m * 16 * u * kAttWarps, splits = most > chunk ? (most + chunk - 1) / chunk : 1;
      if (splits > 1 << 17) continue;  // the kernel steps on by splits * run * 256 tokens in 32 bits
      const int64_t here = most < chunk ? most : chunk;
      const float one = here * token + 0.3f * half * k.row_tiles;
      const float turns = blocks * splits * filled / sms;
      const float shared = turns > per_sm ? (turns + 0.1f * per_sm) * one : ceilf(turns) * one;
      const float alone = step * ((here + 16 * u * kAttWarps - 1) / (16 * u * kAttWarps));
      const float time = (alone > shared ? alone : shared) + (splits > 1 ? 2.4f + of_rows * splits : 0.0f);
      if (k.splits == 0 || time < best) {
        best = time, k.splits = static_cast<int>(splits), k.halves = u;
        k.run = batch == 1 ? 1 : static_cast<int>((m + (m + kAttRun - 1) / kAttRun - 1) / ((m + kAttRun - 1) / kAttRun));
      }
      if (splits == 1) break;
    }
  }
  return k;
}

moe_status_t check_cache(const moe_kv_cache_t* c, Cache* out) {
  MOE_CHECK(c != nullptr, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(c->num_pages >= 0 && c->num_kv_heads >= 1 && isfinite(c->k_scale) && c->k_scale > 0.0f &&
                isfinite(c->v_scale) && c->v_scale > 0.0f,
            MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(c->head_dim == 64 || c->head_dim == 128, MOE_ERR_UNSUPPORTED_SHAPE);
  MOE_CHECK(c->page_size >= 16 && c->page_size <= 256 && (c->page_size & (c->page_size - 1)) == 0,
            MOE_ERR_UNSUPPORTED_SHAPE);
  MOE_CHECK(c->num_kv_heads <= 1024, MOE_ERR_UNSUPPORTED_SHAPE);
  const int64_t page = static_cast<int64_t>(c->num_kv_heads) * c->page_size * c->head_dim;
  MOE_CHECK(c->data_page_stride >= page / 2 && c->sf_page_stride >= page / 16, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(c->data_page_stride % 16 == 0 && c->sf_page_stride % 16 == 0, MOE_ERR_MISALIGNED);
  MOE_CHECK(c->num_pages == 0 || (c->k && c->k_sf && c->v && c->v_sf), MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(aligned16(c->k) && aligned16(c->k_sf) && aligned16(c->v) && aligned16(c->v_sf), MOE_ERR_MISALIGNED);
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  *out = {{c->k, c->v}, {c->k_sf, c->v_sf}, c->data_page_stride, c->sf_page_stride, {c->k_scale, c->v_scale},
          c->num_pages, shift, c->num_kv_heads, c->head_dim};
  return MOE_OK;
}

// whether [p, p + n) touches the cache's codes or scales
bool touches_cache(const moe_kv_cache_t* c, const void* p, size_t n) {
  if (c->num_pages == 0) return false;
  const int64_t page = static_cast<int64_t>(c->num_kv_heads) * c->page_size * c->head_dim;
  const size_t nd = static_cast<size_t>(c->num_pages - 1) * c->data_page_stride + page / 2;
  const size_t ns = static_cast<size_t>(c->num_pages - 1) * c->sf_page_stride + page / 16;
  return overlaps(p, n, c->k, nd) || overlaps(p, n, c->v, nd) || overlaps(p, n, c->k_sf, ns) ||
         overlaps(p, n, c->v_sf, ns);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_kv_append(const moe_kv_cache_t* cache, const uint16_t* k_new, int64_t ld_k,
                                      const uint16_t* v_new, int64_t ld_v, const int64_t* slots, int32_t N,
                                      uint16_t* k_seen, uint16_t* v_seen, int32_t* dev_status, moe_stream_t stream) {
  Cache c;
  moe_status_t st = check_cache(cache, &c);
  if (st != MOE_OK) return st;
  const int64_t width = static_cast<int64_t>(c.heads) * c.dim;
  MOE_CHECK(N >= 0 && ld_k >= width && ld_v >= width && (k_seen != nullptr) == (v_seen != nullptr),
            MOE_ERR_INVALID_ARGUMENT);
  if (N == 0) return MOE_OK;
  MOE_CHECK(k_new && v_new && slots, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(aligned16(k_new) && aligned16(v_new) && aligned16(slots) && aligned16(k_seen) && aligned16(v_seen) &&
                aligned16(dev_status) && ld_k % 8 == 0 && ld_v % 8 == 0,
            MOE_ERR_MISALIGNED);
  const size_t kb = (static_cast<size_t>(N - 1) * ld_k + width) * 2, vb = (static_cast<size_t>(N - 1) * ld_v + width) * 2;
  const size_t sb = k_seen ? static_cast<size_t>(N) * width * 2 : 0;
  MOE_CHECK(!touches_cache(cache, k_new, kb) && !touches_cache(cache, v_new, vb) && !touches_cache(cache, k_seen, sb) &&
                !touches_cache(cache, v_seen, sb) && !touches_cache(cache, slots, static_cast<size_t>(N) * 8) &&
                !overlaps(k_seen, sb, v_seen, sb) && !overlaps(k_seen, sb, k_new, kb) &&
                !overlaps(k_seen, sb, v_new, vb) && !overlaps(v_seen, sb, k_new, kb) && !overlaps(v_seen, sb, v_new, vb),
            MOE_ERR_OVERLAP);
  const int64_t blocks = static_cast<int64_t>(N) * (width / kBlock);
  MOE_CHECK(blocks < (int64_t(1) << 31) * kAppendThreads - kAppendThreads, MOE_ERR_UNSUPPORTED_SHAPE);
  return launch_pdl(kv_append_kernel, dim3(static_cast<unsigned>((blocks + kAppendThreads - 1) / kAppendThreads), 2),
                    dim3(kAppendThreads), 0, as_stream(stream), c, k_new, ld_k, v_new, ld_v, slots,
                    static_cast<int>(N), k_seen, v_seen, dev_status);
}

namespace {

// checks the sizes that the workspace and the launches are made from
moe_status_t attend_cut(const moe_kv_cache_t* cache, Cache* c, int32_t batch, int32_t q_len, int32_t num_q_heads,
                        int32_t max_pages, Cut* cut, size_t* bytes) {
  const moe_status_t st = check_cache(cache, c);
  if (st != MOE_OK) return st;
  MOE_CHECK(batch >= 0 && q_len >= 1 && num_q_heads >= 1 && num_q_heads % c->heads == 0 && max_pages >= 0,
            MOE_ERR_INVALID_ARGUMENT);
  const int64_t most = static_cast<int64_t>(max_pages) << c->page_shift;
  const int64_t rows = static_cast<int64_t>(q_len) * (num_q_heads / c->heads);
  MOE_CHECK(batch <= 65535 && most < (int64_t(1) << 30) && q_len <= 65535 && rows * c->heads <= 65535 &&
                rows * c->heads * (batch > 0 ? batch : 1) < (int64_t(1) << 31),
            MOE_ERR_UNSUPPORTED_SHAPE);
  *cut = cut_attend(batch > 0 ? batch : 1, c->heads, c->dim, static_cast<int>(rows), most);
  const int64_t parts = cut->splits > 1 ? static_cast<int64_t>(batch) * q_len * num_q_heads * cut->splits : 0;
  *bytes = static_cast<size_t>(roundup64(parts * c->dim * 4, 16) + parts * 8 + (parts ? parts / cut->splits * 4 : 0));
  return MOE_OK;
}

}  // namespace

extern "C" size_t moe_kv_attend_workspace_bytes(const moe_kv_cache_t* cache, int32_t batch, int32_t q_len,
                                                int32_t num_q_heads, int32_t max_pages) {
  Cache c;
  Cut cut;
  size_t bytes;
  return attend_cut(cache, &c, batch, q_len, num_q_heads, max_pages, &cut, &bytes) == MOE_OK ? bytes : 0;
}

moe_status_t moe::kv_attend(const moe_kv_cache_t* cache, const uint16_t* q, int64_t ld_q, int32_t batch, int32_t q_len,
                            int32_t num_q_heads, const int32_t* page_table, int64_t ld_table, int32_t max_pages,
                            const int32_t* seq_lens, float softmax_scale, uint16_t* out, float* lse, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, const TestOptions& topt, moe_stream_t stream) {
  Cache c;
  Cut cut;
  size_t need;
  const moe_status_t st = attend_cut(cache, &c, batch, q_len, num_q_heads, max_pages, &cut, &need);
  if (st != MOE_OK) return st;
  MOE_CHECK(ld_table >= max_pages && ld_q >= static_cast<int64_t>(num_q_heads) * c.dim && isfinite(softmax_scale),
            MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(workspace_bytes >= need, MOE_ERR_WORKSPACE_TOO_SMALL);
  if (batch == 0) return MOE_OK;
  MOE_CHECK(q && seq_lens && out && (page_table || max_pages == 0) && (workspace || need == 0),
            MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(aligned16(q) && aligned16(page_table) && aligned16(seq_lens) && aligned16(out) && aligned16(lse) &&
                aligned16(workspace) && aligned16(dev_status) && ld_q % 8 == 0,
            MOE_ERR_MISALIGNED);
  const size_t rows = static_cast<size_t>(batch) * q_len, width = static_cast<size_t>(num_q_heads) * c.dim;
  const void* in[3] = {q, page_table, seq_lens};
  const size_t in_bytes[3] = {((rows - 1) * ld_q + width) * 2,
                              (static_cast<size_t>(batch - 1) * ld_table + max_pages) * 4, static_cast<size_t>(batch) * 4};
  const void* to[3] = {out, lse, workspace};
  const size_t to_bytes[3] = {rows * width * 2, rows * num_q_heads * 4, need};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j) MOE_CHECK(!overlaps(to[i], to_bytes[i], in[j], in_bytes[j]), MOE_ERR_OVERLAP);
    for (int j = 0; j < i; ++j) MOE_CHECK(!overlaps(to[i], to_bytes[i], to[j], to_bytes[j]), MOE_ERR_OVERLAP);
    MOE_CHECK(!touches_cache(cache, to[i], to_bytes[i]), MOE_ERR_OVERLAP);
  }
  const size_t parts = cut.splits > 1 ? rows * num_q_heads * cut.splits : 0;
  float* part_o = parts ? static_cast<float*>(workspace) : nullptr;
  float2* part_ml = parts ? reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + roundup64(parts * c.dim * 4, 16))
                          : nullptr;
  float* row_f = parts ? reinterpret_cast<float*>(part_ml + parts) : nullptr;
  const uint64_t us = (topt.wait_limit_ns + 999) / 1000;
  const uint32_t wait_us = us < UINT32_MAX ? static_cast<uint32_t>(us) : UINT32_MAX;
  const AttendArgs a = {q, page_table, seq_lens, out, lse, part_o, part_ml, row_f, dev_status, ld_q, ld_table, q_len,
                        num_q_heads, num_q_heads / c.heads, cut.row_blocks, max_pages, cut.splits, cut.run,
                        softmax_scale, wait_us, topt.withhold_release ? 0 : -1};
  const dim3 grid(cut.splits, c.heads * cut.row_blocks, batch);
  decltype(&kv_attend_kernel<64, 1, 2>) kern;
  if (c.dim == 64)
    kern = cut.halves == 4      ? kv_attend_kernel<64, 1, 4>
           : cut.row_tiles == 1 ? kv_attend_kernel<64, 1, 2>
           : cut.row_tiles == 2 ? kv_attend_kernel<64, 2, 2>
           : cut.row_tiles == 3 ? kv_attend_kernel<64, 3, 2>
                                : kv_attend_kernel<64, 4, 2>;
  else
    kern = cut.halves == 4      ? kv_attend_kernel<128, 1, 4>
           : cut.row_tiles == 1 ? kv_attend_kernel<128, 1, 2>
                                : kv_attend_kernel<128, 2, 2>;
  // the warps' rings, and after them their sums in the same place
  const int rings = kAttWarps * kAttStages * 16 * cut.halves * c.dim * 9 / 8;
  const int sums = kAttWarps * 8 * cut.row_tiles * (c.dim + 4) * static_cast<int>(sizeof(float));
  const int smem = rings > sums ? rings : sums;
  if (smem > 48 * 1024) MOE_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  const moe_status_t ran = launch_pdl(kern, grid, dim3(kAttWarps * 32), smem, as_stream(stream), c, a);
  if (ran != MOE_OK || cut.splits == 1) return ran;
  // a warp to a row while there are rows enough, or too few parts to share (512 rows of 16 parts:
  // 0.9 us less than a block to a row); else the eight warps of a block (64 rows of 57 parts took a warp each 20 us)
  const bool one = cut.splits <= 16 || rows * num_q_heads >= static_cast<size_t>(num_sms()) * 16;
  auto* join = c.dim == 64 ? (one ? kv_join_kernel<64, 1> : kv_join_kernel<64, 8>)
                           : (one ? kv_join_kernel<128, 1> : kv_join_kernel<128, 8>);
  const int64_t all = static_cast<int64_t>(rows) * num_q_heads, per_block = one ? 8 : 1;
  return launch_pdl(join, dim3(static_cast<unsigned>((all + per_block - 1) / per_block)), dim3(kJoinThreads), 0,
                    as_stream(stream), a, c.g[1], all);
}

extern "C" moe_status_t moe_kv_attend(const moe_kv_cache_t* cache, const uint16_t* q, int64_t ld_q, int32_t batch,
                                      int32_t q_len, int32_t num_q_heads, const int32_t* page_table, int64_t ld_table,
                                      int32_t max_pages, const int32_t* seq_lens, float softmax_scale, uint16_t* out,
                                      float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                      moe_stream_t stream) {
  return kv_attend(cache, q, ld_q, batch, q_len, num_q_heads, page_table, ld_table, max_pages, seq_lens, softmax_scale,
                   out, lse, workspace, workspace_bytes, dev_status, TestOptions(), stream);
}
