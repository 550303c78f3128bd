// One token per row of logits: temperature, top-k, top-p, min-p, drawn by a given random number.
//
// With the row's tokens in the order of their logits (ties: the lower index first) and the weights
// w = exp((l - max) / temperature), each filter keeps a front part of that order: top-k its first k tokens,
// top-p the shortest part whose weights reach top_p times the sum over what top-k kept, min-p the tokens with
// w >= min_p. The token taken is, among the kept ones in the order of their INDEX, the first at which the
// cumulated weight passes u times their sum.
//
// So a row needs no sort, only the last kept logit and how many of the tokens that share it are kept. It is found by
// histograms: 2048 bins of 1/64 in (max - l) / temperature, then the keys (the logits' bits in their order) of the bin in
// which the count or the weight is reached, 2048 ways a pass, until one key is left. BF16 logits mostly share one key by
// then. For top_k only tokens that can matter are counted: of the threads' largest logits the k-th, taken down to its bin's
// end, is no larger than the k-th of all. What is above that bound, what short rows have, and what a bin has goes to a list
// in shared memory, if it fits. Long rows of BF16 logits are counted by their values instead, which are few.
//
// Weights are whole numbers, 2^44 for the largest logit, so that sums are exact in any order and every
// block of a row sees the same ones. A weight is right to 2^-34 of itself (2^-37 on average) and rounded down to a unit. Of 131072
// tokens of like weight the border at which one token follows the next moves by less than 2^-18 of a token's width; the units that
// many small weights lose move it by 2^-44 of the largest each, 2^-26 where 2^18 weights are a unit or two. (With
// float32 exponentials it moves by hundredths of a token, and now and then another token is taken than in exact
// arithmetic.) exp2 in pieces: 1024 steps from a table, a polynomial of degree 2 for the rest, the argument
// carried as two floats.
//
// A row is spread over a cluster of blocks; histograms and totals meet in distributed shared memory. The row
// is read from L2 again for each pass over all of it: two where BF16 logits are counted by their values or no filter is
// set, three or four else.
//
// Bound by the chain of passes and meetings where rows are few (one row of 129021 BF16 logits: all tokens 13 us, top-k 17,
// top-p 18), by the shared-memory additions and the instructions around them where they are many (128 such rows: 35, 37 and
// 49 us; FP32 logits 60, 48 and 134). One row of 1001 FP32 logits: 5 to 12 us.
#include <math.h>

#include <atomic>

#include "cluster.cuh"
#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kBins = 2048;
constexpr int kThreads = 512, kWarps = 16;
constexpr int kMaxBlocks = 16;
constexpr int kMaxVocab = 1 << 18;
constexpr int kList = 4096;
constexpr uint32_t kNone = 0x007FFFFFu;  // the key of -infinity: such a token is never taken
constexpr uint64_t kOne = 1ull << 44;    // the weight of the largest logit
constexpr int kStepBits = 10;            // of the table of powers

// 2^(-j / 1024) in units of 2^-44, by products of repeated square roots of 1/2 in 63-bit fixed point
struct Powers {
  uint64_t t[1 << kStepBits];
  static constexpr uint64_t mul(uint64_t a, uint64_t b) {  // a * b / 2^63
    const uint64_t al = a & 0xFFFFFFFFu, ah = a >> 32, bl = b & 0xFFFFFFFFu, bh = b >> 32;
    const uint64_t mid = ah * bl + ((al * bl) >> 32), mid2 = al * bh + (mid & 0xFFFFFFFFu);
    const uint64_t high = ah * bh + (mid >> 32) + (mid2 >> 32);
    return (high << 1) | ((mid2 >> 31) & 1);
  }
  static constexpr uint64_t root(uint64_t v) {
    uint64_t x = 0;
    for (int b = 62; b >= 0; --b)
      if (mul(x | (1ull << b), x | (1ull << b)) <= v) x |= 1ull << b;
    return x;
  }
  constexpr Powers() : t() {
    uint64_t r[kStepBits] = {};  // r[b] = 2^(-2^b / 1024)
    uint64_t v = 1ull << 62;
    for (int b = kStepBits - 1; b >= 0; --b) r[b] = v = root(v);
    t[0] = 1ull << 63;
    for (int j = 1; j < 1 << kStepBits; ++j) {
      int b = 0;
      while (!((j >> b) & 1)) ++b;
      t[j] = mul(t[j & (j - 1)], r[b]);
    }
    for (int j = 0; j < 1 << kStepBits; ++j) t[j] = (t[j] + (1ull << 18)) >> 19;
    t[0] = kOne - 1;  // its upper half fits 31 bits, as the product below needs
  }
};
__device__ const Powers kPowers = Powers();

struct SampleArgs {
  const void* logits;
  const float *uniform, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  int64_t ld;
  int V, blocks;
};

// BF16 logits take few values. Those of magnitude 2^-8 to 2^7 have a place each in tables, by their bits: the positive ones
// in the first half, the negative ones in the second, zero last. In descending order they are the bins 0 to 2 * kSide, zero
// in the middle; the few nonzero ones nearer to zero (rare) are listed and count with zero.
constexpr uint32_t kSmallest = 0x3B80, kSide = 15 * 128;  // bits of 2^-8; values of a sign
constexpr int kZeroBin = kSide, kValues = 2 * kBins, kZeroPlace = kValues - 1;
__device__ __forceinline__ int value_place(uint32_t b) {  // of BF16 bits; below 0: not one of them, or zero
  const uint32_t off = (b & 0x7FFFu) - kSmallest;
  return off < kSide ? static_cast<int>(off + ((b & 0x8000u) >> 4)) : -1;
}
__device__ __forceinline__ int bin_place(int bin) {
  return bin < kZeroBin ? kSide - 1 - bin : bin == kZeroBin ? kZeroPlace : bin <= 2 * static_cast<int>(kSide) ? kBins + bin - kZeroBin - 1 : kSide;
}
__device__ __forceinline__ float bin_value(int bin) {
  if (bin == kZeroBin || bin > 2 * static_cast<int>(kSide)) return bin == kZeroBin ? 0.0f : -INFINITY;
  const uint32_t b = bin < kZeroBin ? kSmallest + (kSide - 1 - bin) : 0x8000u + kSmallest + (bin - kSide - 1);
  return __uint_as_float(b << 16);
}

struct Shared {
  uint64_t power[1 << kStepBits];
  uint64_t weight[kValues];    // of each of a BF16 logit's values
  union {
    uint64_t total[kBins];     // of every block's histogram
    uint32_t counts[kValues];  // ... of values
  };
  union {
    struct {
      uint32_t lo[kBins], hi[kBins];
    };
    uint32_t count[kValues];
  };
  uint32_t list[kList];        // keys that may be kept; rare values
  uint64_t warp_a[32];
  uint32_t warp_b[32], warp_c[32];
  // what each block of the row has to tell, written by them; one array for each meeting, since blocks may be one apart
  uint64_t peer_sum[kMaxBlocks], peer_rare[kMaxBlocks];
  uint32_t peer_others[kMaxBlocks];
  uint32_t peer_top[kMaxBlocks], peer_far[kMaxBlocks], peer_rares[kMaxBlocks], peer_low[kMaxBlocks], peer_high[kMaxBlocks], peer_same[kMaxBlocks];
  uint64_t before, target;
  int bin, listed;
};

// logits' bits in the order of their values; both zeros are one value
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ void store_cluster(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t at, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t load_cluster(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_scan(T v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T below = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += below;
  }
  return v;
}

// the whole part of v * n, 0 <= v < 1 and n < 2^63, and whether there is a rest
__device__ __forceinline__ uint64_t part_of(float v, uint64_t n, bool& rest) {
  const uint32_t b = __float_as_uint(v);
  const int e = b >> 23;
  const uint64_t m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int shift = 150 - (e ? e : 1);  // v = m / 2^shift, 23 <= shift
  const uint64_t hi = __umul64hi(m, n), lo = m * n;
  if (shift >= 128) return rest = (hi | lo) != 0, 0;
  if (shift >= 64) {
    const int s = shift - 64;
    rest = lo != 0 || (s && (hi << (64 - s)) != 0);
    return hi >> s;
  }
  rest = (lo << (64 - shift)) != 0;
  return (hi << (64 - shift)) | (lo >> shift);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// exp((l - top) / temperature) in units of 2^-44, ch + cl = log2(e) / temperature. Every step rounds by itself, whatever the
// compiler may contract: a multiply-add in place of p's product and a difference would count p's rounding twice (2^-19 of a
// weight), and the places of this function have to agree to the bit.
__device__ __forceinline__ uint64_t weight_of(const uint64_t* power, float top, float ch, float cl, float l) {
  if (l == top) return kOne;
  const float d = __fsub_rn(top, l);
  const float p = __fmul_rn(d, ch);
  if (!(p < 46.0f)) return 0;
  // what d and p lost by rounding
  const float back = __fsub_rn(top, d);
  const float dl = __fadd_rn(__fsub_rn(top, __fadd_rn(d, back)), __fsub_rn(back, l));
  float e = __fmaf_rn(d, ch, -p);
  e = __fmaf_rn(d, cl, e);
  e = __fmaf_rn(dl, ch, e);
  const float magic = 0x1.8p13f;  // rounds to multiples of 2^-10
  const float k = __fadd_rn(p, magic);
  const int steps = static_cast<int>(__float_as_uint(k) - __float_as_uint(magic));
  const float z = __fadd_rn(__fsub_rn(p, __fsub_rn(k, magic)), e);
  // 2^-z - 1, |z| <= 2^-11 and a bit: the cubic term is below 2^-37
  const float x = __fmul_rn(z, __fmaf_rn(z, 0.240226507f, -0.693147181f));
  const int part = __float2int_rn(__fmul_rn(x, 0x1p42f));
  const uint64_t t = power[steps & ((1 << kStepBits) - 1)];
  const int64_t w = static_cast<int64_t>(t) + ((static_cast<int64_t>(static_cast<int32_t>(t >> 13)) * part) >> 29);
  return static_cast<uint64_t>(w) >> (steps >> kStepBits);
}
// the same as a call: most of this kernel's code runs once a row and is slow to fetch, so there is to be little of it
__device__ __noinline__ uint64_t weight_call(const uint64_t* power, float top, float ch, float cl, float l) {
  return weight_of(power, top, ch, cl, l);
}

// A 16-byte piece of a row of V values that begins at value `at`: places outside the row, and NaN, are -infinity.
template <typename T>
__device__ __noinline__ uint4 odd_piece(const T* row, int V, int at) {
  uint32_t w[4] = {};
#pragma unroll
  for (int e = 0; e < 16 / static_cast<int>(sizeof(T)); ++e) {
    uint32_t b = sizeof(T) == 2 ? 0xFF80u : 0xFF800000u;
    if (at + e >= 0 && at + e < V) {
      const uint32_t l = row[at + e];
      if (!isnan(__uint_as_float(sizeof(T) == 2 ? l << 16 : l))) b = l;
    }
    if constexpr (sizeof(T) == 2) w[e / 2] |= b << (e % 2 * 16);
    else w[e] = b;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One row's block. All members but v0, count and rank are the same in all threads of all its blocks.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  Shared& s;
  const T* row;
  int V, skew;            // the row begins `skew` values into a 16-byte piece
  int v0, count;          // this block's pieces, from the one in which the row begins
  int rank, blocks;
  float top;              // the largest logit
  float ch, cl, step;     // log2(e) / temperature as two floats; bins per unit
  uint32_t tau;           // kept: keys above tau, and the first `ties` tokens of key tau
  uint32_t ties;
  uint64_t tie_weight;
  bool listed;            // what may be kept of this block's tokens is in the list

  __device__ __forceinline__ void sync() const {
    __syncwarp();
    if (blocks == 1) {
      __syncthreads();
    } else {
      cluster_arrive();
      cluster_wait();
    }
  }

  __device__ __forceinline__ static void unpack(const uint4& u, float* v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
  __device__ __forceinline__ static float most(const uint4& u) {  // NaN if there is one
    if constexpr (sizeof(T) == 2) {
      const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(u.x, u.y), max_nan_bf16x2(u.z, u.w));
      return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    } else {
      return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)), max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
  }

  __device__ __forceinline__ uint4 raw(int i) const {
    // pieces that lie inside the row are read whole, its ends by the value
    const int at = (v0 + i) * kVec - skew;
    if (at >= 0 && at + kVec <= V) return __ldg(reinterpret_cast<const uint4*>(row + at));
    return odd_piece(row, V, at);
  }
  __device__ __forceinline__ void clean(int i, uint4& u, float& m) const {
    m = most(u);
    if (isnan(m)) {
      u = odd_piece(row, V, (v0 + i) * kVec - skew);
      m = most(u);
    }
  }

  // pieces of a warp: [first, last), a run of neighbours, a warp's width at a time
  __device__ __forceinline__ void segment(int warp, int& first, int& last) const {
    const int per = ((count + kWarps - 1) / kWarps + 31) / 32 * 32;
    first = min(count, warp * per);
    last = min(count, first + per);
  }
  // f(piece, its largest value) for this thread's pieces, the next one in flight
  template <typename F>
  __device__ __forceinline__ void pieces(F&& f) const {
    int first, last;
    segment(threadIdx.x >> 5, first, last);
    int i = first + (threadIdx.x & 31);
    if (i >= last) return;
    uint4 next = raw(i), then = i + 32 < last ? raw(i + 32) : next;
#pragma unroll 1
    for (; i < last; i += 32) {
      uint4 u = next;
      next = then;
      if (i + 64 < last) then = raw(i + 64);
      float m;
      clean(i, u, m);
      f(u, m);
    }
  }
  // f(logit, key) for every token that may be kept
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    if (listed) {
      for (int i = threadIdx.x; i < s.listed; i += kThreads) f(value_of(s.list[i]), s.list[i]);
      return;
    }
    pieces([&](const uint4& u, float) {
      float v[kVec];
      unpack(u, v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(v[e], key_of(v[e]));
    });
  }

  // This block's tokens from `least` on, in the list; none is if they are too many.
  __device__ __forceinline__ void gather(float least) {
    if (threadIdx.x == 0) s.listed = 0;
    __syncthreads();
    pieces([&](const uint4& u, float m) {
      if (!(m >= least) || m == -INFINITY) return;
      float v[kVec];
      unpack(u, v);
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (v[e] >= least && v[e] > -INFINITY) {
          const int at = atomicAdd(&s.listed, 1);
          if (at < kList) s.list[at] = key_of(v[e]);
        }
    });
    __syncthreads();
    listed = s.listed <= kList;
  }

  __device__ __forceinline__ uint64_t weight(float l) const {
    return sizeof(T) == 2 ? weight_call(s.power, top, ch, cl, l) : weight_of(s.power, top, ch, cl, l);
  }

  __device__ __forceinline__ int bin_of(float l) const {
    return min(kBins - 1, static_cast<int>(fminf((top - l) * step, 4096.0f)));
  }

  template <bool WEIGHTS>
  __device__ __forceinline__ void add(int bin, uint64_t w) const {
    if constexpr (WEIGHTS) {
      const uint32_t low = static_cast<uint32_t>(w);
      const uint32_t was = atomicAdd(&s.lo[bin], low);
      const uint32_t high = static_cast<uint32_t>(w >> 32) + (was + low < was);
      if (high) atomicAdd(&s.hi[bin], high);
    } else {
      atomicAdd(&s.lo[bin], 1u);
    }
  }

  // Adds the blocks' histograms up in every block's `total` and clears them.
  __device__ __forceinline__ void meet() const {
    sync();
    if (blocks == 1) {
      for (int i = threadIdx.x; i < kBins; i += kThreads) {
        s.total[i] = static_cast<uint64_t>(s.hi[i]) << 32 | s.lo[i];
        s.lo[i] = s.hi[i] = 0;
      }
      __syncthreads();
      return;
    }
    const int slice = kBins / blocks;
    for (int i = rank * slice + threadIdx.x; i < (rank + 1) * slice; i += kThreads) {
      uint64_t sum = 0;
      for (int p = 0; p < blocks; ++p)
        sum += (static_cast<uint64_t>(load_cluster(cluster_address(&s.hi[i], p))) << 32) +
               load_cluster(cluster_address(&s.lo[i], p));
      for (int p = 0; p < blocks; ++p) store_cluster(cluster_address(&s.total[i], p), sum);
    }
    sync();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
  }

  // The first bin at which the cumulated total reaches the target (that number, or the part `p` of everything,
  // at least 1): bin, before and target in shared memory; bin -1 where it is never reached.
  __device__ __forceinline__ void reach(uint64_t target, const float* p, bool others) const {
    constexpr int own = kBins / kThreads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t mine = 0;
    for (int i = 0; i < own; ++i) mine += s.total[own * threadIdx.x + i];
    const uint64_t upto = warp_scan(mine, lane);
    if (lane == 31) s.warp_a[warp] = upto;
    if (threadIdx.x == 0) s.bin = -1;
    __syncthreads();
    const uint64_t sums = warp_scan(lane < kWarps ? s.warp_a[lane] : 0, lane);
    const uint64_t all = __shfl_sync(0xffffffffu, sums, 31);
    const uint64_t prior = __shfl_sync(0xffffffffu, sums, warp == 0 ? 0 : warp - 1);
    if (p) target = front_of(*p, all, others);
    uint64_t x = (warp == 0 ? 0 : prior) + upto - mine;
    if (x < target && target <= x + mine) {
      int bin = own * threadIdx.x;
      while (x + s.total[bin] < target) x += s.total[bin++];
      s.bin = bin, s.before = x, s.target = target;
    }
    __syncthreads();
  }
  // The least whole number that is at least p times `all`, and 1. Where there are `others` than the largest logit, their
  // weights were rounded down, the true sum is a little more than `all`, and a product without a rest is passed.
  __device__ __forceinline__ static uint64_t front_of(float p, uint64_t all, bool others) {
    bool rest;
    const uint64_t part = part_of(p, all, rest);
    return part + (rest || others) ? part + (rest || others) : 1;
  }

  // Counts this thread's pieces' values; rare ones go to the list. `far`: the largest value of magnitude 2^7 or more.
  __device__ __forceinline__ void count_values(const uint4& u, float& far) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu;
      const int place = value_place(b);
      if (place >= 0) {
        atomicAdd(&s.count[place], 1u);
      } else if ((b & 0x7FFFu) < kSmallest) {
        if ((b & 0x7FFFu) == 0) {
          atomicAdd(&s.count[kZeroPlace], 1u);
        } else {
          const int at = atomicAdd(&s.listed, 1);
          if (at < kList) s.list[at] = b << 16;
        }
      } else {
        far = fmaxf(far, __uint_as_float(b << 16));
      }
    }
  }

  static constexpr int kOwn = kValues / kThreads;  // neighbouring bins of a thread

  // The first of all threads' amounts, in order, at which their sum reaches the target (that number, or the part `p` of
  // everything), as reach() finds bins.
  __device__ __forceinline__ void reach_value(const uint64_t (&part)[kOwn], uint64_t target, const float* p, bool other) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) mine += part[i];
    const uint64_t upto = warp_scan(mine, lane);
    if (lane == 31) s.warp_a[warp] = upto;
    if (threadIdx.x == 0) s.bin = -1;
    other = __syncthreads_or(other);
    const uint64_t sums = warp_scan(lane < kWarps ? s.warp_a[lane] : 0, lane);
    const uint64_t all = __shfl_sync(0xffffffffu, sums, 31);
    const uint64_t prior = __shfl_sync(0xffffffffu, sums, warp == 0 ? 0 : warp - 1);
    if (p) target = front_of(*p, all, other);
    uint64_t x = (warp == 0 ? 0 : prior) + upto - mine;
    if (x < target && target <= x + mine) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (x < target && target <= x + part[i]) s.bin = kOwn * threadIdx.x + i, s.before = x, s.target = target;
        x += part[i];
      }
    }
    __syncthreads();
  }

  // top-k and top-p by the counts of values; the rare ones count with zero. `far`: there are tokens that were not counted.
  // False: the cut lies among the rare ones, and nothing was done.
  __device__ __forceinline__ bool cut_values(uint32_t k, const float* p, bool far) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t rare_weight = 0;
    uint32_t rares = s.listed;
    for (int i = threadIdx.x; i < rares; i += kThreads) rare_weight += weight(__uint_as_float(s.list[i]));
    rare_weight = warp_sum(rare_weight);
    if (lane == 0) s.warp_a[warp] = rare_weight;
    __syncthreads();
    rare_weight = warp_sum(lane < kWarps ? s.warp_a[lane] : 0);
    if (blocks > 1) {
      if (threadIdx.x < blocks) {
        store_cluster(cluster_address(&s.peer_rare[rank], threadIdx.x), rare_weight);
        store_cluster(cluster_address(&s.peer_rares[rank], threadIdx.x), rares);
      }
      sync();
      rare_weight = 0, rares = 0;
      for (int q = 0; q < blocks; ++q) rare_weight += s.peer_rare[q], rares += s.peer_rares[q];
      const int slice = kValues / blocks;
      for (int i = rank * slice + threadIdx.x; i < (rank + 1) * slice; i += kThreads) {
        uint32_t sum = 0;
        for (int q = 0; q < blocks; ++q) sum += load_cluster(cluster_address(&s.count[i], q));
        for (int q = 0; q < blocks; ++q) store_cluster(cluster_address(&s.counts[i], q), sum);
      }
      sync();
    }
    // weights of the values that occur, neighbouring bins by turns to the warps: few values lie in few runs of bins
    const uint32_t* const counts = blocks > 1 ? s.counts : s.count;
    bool other = far;  // than the largest logit
#pragma unroll 1
    for (int bin = threadIdx.x; bin <= 2 * kSide; bin += kThreads) {
      const int at = bin_place(bin);
      if (counts[at]) {
        const float value = bin_value(bin);
        s.weight[at] = weight(value);
        other = other || value != top;
      }
    }
    __syncthreads();
    // from here on a thread's bins are in its registers
    uint32_t n[kOwn];
    uint64_t w[kOwn], part[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) n[i] = counts[bin_place(kOwn * threadIdx.x + i)];  // place kSide, for those past the last, is empty
#pragma unroll
    for (int i = 0; i < kOwn; ++i) w[i] = n[i] ? s.weight[bin_place(kOwn * threadIdx.x + i)] : 0;
    __syncthreads();  // the counts are read
    for (int i = threadIdx.x; i < kValues; i += kThreads) s.count[i] = 0;
    constexpr int zero_thread = kZeroBin / kOwn, zero_at = kZeroBin % kOwn;
    const bool zero = threadIdx.x == zero_thread && rares;
    other = other || zero;
    int end = kValues;
    uint32_t end_count = 0;
    if (k) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) part[i] = (w[i] ? n[i] : 0) + (zero && i == zero_at && rare_weight ? rares : 0);
      reach_value(part, k, nullptr, false);
      if (s.bin >= 0) end = s.bin, end_count = static_cast<uint32_t>(s.target - s.before);
      if (end == kZeroBin && rares) return false;
      if (end < kValues) {
        other = false;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const int bin = kOwn * threadIdx.x + i;
          if (bin > end) n[i] = 0;
          if (bin == end) n[i] = end_count;
          other = other || (n[i] && bin_value(bin) != top);
        }
        other = other || (zero && kZeroBin < end);
      }
    }
    if (p) {
      if (k) __syncthreads();  // s.bin and its company are read
#pragma unroll
      for (int i = 0; i < kOwn; ++i) part[i] = n[i] * w[i] + (zero && i == zero_at && kZeroBin < end ? rare_weight : 0);
      reach_value(part, 0, p, other);
      end = s.bin;
      if (end == kZeroBin && rares) return false;
      const uint64_t each = s.weight[bin_place(end)];
      end_count = static_cast<uint32_t>((s.target - s.before + each - 1) / each);
    }
    if (end < kValues) {
      tau = key_of(bin_value(end)), ties = end_count, tie_weight = s.weight[bin_place(end)];
      __syncthreads();  // ... and from here on the table holds what tokens above tau weigh
      for (int bin = end + threadIdx.x; bin <= 2 * static_cast<int>(kSide); bin += kThreads) s.weight[bin_place(bin)] = 0;
    }
    return true;
  }

  // Cuts the kept tokens to the shortest front part whose count or weight reaches the target.
  template <bool WEIGHTS>
  __device__ __forceinline__ void cut(const float* p, uint64_t target = 0) {
    const bool group = WEIGHTS && ties > 0;            // kept tokens of key tau,
    const bool mine = group && rank == 0 && threadIdx.x == 0;  // added by one thread
    const uint64_t group_weight = ties * tie_weight;
    bool others = group && value_of(tau) != top;       // than the largest logit
    each([&](float l, uint32_t key) {
      if (key <= tau) return;
      others = others || l != top;
      const uint64_t w = WEIGHTS ? weight(l) : 1;
      if (!WEIGHTS || w) add<WEIGHTS>(bin_of(l), w);
    });
    if (mine) add<WEIGHTS>(bin_of(value_of(tau)), group_weight);
    if (WEIGHTS && p) {
      others = __syncthreads_or(others);
      if (blocks > 1 && threadIdx.x < blocks) store_cluster(cluster_address(&s.peer_others[rank], threadIdx.x), others ? 1u : 0u);
    }
    meet();
    if (WEIGHTS && p && blocks > 1)
      for (int q = 0; q < blocks; ++q) others = others || s.peer_others[q];
    reach(target, p, others);
    if (s.bin < 0) return;
    const int bin = s.bin;
    uint64_t left = s.target - s.before;
    uint32_t low = 0xFFFFFFFFu, high = 0;
    // the bin's keys go to the list, if it is free and they are not too many
    const bool had = listed;
    if (!had) {
      if (threadIdx.x == 0) s.listed = 0;
      __syncthreads();
    }
    each([&](float l, uint32_t key) {
      if (key > tau && bin_of(l) == bin) {
        low = min(low, key), high = max(high, key);
        if (!had) {
          const int at = atomicAdd(&s.listed, 1);
          if (at < kList) s.list[at] = key;
        }
      }
    });
    if (mine && bin_of(value_of(tau)) == bin) low = min(low, tau), high = max(high, tau);
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    const int lane = threadIdx.x & 31;
    if (lane == 0) s.warp_b[threadIdx.x >> 5] = low, s.warp_c[threadIdx.x >> 5] = high;
    __syncthreads();
    listed = had || s.listed <= kList;
    low = __reduce_min_sync(0xffffffffu, lane < kWarps ? s.warp_b[lane] : 0xFFFFFFFFu);
    high = __reduce_max_sync(0xffffffffu, lane < kWarps ? s.warp_c[lane] : 0);
    if (blocks > 1) {
      if (threadIdx.x < blocks) {
        store_cluster(cluster_address(&s.peer_low[rank], threadIdx.x), low);
        store_cluster(cluster_address(&s.peer_high[rank], threadIdx.x), high);
      }
      sync();
      for (int q = 0; q < blocks; ++q) low = min(low, s.peer_low[q]), high = max(high, s.peer_high[q]);
    }
    while (low < high) {
      const int shift = max(0, 32 - __clz(high - low) - 11);
      each([&](float l, uint32_t key) {
        if (key <= tau || key < low || key > high) return;
        const uint64_t w = WEIGHTS ? weight(l) : 1;
        if (!WEIGHTS || w) add<WEIGHTS>(static_cast<int>((high - key) >> shift), w);
      });
      if (mine && tau >= low && tau <= high) add<WEIGHTS>(static_cast<int>((high - tau) >> shift), group_weight);
      meet();
      reach(left, nullptr, false);
      left -= s.before;
      high -= static_cast<uint32_t>(s.bin) << shift;
      const uint32_t span = (1u << shift) - 1u;
      if (high - low > span) low = high - span;
    }
    listed = had;
    tau = low;
    tie_weight = weight(value_of(tau));
    ties = static_cast<uint32_t>(WEIGHTS ? (left + tie_weight - 1) / max(tie_weight, uint64_t(1)) : left);
    __syncthreads();
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  constexpr int kVec = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / a.blocks;
  const int rank = static_cast<int>(blockIdx.x % a.blocks);
  if (a.blocks > 1) cluster_arrive();  // this block has started: its shared memory may be written
  for (int i = threadIdx.x; i < 1 << (kStepBits - 1); i += kThreads)
    reinterpret_cast<uint4*>(s.power)[i] = reinterpret_cast<const uint4*>(kPowers.t)[i];
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
  if (threadIdx.x == 0) s.listed = 0;
  pdl_wait();
  pdl_trigger();
  const T* const row = static_cast<const T*>(a.logits) + b * a.ld;
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T) % kVec);
  const int all = (skew + a.V + kVec - 1) / kVec, per = (all + a.blocks - 1) / a.blocks;
  const int v0 = min(all, rank * per), count = min(all, v0 + per) - v0;
  Row<T> r = {s, row, a.V, skew, v0, count, rank, a.blocks, 0.0f, 0.0f, 0.0f, 0.0f, kNone, 0, 0, false};
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.0f, q = a.min_p ? a.min_p[b] : 0.0f;
  float u = a.uniform[b];
  const bool top_k = k > 0 && k < a.V, top_p = p < 1.0f, greedy = !(t >= 0x1p-100f);
  float own = -INFINITY;  // this thread's largest logit
  float away = -INFINITY;
  const bool counted = sizeof(T) == 2 && !greedy && (top_k || top_p) && per * kVec > kList;
  if (counted) __syncthreads();  // the counts are 0
  r.pieces([&](const uint4& w, float m) {
    own = fmaxf(own, m);
    if constexpr (sizeof(T) == 2)
      if (counted) r.count_values(w, away);
  });
  uint32_t best = __reduce_max_sync(0xffffffffu, key_of(own)), far = __reduce_max_sync(0xffffffffu, key_of(away));
  if (lane == 0) s.warp_b[warp] = best, s.warp_c[warp] = far;
  __syncthreads();
  best = __reduce_max_sync(0xffffffffu, lane < kWarps ? s.warp_b[lane] : 0);
  far = __reduce_max_sync(0xffffffffu, lane < kWarps ? s.warp_c[lane] : 0);
  if (s.listed > kList) far = 0xFFFFFFFFu;  // too many rare ones
  if (a.blocks > 1) {
    cluster_wait();
    if (threadIdx.x < a.blocks) {
      store_cluster(cluster_address(&s.peer_top[rank], threadIdx.x), best);
      store_cluster(cluster_address(&s.peer_far[rank], threadIdx.x), far);
    }
    r.sync();
    for (int i = 0; i < a.blocks; ++i) best = max(best, s.peer_top[i]), far = max(far, s.peer_far[i]);
  } else {
    __syncthreads();
  }
  if (best <= kNone) {
    if (rank == 0 && threadIdx.x == 0) a.tokens[b] = -1;
    return;
  }
  r.top = value_of(best);
  uint64_t least = 0;  // weight of a kept token
  bool valued = false, table = false;  // the weights of values are there; and those of no others than are kept
  if (greedy) {
    r.tau = best, r.ties = 1, r.tie_weight = kOne;
  } else {
    const float limited = fminf(t, 0x1p100f);
    const float high = 1.44269502f, low = 1.92596299e-8f;  // log2(e)
    r.ch = __fdiv_rn(high, limited);
    r.cl = __fdiv_rn(__fadd_rn(__fmaf_rn(-r.ch, limited, high), low), limited);
    r.step = r.ch * 44.3614196f;  // 64 ln 2: 64 bins where the weight falls by e
    // a bound is a little lower than its arithmetic in 32 bits says
    const auto below = [&](float units, float scale) { return r.top - units / scale * 1.0001f - fabsf(r.top) * 0x1p-20f; };
    const float part = fmaxf(p, 0.0f);
    bool cut = false;
    if constexpr (sizeof(T) == 2) {
      // values of magnitude 2^7 and more are not counted: none may have a weight
      valued = isfinite(r.top) && far != 0xFFFFFFFFu && !((r.top - value_of(far)) * r.ch < 46.0f);
      if (!counted) {  // without counts, a table of all values pays for long rows only
        valued = valued && per * kVec > 2 * kValues;
        if (valued) {
          for (int i = threadIdx.x; i <= 2 * static_cast<int>(kSide); i += kThreads)
            s.weight[bin_place(i)] = bin_value(i) > r.top ? 0 : r.weight(bin_value(i));
          __syncthreads();
        }
      } else if (valued) {
        cut = r.cut_values(top_k ? k : 0, top_p ? &part : nullptr, far > kNone);
      } else {
        for (int i = threadIdx.x; i < kValues; i += kThreads) s.count[i] = 0;
      }
      if (counted) __syncthreads();
    }
    table = valued && (cut || !counted);
    if (!cut) {
      if (top_k) {
        // a row's blocks have like numbers of tokens, and agree on what they do together
        if (per * kVec <= kList) {
          r.gather(-INFINITY);
        } else if (k <= a.blocks * kThreads / 2) {
          if (own > -INFINITY) r.template add<false>(r.bin_of(own), 1);
          r.meet();
          r.reach(k, nullptr, false);
          const int bin = s.bin;
          if (bin >= 0 && bin < kBins - 1 && isfinite(r.top)) r.gather(below(bin + 1.0f, r.step));
        }
        r.template cut<false>(nullptr, k);
      }
      if (top_p) {
        if (!top_k && per * kVec <= kList) r.gather(-INFINITY);
        r.template cut<true>(&part);
      }
    }
    if (q > 0.0f) {
      bool rest = false;
      least = kOne;
      if (q < 1.0f) least = part_of(q, kOne, rest);
      least += rest;  // the least whole number that is at least min_p
      if (r.tie_weight < least) r.ties = 0;
      table = false;
    }
  }

  // the kept weight of a piece, without the tokens of key tau; how many of these it has
  const float last_kept = value_of(r.tau);
  const auto kept = [&](const uint4& piece, float m, uint64_t& sum, uint32_t& same) {
    if (!(m >= last_kept) || m == -INFINITY) return;
    if constexpr (sizeof(T) == 2) {
      if (table && last_kept != 0.0f) {  // by the table alone
        const uint32_t tie = __float_as_uint(last_kept) >> 16;
        const uint32_t w[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const uint32_t b = e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu;
          const int place = value_place(b);
          if (place >= 0) sum += s.weight[place];
          else if (__uint_as_float(b << 16) > last_kept) sum += r.weight(__uint_as_float(b << 16));
          same += b == tie;
        }
        return;
      }
    }
    float v[kVec];
    Row<T>::unpack(piece, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (v[e] > last_kept) {
        const int place = sizeof(T) == 2 && valued ? value_place(__float_as_uint(v[e]) >> 16) : -1;
        uint64_t x;
        if (place >= 0) x = s.weight[place];
        else x = r.weight(v[e]);
        if (x >= least) sum += x;
      }
      same += v[e] == last_kept;
    }
  };
  // of every warp's segment
  uint64_t sum = 0;
  uint32_t same = 0;
  r.pieces([&](const uint4& piece, float m) { kept(piece, m, sum, same); });
  sum = warp_sum(sum);
  same = warp_sum(same);
  if (lane == 0) s.warp_a[warp] = sum, s.warp_b[warp] = same;
  __syncthreads();
  sum = lane < kWarps ? s.warp_a[lane] : 0, same = lane < kWarps ? s.warp_b[lane] : 0;
  const uint64_t block_sum = warp_sum(sum);
  const uint32_t block_same = warp_sum(same);
  uint64_t total = 0, prior = 0;
  uint32_t seen = 0, seen_prior = 0;
  if (a.blocks > 1) {
    if (threadIdx.x < a.blocks) {
      store_cluster(cluster_address(&s.peer_sum[rank], threadIdx.x), block_sum);
      store_cluster(cluster_address(&s.peer_same[rank], threadIdx.x), block_same);
    }
    r.sync();
    for (int i = 0; i < a.blocks; ++i) {
      if (i == rank) prior = total, seen_prior = seen;
      const uint32_t here = min(s.peer_same[i], r.ties - min(r.ties, seen));
      seen += here;
      total += s.peer_sum[i] + here * r.tie_weight;
    }
  } else {
    total = block_sum + min(block_same, r.ties) * r.tie_weight;
  }
  bool rest;
  u = u >= 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
  uint64_t target = part_of(u, total, rest) + 1;
  if (target <= prior) return;
  target -= prior;
  uint32_t free_ties = r.ties - min(r.ties, seen_prior);  // kept tokens of key tau from here on
  // Of 32 runs' sums and ties in order, a run a lane: the one in which the target lies, or -1; the target and the free ties
  // become those from that run, or from behind all of them, on.
  const auto find = [&](uint64_t run_sum, uint32_t run_same) {
    const uint32_t upto_same = warp_scan(run_same, lane), before_same = upto_same - run_same;
    run_sum += min(run_same, free_ties - min(free_ties, before_same)) * r.tie_weight;
    const uint64_t upto = warp_scan(run_sum, lane);
    const unsigned reached = __ballot_sync(0xffffffffu, upto >= target);
    const int at = reached ? __ffs(reached) - 1 : 31;
    target -= __shfl_sync(0xffffffffu, reached ? upto - run_sum : upto, at);
    const uint32_t gone = __shfl_sync(0xffffffffu, reached ? before_same : upto_same, at);
    free_ties -= min(free_ties, gone);
    return reached ? at : -1;
  };
  const int w = find(sum, same);
  if (w < 0) return;  // another block's
  // The segment's rounds of 32 pieces are dealt out to the warps, and the first of them looks into the one it is.
  int first, last;
  r.segment(w, first, last);
  const int rounds = (last - first + 31) / 32;
  uint64_t* const round_sum = s.total;
  uint32_t* const round_same = s.lo;
  for (int i = warp; i < rounds; i += kWarps) {
    uint64_t x = 0;
    uint32_t n = 0;
    const int at = first + 32 * i + lane;
    if (at < last) {
      uint4 piece = r.raw(at);
      float m;
      r.clean(at, piece, m);
      kept(piece, m, x, n);
    }
    x = warp_sum(x);
    n = warp_sum(n);
    if (lane == 0) round_sum[i] = x, round_same[i] = n;
  }
  __syncthreads();
  if (warp != 0) return;
  int round = -1;
  for (int i = 0; round < 0 && i < rounds; i += 32) {
    const int at = find(i + lane < rounds ? round_sum[i + lane] : 0, i + lane < rounds ? round_same[i + lane] : 0);
    if (at >= 0) round = i + at;
  }
  if (round < 0) return;
  const int i = first + 32 * round + lane;
  float v[kVec], m = -INFINITY;
#pragma unroll
  for (int e = 0; e < kVec; ++e) v[e] = -INFINITY;
  if (i < last) {
    uint4 piece = r.raw(i);
    r.clean(i, piece, m);
    Row<T>::unpack(piece, v);
  }
  uint32_t n = 0;
#pragma unroll
  for (int e = 0; e < kVec; ++e) n += v[e] == last_kept;
  uint32_t free = free_ties - min(free_ties, warp_scan(n, lane) - n);
  uint64_t part[kVec], whole = 0;
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    part[e] = v[e] > last_kept ? r.weight(v[e]) : 0;
    if (part[e] < least) part[e] = 0;
    if (v[e] == last_kept && free > 0) part[e] = r.tie_weight, --free;
    whole += part[e];
  }
  uint64_t x = warp_scan(whole, lane) - whole;
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    if (x < target && target <= x + part[e]) a.tokens[b] = static_cast<int32_t>(static_cast<int64_t>(v0 + i) * kVec - skew + e);
    x += part[e];
  }
}

// Whether the current device runs clusters of kMaxBlocks, more than every device does: looked up once.
template <typename T>
moe_status_t large_clusters(bool& run) {
  static std::atomic<int> known[64];  // 0: not asked yet, 1: no, 2: yes
  int dev = 0;
  MOE_CUDA(cudaGetDevice(&dev));
  int answer = known[dev & 63].load(std::memory_order_relaxed);
  if (answer == 0) {
    MOE_CUDA(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxBlocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxBlocks, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    MOE_CUDA(cudaOccupancyMaxActiveClusters(&clusters, reinterpret_cast<const void*>(sample_kernel<T>), &cfg));
    answer = clusters >= 4 ? 2 : 1;
    known[dev & 63].store(answer, std::memory_order_relaxed);
  }
  run = answer == 2;
  return MOE_OK;
}

// Blocks of a row: more while they all fit the SMs twice and their parts are longer than 4096 tokens; 16 where few rows leave
// half of the SMs free (129021 BF16 logits by top-p: one to four rows 20.4 -> 18.4 us, eight 20.6 -> 24.2; 40000 logits,
// of which a block then has too few to count them by value, 17.0 -> 19.3).
template <typename T>
moe_status_t blocks_of(int B, int V, int& n) {
  n = 1;
  while (n < 8 && static_cast<int64_t>(B) * n * 2 <= 2 * num_sms() && V > 4096 * n) n *= 2;
  if (n == 8 && B * kMaxBlocks <= num_sms() / 2 && V > 4096 * kMaxBlocks) {
    bool large = false;
    const moe_status_t st = large_clusters<T>(large);
    if (st != MOE_OK) return st;
    if (large) n = kMaxBlocks;
  }
  return MOE_OK;
}

template <typename T>
moe_status_t launch_sample(SampleArgs a, int B, cudaStream_t s) {
  MOE_CUDA(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared)));
  const moe_status_t cut = blocks_of<T>(B, a.V, a.blocks);
  if (cut != MOE_OK) return cut;
  return launch_clusters(sample_kernel<T>, a.blocks, dim3(static_cast<unsigned>(B) * a.blocks), dim3(kThreads), sizeof(Shared), s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_sample(const void* logits, int32_t logits_dtype, int64_t ld_logits, int32_t B, int32_t V,
                                   const float* uniform, const float* temperature, const int32_t* top_k, const float* top_p,
                                   const float* min_p, int32_t* tokens, moe_stream_t stream) {
  MOE_CHECK(B >= 0 && V > 0 && ld_logits >= V, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(logits_dtype == MOE_LOGITS_F32 || logits_dtype == MOE_LOGITS_BF16, MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(V <= kMaxVocab && B <= (1 << 24), MOE_ERR_UNSUPPORTED_SHAPE);
  if (B == 0) return MOE_OK;
  MOE_CHECK(logits && uniform && tokens, MOE_ERR_INVALID_ARGUMENT);
  const size_t size = logits_dtype == MOE_LOGITS_F32 ? 4 : 2;
  MOE_CHECK(reinterpret_cast<uintptr_t>(logits) % size == 0 &&
                ((reinterpret_cast<uintptr_t>(uniform) | reinterpret_cast<uintptr_t>(temperature) | reinterpret_cast<uintptr_t>(top_k) |
                  reinterpret_cast<uintptr_t>(top_p) | reinterpret_cast<uintptr_t>(min_p) | reinterpret_cast<uintptr_t>(tokens)) & 3) == 0,
            MOE_ERR_MISALIGNED);
  const size_t n = static_cast<size_t>(B) * 4;
  MOE_CHECK(!overlaps(tokens, n, logits, (static_cast<size_t>(B - 1) * ld_logits + V) * size), MOE_ERR_OVERLAP);
  for (const void* p : {static_cast<const void*>(uniform), static_cast<const void*>(temperature), static_cast<const void*>(top_k),
                        static_cast<const void*>(top_p), static_cast<const void*>(min_p)})
    MOE_CHECK(!overlaps(tokens, n, p, n), MOE_ERR_OVERLAP);
  const SampleArgs a = {logits, uniform, temperature, top_p, min_p, top_k, tokens, ld_logits, V, 1};
  if (logits_dtype == MOE_LOGITS_F32) return launch_sample<uint32_t>(a, B, as_stream(stream));
  return launch_sample<uint16_t>(a, B, as_stream(stream));
}
