// One token per row of logits: temperature, top-k, top-p, min-p, drawn by a given random number.
//
// With the row's tokens in the order of their logits (ties: the lower index first) and the weights
// w = exp((l - max) / temperature), each filter keeps a front part of that order: top-k its first k tokens,
// top-p the shortest part whose weights reach top_p times the sum over what top-k kept, min-p the tokens with
// w >= min_p. The token taken is, among the kept ones in the order of their INDEX, the first at which the
// cumulated weight passes u times their sum.
//
// So a row needs no sort, only the last kept logit and how many of the tokens that share it are kept. It
// is found by histograms over all values: 2048 bins of 1/64 in (max - l) / temperature, then the keys (the
// logits' bits in their order) of the bin in which the count or the weight is reached, 2048 ways a pass, until
// one key is left. BF16 logits mostly share one key by then.
//
// Weights are whole numbers, 2^44 for the largest logit, so that sums are exact in any order and every
// block of a row sees the same ones. A weight is right to 2^-36 of itself and to a unit: of 131072 tokens of like
// weight the border at which one token follows the next moves by less than 2^-19 of a token's width. (With
// float32 exponentials it moves by hundredths, and now and then another token is taken than in exact
// arithmetic.) exp2 in pieces: 4096 steps from a table, a polynomial of degree 2 for the rest, the argument
// carried as two floats.
//
// A row is spread over a cluster of blocks, each holding its part in shared memory; histograms and
// totals meet in distributed shared memory.
#include <math.h>

#include "cluster.cuh"
#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWarps = 32;
constexpr int kBins = 2048;
constexpr int kMaxBlocks = 8;
constexpr int kMaxVocab = 1 << 18;
constexpr uint32_t kNone = 0x007FFFFFu;  // the key of -infinity: such a token is never taken
constexpr uint64_t kOne = 1ull << 44;    // the weight of the largest logit

// 2^(-j / 4096) in units of 2^-44, by products of repeated square roots of 1/2 in 63-bit fixed point
struct Powers {
  uint64_t t[4096];
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
    uint64_t r[12] = {};  // r[b] = 2^(-2^b / 4096)
    uint64_t v = 1ull << 62;
    for (int b = 11; b >= 0; --b) r[b] = v = root(v);
    t[0] = 1ull << 63;
    for (int j = 1; j < 4096; ++j) {
      int b = 0;
      while (!((j >> b) & 1)) ++b;
      t[j] = mul(t[j & (j - 1)], r[b]);
    }
    for (int j = 0; j < 4096; ++j) t[j] = (t[j] + (1ull << 18)) >> 19;
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

struct Shared {
  uint64_t power[4096];
  uint64_t total[kBins];  // of every block's histogram
  uint32_t lo[kBins], hi[kBins];
  uint64_t warp_a[kWarps];
  uint32_t warp_b[kWarps], warp_c[kWarps];
  // what each block of the row has to tell, written by them; one array for each meeting, since blocks may be one apart
  uint64_t peer_best[kMaxBlocks], peer_sum[kMaxBlocks];
  uint32_t peer_low[kMaxBlocks], peer_high[kMaxBlocks], peer_same[kMaxBlocks];
  uint64_t before, sum, target;
  double below;  // temperature * ln(min_p), -infinity without one
  float ch, cl, step;
  int bin;
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

// One row's block. All members but data, count and rank are the same in all threads of all its blocks.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / sizeof(T);
  Shared& s;
  const uint4* data;  // this block's vectors
  int count, rank, blocks;
  float top;          // the largest logit
  uint32_t tau;       // kept: keys above tau, and the first `ties` tokens of key tau
  uint32_t ties;
  uint64_t tie_weight;

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

  // vectors of this warp: [first, last), a run of neighbours, a warp's width at a time
  __device__ __forceinline__ void segment(int warp, int& first, int& last) const {
    const int per = ((count + kWarps - 1) / kWarps + 31) / 32 * 32;
    first = min(count, warp * per);
    last = min(count, first + per);
  }

  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    int first, last;
    segment(threadIdx.x >> 5, first, last);
    for (int i = first + (threadIdx.x & 31); i < last; i += 32) {
      float v[kVec];
      unpack(data[i], v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) f(v[e], key_of(v[e]));
    }
  }

  __device__ __forceinline__ uint64_t weight(float l) const {
    if (l == top) return kOne;
    const float d = top - l;
    const float p = d * s.ch;
    if (!(p < 46.0f)) return 0;
    // what d and p lost by rounding
    const float back = top - d;
    const float dl = (top - (d + back)) + (back - l);
    float e = fmaf(d, s.ch, -p);
    e = fmaf(d, s.cl, e);
    e = fmaf(dl, s.ch, e);
    const float magic = 0x1.8p11f;  // rounds to multiples of 2^-12
    const float k = p + magic;
    const int steps = static_cast<int>(__float_as_uint(k) - __float_as_uint(magic));
    const float z = (p - (k - magic)) + e;
    // 2^-z - 1, |z| <= 2^-13 and a bit: the cubic term is below 2^-43
    const float x = z * fmaf(z, 0.240226507f, -0.693147181f);
    const int part = __float2int_rn(x * 0x1p44f);
    const uint64_t t = s.power[steps & 4095];
    const int64_t w = static_cast<int64_t>(t) + ((static_cast<int64_t>(static_cast<int32_t>(t >> 13)) * part) >> 31);
    return static_cast<uint64_t>(w) >> (steps >> 12);
  }

  __device__ __forceinline__ int bin_of(float l) const {
    return min(kBins - 1, static_cast<int>(fminf((top - l) * s.step, 4096.0f)));
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
  __device__ __forceinline__ void reach(uint64_t target, const float* p) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t a = s.total[2 * threadIdx.x], b = s.total[2 * threadIdx.x + 1];
    const uint64_t upto = warp_scan(a + b, lane);
    if (lane == 31) s.warp_a[warp] = upto;
    if (threadIdx.x == 0) s.bin = -1;
    __syncthreads();
    const uint64_t warps = warp_scan(s.warp_a[lane], lane);
    const uint64_t all = __shfl_sync(0xffffffffu, warps, 31);
    const uint64_t prior = __shfl_sync(0xffffffffu, warps, warp == 0 ? 0 : warp - 1);
    if (p) {
      bool rest;
      target = part_of(*p, all, rest);
      target += rest;
      if (target == 0) target = 1;
    }
    const uint64_t x = (warp == 0 ? 0 : prior) + upto - (a + b);
    if (x < target && target <= x + a) {
      s.bin = 2 * threadIdx.x, s.before = x, s.target = target;
    } else if (x + a < target && target <= x + a + b) {
      s.bin = 2 * threadIdx.x + 1, s.before = x + a, s.target = target;
    }
    __syncthreads();
  }

  // Cuts the kept tokens to the shortest front part whose count or weight reaches the target.
  template <bool WEIGHTS>
  __device__ void cut(uint64_t target, const float* p) {
    const bool group = WEIGHTS && ties > 0;            // kept tokens of key tau,
    const bool mine = group && rank == 0 && threadIdx.x == 0;  // added by one thread
    const uint64_t group_weight = ties * tie_weight;
    each([&](float l, uint32_t key) {
      if (key <= tau) return;
      const uint64_t w = WEIGHTS ? weight(l) : 1;
      if (!WEIGHTS || w) add<WEIGHTS>(bin_of(l), w);
    });
    if (mine) add<WEIGHTS>(bin_of(value_of(tau)), group_weight);
    meet();
    reach(target, p);
    if (s.bin < 0) return;
    const int bin = s.bin;
    uint64_t left = s.target - s.before;
    uint32_t low = 0xFFFFFFFFu, high = 0;
    each([&](float l, uint32_t key) {
      if (key > tau && bin_of(l) == bin) low = min(low, key), high = max(high, key);
    });
    if (mine && bin_of(value_of(tau)) == bin) low = min(low, tau), high = max(high, tau);
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if ((threadIdx.x & 31) == 0) s.warp_b[threadIdx.x >> 5] = low, s.warp_c[threadIdx.x >> 5] = high;
    __syncthreads();
    low = __reduce_min_sync(0xffffffffu, s.warp_b[threadIdx.x & 31]);
    high = __reduce_max_sync(0xffffffffu, s.warp_c[threadIdx.x & 31]);
    if (threadIdx.x < blocks) {
      store_cluster(cluster_address(&s.peer_low[rank], threadIdx.x), low);
      store_cluster(cluster_address(&s.peer_high[rank], threadIdx.x), high);
    }
    sync();
    for (int q = 0; q < blocks; ++q) low = min(low, s.peer_low[q]), high = max(high, s.peer_high[q]);
    while (low < high) {
      const int shift = max(0, 32 - __clz(high - low) - 11);
      each([&](float l, uint32_t key) {
        if (key <= tau || key < low || key > high) return;
        const uint64_t w = WEIGHTS ? weight(l) : 1;
        if (!WEIGHTS || w) add<WEIGHTS>(static_cast<int>((high - key) >> shift), w);
      });
      if (mine && tau >= low && tau <= high) add<WEIGHTS>(static_cast<int>((high - tau) >> shift), group_weight);
      meet();
      reach(left, nullptr);
      left -= s.before;
      high -= static_cast<uint32_t>(s.bin) << shift;
      const uint32_t span = (1u << shift) - 1u;
      if (high - low > span) low = high - span;
    }
    tau = low;
    tie_weight = weight(value_of(tau));
    ties = static_cast<uint32_t>(WEIGHTS ? (left + tie_weight - 1) / max(tie_weight, uint64_t(1)) : left);
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(SampleArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& s = *reinterpret_cast<Shared*>(raw);
  uint4* const data = reinterpret_cast<uint4*>(raw + sizeof(Shared));
  constexpr int kVec = 16 / sizeof(T);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t b = blockIdx.x / a.blocks;
  const int rank = static_cast<int>(blockIdx.x % a.blocks);
  for (int i = threadIdx.x; i < 2048; i += kThreads)
    reinterpret_cast<uint4*>(s.power)[i] = reinterpret_cast<const uint4*>(kPowers.t)[i];
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
  pdl_wait();
  pdl_trigger();
  const float t = a.temperature ? a.temperature[b] : 1.0f;
  const bool greedy = !(t >= 0x1p-100f);
  if (threadIdx.x == kThreads - 1) {
    const double c = 1.4426950408889634074 / fmin(static_cast<double>(t), 0x1p100);
    s.ch = static_cast<float>(c);
    s.cl = static_cast<float>(c - s.ch);
    s.step = s.ch * 44.3614196f;  // 64 ln 2: 64 bins where the weight falls by e
    const float q = a.min_p ? a.min_p[b] : 0.0f;
    s.below = q > 0.0f ? fmin(static_cast<double>(t), 0x1p100) * log(static_cast<double>(q)) : -INFINITY;
  }
  // This block's part of the row, from the 16-byte piece in which the row begins: places outside the row and
  // NaN become -infinity. Vectors that lie inside are read whole, the row's ends by the value.
  const T* const row = static_cast<const T*>(a.logits) + b * a.ld;
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T) % kVec);
  const int vectors = (skew + a.V + kVec - 1) / kVec, per = (vectors + a.blocks - 1) / a.blocks;
  const int v0 = min(vectors, rank * per), count = min(vectors, v0 + per) - v0;
  uint64_t best = 0;  // key, then the lower index
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const int64_t at = static_cast<int64_t>(v0 + i) * kVec - skew;  // the vector's first token
    uint4 u;
    if (at >= 0 && at + kVec <= a.V) {
      u = __ldg(reinterpret_cast<const uint4*>(row + at));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          const uint32_t l = at + 2 * e >= 0 && at + 2 * e < a.V ? row[at + 2 * e] : 0xFF80u;
          const uint32_t h = at + 2 * e + 1 >= 0 && at + 2 * e + 1 < a.V ? row[at + 2 * e + 1] : 0xFF80u;
          w[e] = l | h << 16;
        } else {
          w[e] = at + e >= 0 && at + e < a.V ? row[at + e] : 0xFF800000u;
        }
      }
      u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    float v[kVec];
    Row<T>::unpack(u, v);
    bool nan = false;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (isnan(v[e])) {
        nan = true;
        v[e] = -INFINITY;
      }
      const uint64_t k = static_cast<uint64_t>(key_of(v[e])) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(at + e));
      best = k > best ? k : best;
    }
    if (nan) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2)
          w[e] = __float_as_uint(v[2 * e]) >> 16 | (__float_as_uint(v[2 * e + 1]) & 0xFFFF0000u);
        else
          w[e] = __float_as_uint(v[e]);
      }
      u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    data[i] = u;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t k = __shfl_xor_sync(0xffffffffu, best, o);
    best = k > best ? k : best;
  }
  if (lane == 0) s.warp_a[warp] = best;
  __syncthreads();
  Row<T> r = {s, data, count, rank, a.blocks, 0.0f, kNone, 0, 0};
  if (warp == 0) {
    best = s.warp_a[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t k = __shfl_xor_sync(0xffffffffu, best, o);
      best = k > best ? k : best;
    }
    if (lane < a.blocks) store_cluster(cluster_address(&s.peer_best[rank], lane), best);
  }
  r.sync();
  best = 0;
  for (int q = 0; q < a.blocks; ++q) best = s.peer_best[q] > best ? s.peer_best[q] : best;
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  if (top_key <= kNone || greedy) {
    if (rank == 0 && threadIdx.x == 0)
      a.tokens[b] = top_key <= kNone ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
    return;
  }
  r.top = value_of(top_key);

  const int k = a.top_k ? a.top_k[b] : 0;
  if (k > 0 && k < a.V) r.template cut<false>(static_cast<uint64_t>(k), nullptr);
  const float p = a.top_p ? fmaxf(a.top_p[b], 0.0f) : 1.0f;
  if (a.top_p && a.top_p[b] < 1.0f) r.template cut<true>(0, &p);
  if (s.below > -INFINITY) {
    const double least = fmin(static_cast<double>(r.top) + s.below, static_cast<double>(r.top));
    const uint32_t key = key_of(__double2float_ru(least));
    if (key > r.tau) r.tau = key - 1, r.ties = 0;
  }

  // the kept weight of every warp's segment, without the tokens of key tau; how many of these it has
  uint64_t sum = 0;
  uint32_t same = 0;
  r.each([&](float l, uint32_t key) {
    if (key > r.tau) sum += r.weight(l);
    same += key == r.tau;
  });
  sum = warp_sum(sum);
  same = warp_sum(same);
  __syncthreads();
  if (lane == 0) s.warp_a[warp] = sum, s.warp_b[warp] = same;
  __syncthreads();
  sum = s.warp_a[lane], same = s.warp_b[lane];
  const uint64_t block_sum = warp_sum(sum);
  const uint32_t block_same = warp_sum(same);
  if (threadIdx.x < a.blocks) {
    store_cluster(cluster_address(&s.peer_sum[rank], threadIdx.x), block_sum);
    store_cluster(cluster_address(&s.peer_same[rank], threadIdx.x), block_same);
  }
  r.sync();
  if (warp != 0) return;
  uint64_t total = 0, prior = 0;
  uint32_t seen = 0, seen_prior = 0;
  for (int q = 0; q < a.blocks; ++q) {
    if (q == rank) prior = total, seen_prior = seen;
    const uint32_t here = min(s.peer_same[q], r.ties - min(r.ties, seen));
    seen += here;
    total += s.peer_sum[q] + here * r.tie_weight;
  }
  bool rest;
  float u = a.uniform[b];
  u = u >= 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;
  uint64_t target = part_of(u, total, rest) + 1;
  if (target <= prior) return;
  target -= prior;
  uint32_t free_ties = r.ties - min(r.ties, seen_prior);  // kept tokens of key tau from here on
  // the warp's segment in which it lies
  const uint32_t upto_same = warp_scan(same, lane), before_same = upto_same - same;
  sum += min(same, free_ties - min(free_ties, before_same)) * r.tie_weight;
  const uint64_t upto = warp_scan(sum, lane);
  const unsigned reached = __ballot_sync(0xffffffffu, upto >= target);
  if (!reached) return;  // another block's
  const int w = __ffs(reached) - 1;
  target -= __shfl_sync(0xffffffffu, upto - sum, w);
  const uint32_t gone = __shfl_sync(0xffffffffu, before_same, w);
  free_ties -= min(free_ties, gone);
  int first, last;
  r.segment(w, first, last);
  for (int i0 = first; i0 < last; i0 += 32) {
    const int i = i0 + lane;
    float v[kVec];
    uint32_t n = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = -INFINITY;
    if (i < last) Row<T>::unpack(data[i], v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) n += key_of(v[e]) == r.tau;
    const uint32_t n_upto = warp_scan(n, lane);
    uint32_t free = free_ties - min(free_ties, n_upto - n);
    uint64_t part[kVec], own = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const uint32_t key = key_of(v[e]);
      part[e] = key > r.tau ? r.weight(v[e]) : 0;
      if (key == r.tau && free > 0) part[e] = r.tie_weight, --free;
      own += part[e];
    }
    const uint64_t own_upto = warp_scan(own, lane);
    if (own_upto >= target && own_upto - own < target) {
      uint64_t x = own_upto - own;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (x < target && target <= x + part[e])
          a.tokens[b] = static_cast<int32_t>(static_cast<int64_t>(v0 + i) * kVec - skew + e);
        x += part[e];
      }
    }
    const uint64_t all = __shfl_sync(0xffffffffu, own_upto, 31);
    if (all >= target) return;
    target -= all;
    free_ties -= min(free_ties, __shfl_sync(0xffffffffu, n_upto, 31));
  }
}

// Blocks of a row: enough that its part fits shared memory, and more while blocks are fewer than SMs
// and parts longer than 8192 tokens.
int blocks_of(int B, int V, int size) {
  int n = 1;
  while (n < kMaxBlocks && ((static_cast<int64_t>(V) + 8) * size > n * int64_t(144 << 10) ||
                            (static_cast<int64_t>(B) * n * 2 <= num_sms() && V > 8192 * n)))
    n *= 2;
  return n;
}

template <typename T>
moe_status_t launch_sample(SampleArgs a, int B, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(T);
  a.blocks = blocks_of(B, a.V, sizeof(T));
  const size_t smem = sizeof(Shared) + static_cast<size_t>((a.V + 2 * kVec - 2) / kVec / a.blocks + 1) * 16;
  MOE_CUDA(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024));
  return launch_clusters(sample_kernel<T>, a.blocks, dim3(static_cast<unsigned>(B) * a.blocks), dim3(kThreads), smem, s, a);
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
