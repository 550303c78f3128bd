// A paged key/value cache in NVFP4: the append that encodes new tokens into it and the
// attention of a decode step that reads it.
#include <math.h>

#include "common.cuh"
#include "host_util.h"

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

__device__ __forceinline__ float e2m1_to_f32(uint32_t c) {
  const uint32_t e = (c >> 1) & 3, m = c & 1;
  const float v = e == 0 ? 0.5f * m : (1.0f + 0.5f * m) * static_cast<float>(1u << (e - 1));
  return (c & 8) ? -v : v;
}

// One thread per 16-value block of one token's keys or values.
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(Cache c, const uint16_t* __restrict__ k_new,
                                                                   int64_t ld_k, const uint16_t* __restrict__ v_new,
                                                                   int64_t ld_v, const int64_t* __restrict__ slots,
                                                                   int64_t N, uint16_t* k_seen, uint16_t* v_seen,
                                                                   int32_t* dev_status) {
  pdl_wait();
  pdl_trigger();
  const int per_head = c.dim / kBlock, per_token = c.heads * per_head;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x;
  if (i >= N * 2 * per_token) return;
  const int64_t n = i / (2 * per_token);
  const int in_token = static_cast<int>(i - n * 2 * per_token);
  const int which = in_token >= per_token;
  const int b = in_token - which * per_token;
  const int head = b / per_head, blk = b - head * per_head;
  float v[16];
  load_block16(which ? v_new + n * ld_v + b * kBlock : k_new + n * ld_k + b * kBlock, v);
  uint32_t codes[2];
  const float g = c.g[which];
  const uint32_t q = quantize_block16(v, g, codes);
  const int64_t slot = slots[n];
  const int64_t page = slot >> c.page_shift;
  if (slot >= 0 && page < c.pages) {
    const int64_t row = (static_cast<int64_t>(head) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
    *reinterpret_cast<uint2*>(c.data[which] + page * c.data_page + row * (c.dim / 2) + blk * 8) =
        make_uint2(codes[0], codes[1]);
    c.sf[which][page * c.sf_page + row * per_head + blk] = static_cast<uint8_t>(q);
  } else if (slot >= 0 && dev_status && in_token == 0) {
    atomicOr(dev_status, MOE_DEV_BAD_INDEX);
  }
  uint16_t* seen = which ? v_seen : k_seen;
  if (seen) {
    const float s = e4m3_to_f32(q);
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t byte = codes[j >> 2] >> (8 * (j & 3));
      const float lo = __fdiv_rn(e2m1_to_f32(byte & 15) * s, g), hi = __fdiv_rn(e2m1_to_f32((byte >> 4) & 15) * s, g);
      o[j] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(lo))) |
             static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(hi))) << 16;
    }
    uint4* dst = reinterpret_cast<uint4*>(seen + (n * per_token + b) * kBlock);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

struct AttendArgs {
  const uint16_t* q;
  const int32_t* table;
  const int32_t* lens;
  uint16_t* out;
  float* lse;
  int32_t* dev_status;
  int64_t ld_q, ld_table;
  int q_len, q_heads, max_pages;
  float scale;
};

constexpr int kAttWarps = 8;

// One block per query row and head: warps take tokens in turn, each with its own running
// maximum and sum; lanes hold D / 32 neighbouring dimensions.
template <int D>
__global__ void __launch_bounds__(kAttWarps * 32) kv_attend_kernel(Cache c, AttendArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int P = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
  const int kvh = head / (a.q_heads / c.heads);
  const int64_t row = static_cast<int64_t>(b) * a.q_len + t;
  int len = max(a.lens[b], 0);
  const int64_t most = static_cast<int64_t>(a.max_pages) << c.page_shift;
  if (len > most) {
    len = static_cast<int>(most);
    if (a.dev_status && threadIdx.x == 0) atomicOr(a.dev_status, MOE_DEV_BAD_INDEX);
  }
  const int limit = len - (a.q_len - 1) + t;
  float q[P], o[P], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(a.q[row * a.ld_q + head * D + lane * P + i]) << 16);
    o[i] = 0.0f;
  }
  for (int j = warp; j < limit; j += kAttWarps) {
    const int page = a.table[b * a.ld_table + (j >> c.page_shift)];
    if (page < 0 || page >= c.pages) {
      if (a.dev_status && lane == 0) atomicOr(a.dev_status, MOE_DEV_BAD_INDEX);
      continue;
    }
    const int64_t place = (static_cast<int64_t>(kvh) << c.page_shift) + (j & ((1 << c.page_shift) - 1));
    float kv[2][P];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint8_t* d = c.data[w] + page * c.data_page + place * (D / 2) + lane * P / 2;
      const float s = e4m3_to_f32(c.sf[w][page * c.sf_page + place * (D / 16) + lane * P / 16]) / c.g[w];
#pragma unroll
      for (int i = 0; i < P; ++i) kv[w][i] = e2m1_to_f32((d[i / 2] >> (4 * (i & 1))) & 15) * s;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) s += q[i] * kv[0][i];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale;
    const float top = fmaxf(m, s), keep = expf(m - top), p = expf(s - top);
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = o[i] * keep + p * kv[1][i];
    m = top;
  }
  __shared__ float sm[kAttWarps], sl[kAttWarps], so[kAttWarps][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) so[warp][lane * P + i] = o[i];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, sm[w]);
  float total = 0.0f;
  for (int w = 0; w < kAttWarps; ++w) total += sl[w] == 0.0f ? 0.0f : sl[w] * expf(sm[w] - top);
  const int64_t at = row * a.q_heads + head;
  for (int i = threadIdx.x; i < D; i += kAttWarps * 32) {
    float v = 0.0f;
    for (int w = 0; w < kAttWarps; ++w)
      if (sl[w] != 0.0f) v += so[w][i] * expf(sm[w] - top);
    a.out[at * D + i] = __bfloat16_as_ushort(__float2bfloat16_rn(total == 0.0f ? 0.0f : v / total));
  }
  if (a.lse && threadIdx.x == 0) a.lse[at] = total == 0.0f ? -INFINITY : top + logf(total);
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
  const int64_t blocks = static_cast<int64_t>(N) * 2 * (width / kBlock);
  return launch_pdl(kv_append_kernel, dim3(static_cast<unsigned>((blocks + kAppendThreads - 1) / kAppendThreads)),
                    dim3(kAppendThreads), 0, as_stream(stream), c, k_new, ld_k, v_new, ld_v, slots,
                    static_cast<int64_t>(N), k_seen, v_seen, dev_status);
}

extern "C" size_t moe_kv_attend_workspace_bytes(const moe_kv_cache_t* cache, int32_t batch, int32_t q_len,
                                                int32_t num_q_heads, int32_t max_pages) {
  (void)cache, (void)batch, (void)q_len, (void)num_q_heads, (void)max_pages;
  return 0;
}

extern "C" moe_status_t moe_kv_attend(const moe_kv_cache_t* cache, const uint16_t* q, int64_t ld_q, int32_t batch,
                                      int32_t q_len, int32_t num_q_heads, const int32_t* page_table, int64_t ld_table,
                                      int32_t max_pages, const int32_t* seq_lens, float softmax_scale, uint16_t* out,
                                      float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                      moe_stream_t stream) {
  Cache c;
  moe_status_t st = check_cache(cache, &c);
  if (st != MOE_OK) return st;
  MOE_CHECK(batch >= 0 && q_len >= 1 && num_q_heads >= 1 && num_q_heads % c.heads == 0 && max_pages >= 0 &&
                ld_table >= max_pages && ld_q >= static_cast<int64_t>(num_q_heads) * c.dim && isfinite(softmax_scale),
            MOE_ERR_INVALID_ARGUMENT);
  MOE_CHECK(batch <= 65535 && q_len <= 65535 && (static_cast<int64_t>(max_pages) << c.page_shift) < (int64_t(1) << 31),
            MOE_ERR_UNSUPPORTED_SHAPE);
  const size_t need = moe_kv_attend_workspace_bytes(cache, batch, q_len, num_q_heads, max_pages);
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
  AttendArgs a = {q, page_table, seq_lens, out, lse, dev_status, ld_q, ld_table, q_len, num_q_heads, max_pages,
                  softmax_scale};
  const dim3 grid(num_q_heads, q_len, batch);
  return launch_pdl(c.dim == 64 ? kv_attend_kernel<64> : kv_attend_kernel<128>, grid, dim3(kAttWarps * 32), 0,
                    as_stream(stream), c, a);
}
