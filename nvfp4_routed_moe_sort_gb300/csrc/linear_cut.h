// How moe_linear_fp4 cuts a product into blocks and clusters; the rule is in linear.cu.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kLinWarps = 16;   // most warps of a block, and of an SM: 128 registers a thread
constexpr int kLinTokens = 16;  // most tokens of a block
constexpr int kLinChunk = 128;  // values of K that are summed on their own

// How rows are aligned: K % 256 == 0 (codes and scales to 16 bytes), K % 32 == 0 (codes to 16, scales to
// 2), or only K % 16 == 0 (codes to 8, scales to 1). Copies are of 16 aligned bytes; where a row
// starts inside such a piece, one more of them is copied and the row is read at its offset.
enum Align : int { kAlign256, kAlign32, kAlign16 };
__host__ __device__ constexpr int align_of(int K) { return K % 256 == 0 ? kAlign256 : K % 32 == 0 ? kAlign32 : kAlign16; }
__host__ __device__ constexpr int code_row(int align) { return align == kAlign16 ? 144 : 128; }
__host__ __device__ constexpr int scale_row(int align) { return align == kAlign256 ? 16 : 48; }
__host__ __device__ constexpr int stage_bytes(int align) { return 16 * (code_row(align) + scale_row(align)); }

struct LinCut {
  int tokens, warps, across, slices, slice, stages, buffers;
  int at_once;  // clusters that run at once
  int64_t groups;
};

// the cut of M x n_out (x 2 if gated) x K on `sms` SMs; false where none fits
bool cut_linear(int64_t M, int K, int n_out, bool gated, int align, int sms, LinCut* cut);

}  // namespace moe
