// FP4 operands on mma.m16n8k16 (FP16 or BF16 in, FP32 sums): the conversions and instructions that the
// dense linear and the cache's attention share. Both read each 4-bit value once, for at most 16
// tokens or 32 query rows, and convert it in registers, where the legacy warp-level MMA takes its
// operands from. Per two values that is one conversion and one multiplication by the scale, either at
// half rate; the MMA pipe itself is busy a quarter of the time. An E2M1 code times an E4M3 scale
// has 6 significant bits between 2^-10 and 2688: exact in FP16, and in BF16.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

// the eight codes of a word, a byte's two to one register. Naming the word's bytes costs nothing;
// shifting and masking them out costs two more instructions of the pipe that converts.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t* f) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// the same with nothing to add to
__device__ __forceinline__ void mma_f16_first(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.0f));
}

// the same in BF16, for BF16 operands whose range does not fit FP16
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, const uint32_t* b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// two FP16 values as BF16; a code times its scale keeps its 6 significant bits
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 h0, h1;\n .reg .f32 f0, f1;\n mov.b32 {h0, h1}, %1;\n cvt.f32.f16 f0, h0;\n cvt.f32.f16 f1, h1;\n"
      " cvt.rn.bf16x2.f32 %0, f1, f0;\n}\n"
      : "=r"(r) : "r"(two));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t two) { return __uint_as_float(two << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t two) { return __uint_as_float(two & 0xFFFF0000u); }

// The power of two that takes a largest magnitude `amax` into [2^14, 2^15), and its inverse: BF16
// values so scaled are exact in FP16 from 2^-17 on. Zero and the
// smallest take 2^126; infinity and NaN (whose amax is that of the rest) stay what they are.
__device__ __forceinline__ void f16_range(float amax, float* up, float* down) {
  const int shift = min(14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), 126);
  *up = __uint_as_float(static_cast<uint32_t>(shift + 127) << 23);
  *down = __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
}

// a mask that is not zero where one of two BF16 values is so small that its FP16 form, scaled by f16_range's
// factor, may have lost bits of it
__device__ __forceinline__ uint32_t below_f16(uint32_t two_bf16, uint32_t two_f16) {
  const __half2 f = *reinterpret_cast<const __half2*>(&two_f16);
  const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162*>(&two_bf16);
  return __hlt2_mask(__habs2(f), __half2half2(__ushort_as_half(0x0080))) &  // 2^-17
         __hne2_mask(b, __bfloat162bfloat162(__ushort_as_bfloat16(0)));
}

}  // namespace moe
