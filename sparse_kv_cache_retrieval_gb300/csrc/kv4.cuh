// The 4-bit record of one position of one KV head: 64 bytes of K codes
// (e2m1, two a byte), 64 bytes of V codes, 8 e4m3 scales each. A product code
// * scale has at most 6 significant bits and lies in [2^-10, 2688] (or is 0),
// so it is exact in fp16 and in bf16.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "spc_device.cuh"

namespace spc {

constexpr int kKv4Rec = SPC_KV4_RECORD;
constexpr int kKv4V = 64;            // byte offset of the V codes
constexpr int kKv4Scale = 128;       // of the K scales; the V scales are 8 bytes behind

// eight e2m1 codes of a word (lowest nibble first) as four fp16 pairs
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// eight fp32 values rounded to e2m1 (to nearest, ties to even, at most 6), the first in the lowest nibble
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float (&v)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}

// two e4m3 bytes (low half of w) as an fp16 pair
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xffffu))); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

// the fp16 of one e4m3 byte in both halves of a pair
__device__ __forceinline__ uint32_t e4m3_dup_f16(uint32_t byte) { return e4m3x2_to_f16((byte & 0xffu) * 0x0101u); }

}  // namespace spc
