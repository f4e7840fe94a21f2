// fp4.cuh -- the 4-bit KV pool's element format: e2m1 codes, two a byte
// (element 2i in the low nibble of byte i, 2i + 1 in the high one), with one
// e4m3 block scale for every 16 elements of a row.  An element reads
// code * block_scale * tensor_scale.
//
// The product code * block_scale has at most 6 significant bits and lies in
// [2^-10, 2688], so it is exact in f16, in bf16 and in fp32: reading a pool
// into either 16-bit type loses nothing, and the tensor scale joins the logit
// scale or the output.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace pkx {

constexpr int kFp4Block = 16;  // elements per block scale

// Two e4m3 codes (the low 16 bits) as two f16 of the same values; a NaN code
// stays NaN.
__device__ __forceinline__ __half2 e4m3x2_to_f16x2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}

// The eight e2m1 codes of a word as four f16 pairs (out[i]: the codes of byte
// i, low nibble in the low half), by the hardware's converter.  Spreading the
// codes' bits by hand (sign to bit 15, magnitude to bits 11..9: the value
// times 2^-14) takes four integer operations a pair: decode over 64 x 8192
// keys ran in 162 us with that, 149 us with half of each, 138 us with the
// converter alone and shifts for its bytes, and 122 us with the bytes taken
// apart as operands, as here.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t x, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(x));
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a),
                            *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// The e2m1 code nearest to t / s for t >= 0 (ties to the even code, values
// past 6 s saturate), by comparing t with the midpoints of neighbouring
// values times s.  s is an e4m3 value, so the products (at most 7 significant
// bits) and with them the choice are exact; no quotient is rounded on the way.
__device__ __forceinline__ uint32_t e2m1_magnitude(float t, float s) {
  const bool b2 = t >= 1.75f * s;                     // codes 4..7
  const bool b1 = t >= (b2 ? 3.5f * s : 0.75f * s);   // 6, 7 or 2, 3
  const float odd = b2 ? (b1 ? 5.0f * s : 2.5f * s) : (b1 ? 1.25f * s : 0.25f * s);
  return (b2 ? 4u : 0u) | (b1 ? 2u : 0u) | (t > odd ? 1u : 0u);
}

}  // namespace pkx
