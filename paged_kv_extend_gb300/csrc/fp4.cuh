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
#include <cuda_fp4.h>
#include <cuda_fp8.h>

namespace pkx {

constexpr int kFp4Block = 16;  // elements per block scale

// Two e4m3 codes (the low 16 bits) as two f16 of the same values; a NaN code
// stays NaN.
__device__ __forceinline__ __half2 e4m3x2_to_f16x2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}

// An e2m1 code becomes f16 in one of two ways.
//  * By bits: the sign to bit 15 and the three magnitude bits to bits 11..9
//    (the low exponent bits and the top mantissa bit), which is the value
//    times 2^-14, the subnormal 0.5 included: three or four integer
//    operations for a pair, one code in each half of the word.
//  * By the hardware's converter, which takes the two codes of a byte: one
//    instruction, but it issues once in about nine clocks a quarter SM.
// Measured on its own with the block scale and the product behind it
// (elements a clock and SM; the copy bandwidth delivers 41): 38.5 all by bits,
// 44.1 with two of a word's four pairs by the converter, 39.6 all by it.

// Code i of each 16-bit half of x (i = 0..3) as a pair of f16 times 2^-14.
template <int I>
__device__ __forceinline__ uint32_t e2m1_bits(uint32_t x) {
  constexpr uint32_t S = 0x80008000u, M = 0x0E000E00u;
  if constexpr (I == 3) return (x & S) | ((x >> 3) & M);
  else return ((x << (12 - 4 * I)) & S) | ((x << (9 - 4 * I)) & M);
}

// Eight e2m1 codes of a word as four f16 pairs times 2^-14: out[i] holds
// element i in its low half and element i + 4 in its high half.
__device__ __forceinline__ void e2m1x8_to_f16_pairs(uint32_t x, uint32_t (&out)[4]) {
  out[0] = e2m1_bits<0>(x);
  out[1] = e2m1_bits<1>(x);
  out[2] = e2m1_bits<2>(x);
  out[3] = e2m1_bits<3>(x);
}

// The two e2m1 codes of x's low byte as a pair of f16 (low nibble in the low half).
__device__ __forceinline__ uint32_t e2m1x2_convert(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(x));
  return r;
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
