// fp8.cuh -- eight elements of an fp8 pool (FMT 1: e4m3, 2: e5m2; the values of
// include/pkx.h's PKX_KV_*) to and from bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace pkx {

// Eight fp8 codes (e4m3 for FMT 1, e5m2 for FMT 2) as eight bf16 of the same
// values (exact: every code is a bf16 value), in element order (the code in
// the lowest byte first).
template <int FMT>
__device__ __forceinline__ uint4 fp8x8_to_bf16x8(uint2 raw) {
  constexpr __nv_fp8_interpretation_t kind = FMT == 1 ? __NV_E4M3 : __NV_E5M2;
  const uint32_t w[2] = {raw.x, raw.y};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), kind));
    const float2 f = __half22float2(h);
    out[i] = pack_bf16(f.x, f.y);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Eight bf16 as the codes nearest to element / scale (an IEEE fp32 division),
// ties to even, saturating at the largest finite one.
template <int FMT>
__device__ __forceinline__ uint2 bf16x8_to_fp8x8(uint4 in, float scale) {
  constexpr __nv_fp8_interpretation_t kind = FMT == 1 ? __NV_E4M3 : __NV_E5M2;
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
    const float2 f = __bfloat1622float2(b);
    const float2 q = make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale));
    const uint32_t two = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, kind);
    out[i >> 1] |= (two & 0xFFFFu) << (16 * (i & 1));
  }
  return make_uint2(out[0], out[1]);
}

}  // namespace pkx
