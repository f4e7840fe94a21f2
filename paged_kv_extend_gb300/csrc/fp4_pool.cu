// fp4_pool.cu -- the KV write into a 4-bit pool and the read back of its rows.
//
// Write.  For a block of 16 consecutive elements x of a K or V row:
//   q = x / tensor_scale (IEEE fp32),  s = e4m3(max|q| / 6) (nearest, ties to
//   even, at most 448),  code = the e2m1 value nearest to q / s (ties to
//   even, saturating at 6).  s = 0 (a block of zeros, or one below the
//   smallest scale) stores zeros; a NaN in the block makes s NaN, so that the
//   block reads NaN instead of hiding it.
// Read.  element = bf16(code * s * tensor_scale): the first product is exact
//   in fp32, the second rounds to fp32, then once to bf16.
//
// Both move each byte once and are bounded by HBM: the write takes 2 bytes
// and stores 0.5625 bytes an element, the read back the reverse.  A thread is
// given one place in a token's rows (head and block, of K or of V), found by
// division once, and walks over the tokens with it: no division per block, and
// a warp's accesses are runs of whole rows.  Several tokens' loads are in
// flight per thread; the grid is one resident wave.  Measured for 8 KV heads of
// 128 (K and V): write of 16384 tokens 18 us with a power-of-two tensor scale
// (4.7 TB/s, 0.70 of the copy bandwidth; 63 % of the issue slots) and 41 us with
// another one (2.1 TB/s, 76 % of the issue slots, which bound it); the write and
// the read back together 35 us, 70 us with a division per block; read back of
// 131072 rows 120 us (5.7 TB/s, 0.84 of the copy bandwidth), bound by HBM.
#include <algorithm>
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

constexpr int kFp4Threads = 256;
constexpr int kMaxPlaces = 1 << 20;  // grid y stays below its limit
constexpr int64_t kMaxRows = 1ll << 40;  // (offsets are 64-bit: more than any device holds)

// How `places` (a token's blocks or chunks) lie over CTAs: tokens of a CTA's
// pass, and CTAs (grid y) that share a token's places.
struct Fp4Places {
  int places, tokens, slices;
};

static Fp4Places fp4_places(int64_t places) {
  if (places >= kFp4Threads) return {(int)places, 1, (int)((places + kFp4Threads - 1) / kFp4Threads)};
  return {(int)places, kFp4Threads / (int)places, 1};
}

// This thread's place (-1: none) and first token; tokens advance by `step`.
__device__ __forceinline__ int fp4_place(const Fp4Places &p, int64_t &token, int64_t &step) {
  const int tt = p.slices > 1 ? 0 : (int)threadIdx.x / p.places;
  const int at = p.slices > 1 ? (int)(blockIdx.y * kFp4Threads + threadIdx.x)
                              : (int)threadIdx.x - tt * p.places;
  token = (int64_t)blockIdx.x * p.tokens + tt;
  step = (int64_t)gridDim.x * p.tokens;
  return tt < p.tokens && at < p.places ? at : -1;
}

// CTAs over the tokens: one resident wave of `kernel`, `unroll` tokens a thread.
template <typename K>
static dim3 wave_grid(K kernel, const Fp4Places &p, int64_t n_tokens, int unroll) {
  static PerDevice known;  // (one kernel per argument type)
  const int resident = resident_ctas(kernel, kFp4Threads, known);
  const int64_t cap = std::max<int64_t>((int64_t)num_sms_current_device() * resident / p.slices, 1);
  const int64_t need = (n_tokens + (int64_t)p.tokens * unroll - 1) / ((int64_t)p.tokens * unroll);
  return dim3((unsigned)std::max<int64_t>(std::min(need, cap), 1), (unsigned)p.slices);
}

// ------------------------------------------------------------------- write
struct Fp4WriteArgs {
  const uint4 *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;  // input strides in 16-byte chunks
  const int64_t *cache_loc;
  Fp4Pool pool;
  int64_t n_tokens;
  int hkv, nk, nv;  // heads; blocks of a K row, of a V row (0: K only)
  Fp4Places places;
  float k_scale, v_scale;
};

// Two fp32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t &>(r))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
        "l"(reinterpret_cast<uint64_t &>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(r))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return r;
}
// The e2m1 codes of two fp32 (nearest, ties to even, saturating) as a byte,
// `lo` in the low nibble.
__device__ __forceinline__ uint32_t e2m1x2_of(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

// The sign bits of four words of bf16 pairs, each at the top of its code's nibble.
__device__ __forceinline__ uint32_t sign_nibbles(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  auto two = [](uint32_t w) { return ((w >> 12) & 8u) | ((w >> 24) & 0x80u); };
  return two(a) | (two(b) << 8) | (two(c) << 16) | (two(d) << 24);
}

// One block of 16 bf16: the 8 code bytes and the scale code.  POW2: the
// tensor scale is a power of two in [2^-64, 2^64].  Then q = x / tensor_scale
// has bf16's 8 significant bits, and q / s, where it is not a midpoint of two
// e2m1 values m exactly, is at least 2^-10 away from it: |q - m s| is a
// multiple of the last place of q (2^-8 q at least) or of m s (2^-7 m s), and
// m >= 1/4.  So q * (1 / s) with its error of 2^-21 at most, rounded to a
// multiple of 2^-18 by adding and taking away 48, is on the right side of
// every midpoint and exactly on it where q / s is, and the hardware's rounding
// gives the definition's code.  Any other scale compares q with the midpoints
// times s (exact too, 2.9 times the instructions and 2.3 times the time).
template <bool POW2>
__device__ __forceinline__ uint2 quantise_block(const uint4 (&in)[2], float tensor_scale,
                                                uint8_t &scale_code) {
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  // largest magnitude by the bits (a NaN is largest of all)
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  const bool nan = top > 0x7F80u;
  const float xmax = __uint_as_float(top << 16);
  const float amax = POW2 ? xmax * (1.0f / tensor_scale) : __fdiv_rn(xmax, tensor_scale);
  const __nv_fp8_storage_t sc =
      __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f), __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(sc, __NV_E4M3)));
  scale_code = nan ? (uint8_t)0x7F : (uint8_t)sc;
  if (nan || s == 0.f) return make_uint2(0u, 0u);
  uint32_t out[2] = {0u, 0u};
  if constexpr (POW2) {
    const float r = __frcp_rn(s) * (1.0f / tensor_scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      const float2 y = add2(fma2(x, make_float2(r, r), make_float2(48.f, 48.f)),
                            make_float2(-48.f, -48.f));
      out[i >> 2] |= e2m1x2_of(y.x, y.y) << (8 * (i & 3));
    }
    // a negative value that rounds to zero keeps its sign (y is +0 there)
    const uint32_t neg[2] = {sign_nibbles(w[0], w[1], w[2], w[3]), sign_nibbles(w[4], w[5], w[6], w[7])};
    out[0] |= neg[0];
    out[1] |= neg[1];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
      const float q = __fdiv_rn(x, tensor_scale);
      out[i >> 3] |= (e2m1_magnitude(fabsf(q), s) | ((__float_as_uint(q) >> 28) & 8u)) << (4 * (i & 7));
    }
  }
  return make_uint2(out[0], out[1]);
}

constexpr int kWriteUnroll = 2;

__global__ void __launch_bounds__(kFp4Threads) set_kv_buffer_fp4_kernel(const Fp4WriteArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  int64_t token, step;
  int c = fp4_place(a.places, token, step);
  if (c < 0) return;
  const bool is_k = c < a.hkv * a.nk;
  if (!is_k) c -= a.hkv * a.nk;
  const int nb = is_k ? a.nk : a.nv;
  const int h = c / nb;
  c -= h * nb;
  const int64_t ts = is_k ? a.k_ts : a.v_ts;
  const uint4 *src = (is_k ? a.k + h * a.k_hs : a.v + h * a.v_hs) + 2 * c;
  const int64_t css = is_k ? a.pool.k_ss : a.pool.v_ss, sss = is_k ? a.pool.ks_ss : a.pool.vs_ss;
  uint8_t *codes = (is_k ? a.pool.k + h * a.pool.k_sh : a.pool.v + h * a.pool.v_sh) + 8 * c;
  uint8_t *scales = (is_k ? a.pool.ks + h * a.pool.ks_sh : a.pool.vs + h * a.pool.vs_sh) + c;
  const float tensor_scale = is_k ? a.k_scale : a.v_scale;
  const int e = (int)((__float_as_uint(tensor_scale) >> 23) & 0xFFu) - 127;
  const bool pow2 = (__float_as_uint(tensor_scale) & 0x7FFFFFu) == 0 && e >= -64 && e <= 64;
  for (; token < a.n_tokens; token += step * kWriteUnroll) {
    uint4 val[kWriteUnroll][2];
    int64_t slot[kWriteUnroll];
#pragma unroll
    for (int u = 0; u < kWriteUnroll; ++u) {
      const int64_t t = token + u * step;
      slot[u] = -1;
      if (t < a.n_tokens) {
        slot[u] = __ldg(a.cache_loc + t);
        val[u][0] = __ldg(src + t * ts);
        val[u][1] = __ldg(src + t * ts + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kWriteUnroll; ++u) {
      if (slot[u] < 0 || slot[u] >= a.pool.num_slots) continue;  // outside the pool: skipped
      uint8_t sc;
      const uint2 q = pow2 ? quantise_block<true>(val[u], tensor_scale, sc)
                           : quantise_block<false>(val[u], tensor_scale, sc);
      *reinterpret_cast<uint2 *>(codes + slot[u] * css) = q;
      scales[slot[u] * sss] = sc;
    }
  }
}

int launch_set_kv_buffer_fp4(const void *k, int64_t k_ts, int64_t k_hs, const void *v,
                             int64_t v_ts, int64_t v_hs, const int64_t *cache_loc,
                             int64_t n_tokens, int hkv, int lk, int lv, float k_scale,
                             float v_scale, const Fp4Pool &pool, cudaStream_t st) {
  Fp4WriteArgs a;
  a.k = static_cast<const uint4 *>(k);
  a.v = static_cast<const uint4 *>(v);
  a.k_ts = k_ts / 8; a.k_hs = k_hs / 8; a.v_ts = v_ts / 8; a.v_hs = v_hs / 8;
  a.cache_loc = cache_loc;
  a.pool = pool;
  a.n_tokens = n_tokens;
  a.hkv = hkv;
  a.nk = lk / kFp4Block;
  a.nv = v ? lv / kFp4Block : 0;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const int64_t places = (int64_t)hkv * (a.nk + a.nv);
  if (places > kMaxPlaces)
    return set_error(PKX_EUNSUPPORTED, "set_kv_buffer_fp4: more than %d blocks a token", kMaxPlaces);
  if (n_tokens >= kMaxRows)
    return set_error(PKX_EUNSUPPORTED, "set_kv_buffer_fp4: 2^40 tokens or more");
  a.places = fp4_places(places);
  cudaError_t e = launch_pdl(set_kv_buffer_fp4_kernel,
                             wave_grid(set_kv_buffer_fp4_kernel, a.places, n_tokens, kWriteUnroll),
                             dim3(kFp4Threads), 0, st, a);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "set_kv_buffer_fp4 launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

// --------------------------------------------------------------- read back
struct Fp4ReadArgs {
  Fp4Pool pool;
  const int32_t *kv_indices;
  uint4 *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;  // output strides in 16-byte chunks
  int64_t n_rows;
  int hkv, ck, cv;                 // heads; 8-element chunks of a K row, of a V row (0: K only)
  Fp4Places places;
  float k_scale, v_scale;
};

constexpr int kReadUnroll = 4;

__global__ void __launch_bounds__(kFp4Threads) get_kv_buffer_fp4_kernel(const Fp4ReadArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  int64_t token, step;
  int c = fp4_place(a.places, token, step);
  if (c < 0) return;
  const bool is_k = c < a.hkv * a.ck;
  if (!is_k) c -= a.hkv * a.ck;
  const int nc = is_k ? a.ck : a.cv;
  const int h = c / nc;
  c -= h * nc;
  const int64_t css = is_k ? a.pool.k_ss : a.pool.v_ss, sss = is_k ? a.pool.ks_ss : a.pool.vs_ss;
  const uint8_t *codes = (is_k ? a.pool.k + h * a.pool.k_sh : a.pool.v + h * a.pool.v_sh) + 4 * c;
  const uint8_t *scales =
      (is_k ? a.pool.ks + h * a.pool.ks_sh : a.pool.vs + h * a.pool.vs_sh) + (c >> 1);
  const int64_t ts = is_k ? a.k_ts : a.v_ts;
  uint4 *dst = (is_k ? a.k + h * a.k_hs : a.v + h * a.v_hs) + c;
  const float tensor_scale = is_k ? a.k_scale : a.v_scale;
  for (; token < a.n_rows; token += step * kReadUnroll) {
    uint32_t code[kReadUnroll], sc[kReadUnroll];
    int slot[kReadUnroll];
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int64_t t = token + u * step;
      slot[u] = t < a.n_rows ? __ldg(a.kv_indices + t) : -1;
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      code[u] = sc[u] = 0u;
      if (slot[u] >= 0 && slot[u] < a.pool.num_slots) {  // else the row reads zero
        code[u] = __ldg(reinterpret_cast<const uint32_t *>(codes + slot[u] * css));
        sc[u] = __ldg(scales + slot[u] * sss);
      }
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const int64_t t = token + u * step;
      if (t >= a.n_rows) break;
      const __half2 s2 = e4m3x2_to_f16x2(sc[u] | (sc[u] << 8));
      uint32_t x[4], out[4];
      e2m1x8_to_f16(code[u], x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // the f16 product is exact, the next one rounds to fp32
        const float2 f = __half22float2(__hmul2(*reinterpret_cast<const __half2 *>(&x[i]), s2));
        out[i] = pack_bf16(f.x * tensor_scale, f.y * tensor_scale);
      }
      dst[t * ts] = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

int launch_get_kv_buffer_fp4(const Fp4Pool &pool, const int32_t *kv_indices, int64_t n_rows,
                             int hkv, int lk, int lv, float k_scale, float v_scale, void *k,
                             int64_t k_ts, int64_t k_hs, void *v, int64_t v_ts, int64_t v_hs,
                             cudaStream_t st) {
  Fp4ReadArgs a;
  a.pool = pool;
  a.kv_indices = kv_indices;
  a.k = static_cast<uint4 *>(k);
  a.v = static_cast<uint4 *>(v);
  a.k_ts = k_ts / 8; a.k_hs = k_hs / 8; a.v_ts = v_ts / 8; a.v_hs = v_hs / 8;
  a.n_rows = n_rows;
  a.hkv = hkv;
  a.ck = lk / 8;
  a.cv = v ? lv / 8 : 0;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const int64_t places = (int64_t)hkv * (a.ck + a.cv);
  if (places > kMaxPlaces)
    return set_error(PKX_EUNSUPPORTED, "get_kv_buffer_fp4: more than %d chunks a token", kMaxPlaces);
  if (n_rows >= kMaxRows)
    return set_error(PKX_EUNSUPPORTED, "get_kv_buffer_fp4: 2^40 rows or more");
  a.places = fp4_places(places);
  cudaError_t e = launch_pdl(get_kv_buffer_fp4_kernel,
                             wave_grid(get_kv_buffer_fp4_kernel, a.places, n_rows, kReadUnroll),
                             dim3(kFp4Threads), 0, st, a);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "get_kv_buffer_fp4 launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
