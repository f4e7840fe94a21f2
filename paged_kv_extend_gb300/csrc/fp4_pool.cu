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
// and stores 0.5625 bytes an element, the read back the reverse.  The write
// gives a thread one block (two 16-byte loads, an 8-byte and a one-byte
// store: a row's stores are whole sectors); the read back gives a thread 8
// elements, so that a warp stores 512 consecutive bytes.  Both keep several
// blocks in flight per thread and run a grid of one resident wave over a flat
// list of chunks, as the bf16 KV write does.
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

constexpr int kFp4Threads = 256;

// ------------------------------------------------------------------- write
struct Fp4WriteArgs {
  const uint4 *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;  // input strides in 16-byte chunks
  const int64_t *cache_loc;
  Fp4Pool pool;
  uint32_t hkv, nk, nv;  // heads; blocks of a K row, of a V row (0: K only)
  uint32_t total;        // n_tokens * hkv * (nk + nv), below 2^31
  float k_scale, v_scale;
};

// One block of 16 bf16: the 8 code bytes and the scale code.
__device__ __forceinline__ uint2 quantise_block(const uint4 (&in)[2], float tensor_scale,
                                                uint8_t &scale_code) {
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  float q[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[2 * i] = __uint_as_float(w[i] << 16);
    q[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if (tensor_scale != 1.0f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __fdiv_rn(q[i], tensor_scale);
  }
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    amax = fmaxf(amax, fabsf(q[i]));  // drops a NaN
    nan |= q[i] != q[i];
  }
  const __nv_fp8_storage_t sc =
      __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f), __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(sc, __NV_E4M3)));
  scale_code = nan ? (uint8_t)0x7F : (uint8_t)sc;
  uint32_t out[2] = {0u, 0u};
  if (!nan && s > 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t code =
          e2m1_magnitude(fabsf(q[i]), s) | ((__float_as_uint(q[i]) >> 28) & 8u);
      out[i >> 3] |= code << (4 * (i & 7));
    }
  }
  return make_uint2(out[0], out[1]);
}

constexpr int kWriteUnroll = 2;

__global__ void __launch_bounds__(kFp4Threads) set_kv_buffer_fp4_kernel(const Fp4WriteArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t stride = gridDim.x * kFp4Threads;
  const uint32_t per_row = a.nk + a.nv;
  for (uint64_t base = blockIdx.x * kFp4Threads + threadIdx.x; base < a.total;
       base += (uint64_t)stride * kWriteUnroll) {
    uint4 val[kWriteUnroll][2];
    int64_t slot[kWriteUnroll];
    uint32_t hh[kWriteUnroll], cc[kWriteUnroll];
#pragma unroll
    for (int u = 0; u < kWriteUnroll; ++u) {
      const uint64_t i64 = base + (uint64_t)u * stride;
      slot[u] = -1;
      if (i64 < a.total) {
        const uint32_t i = (uint32_t)i64;
        const uint32_t row = i / per_row;
        cc[u] = i - row * per_row;
        const uint32_t t = row / a.hkv;
        hh[u] = row - t * a.hkv;
        slot[u] = __ldg(a.cache_loc + t);
        const uint4 *src =
            cc[u] < a.nk ? a.k + (int64_t)t * a.k_ts + (int64_t)hh[u] * a.k_hs + 2 * cc[u]
                         : a.v + (int64_t)t * a.v_ts + (int64_t)hh[u] * a.v_hs + 2 * (cc[u] - a.nk);
        val[u][0] = __ldg(src);
        val[u][1] = __ldg(src + 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kWriteUnroll; ++u) {
      if (slot[u] < 0 || slot[u] >= a.pool.num_slots) continue;  // outside the pool: skipped
      const bool is_k = cc[u] < a.nk;
      const uint32_t c = is_k ? cc[u] : cc[u] - a.nk;
      uint8_t sc;
      const uint2 codes = quantise_block(val[u], is_k ? a.k_scale : a.v_scale, sc);
      uint8_t *dst = is_k ? a.pool.k + slot[u] * a.pool.k_ss + (int64_t)hh[u] * a.pool.k_sh
                          : a.pool.v + slot[u] * a.pool.v_ss + (int64_t)hh[u] * a.pool.v_sh;
      uint8_t *dsc = is_k ? a.pool.ks + slot[u] * a.pool.ks_ss + (int64_t)hh[u] * a.pool.ks_sh
                          : a.pool.vs + slot[u] * a.pool.vs_ss + (int64_t)hh[u] * a.pool.vs_sh;
      *reinterpret_cast<uint2 *>(dst + 8 * c) = codes;
      dsc[c] = sc;
    }
  }
}

// CTAs of one resident wave of `kernel`, at most `need`.
template <typename K>
static unsigned wave_grid(K kernel, uint64_t need) {
  static int resident = 0;  // CTAs per SM (one kernel per argument type)
  if (resident == 0) {
    int r = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&r, kernel, kFp4Threads, 0) != cudaSuccess ||
        r < 1)
      r = 4;
    resident = r;
  }
  const uint64_t cap = (uint64_t)num_sms_current_device() * resident;
  const uint64_t g = need < cap ? need : cap;
  return (unsigned)(g > 0 ? g : 1);
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
  a.hkv = (uint32_t)hkv;
  a.nk = (uint32_t)(lk / kFp4Block);
  a.nv = v ? (uint32_t)(lv / kFp4Block) : 0u;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const uint64_t per_token = (uint64_t)a.hkv * (a.nk + a.nv);
  if ((uint64_t)n_tokens >= (1ull << 31) / per_token)
    return set_error(PKX_EUNSUPPORTED, "set_kv_buffer_fp4: 2^31 or more blocks in one call");
  a.total = (uint32_t)(n_tokens * per_token);
  const uint64_t need = (a.total + kFp4Threads * kWriteUnroll - 1) / (kFp4Threads * kWriteUnroll);
  cudaError_t e = launch_pdl(set_kv_buffer_fp4_kernel, dim3(wave_grid(set_kv_buffer_fp4_kernel, need)),
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
  uint32_t hkv, ck, cv;            // heads; 8-element chunks of a K row, of a V row (0: K only)
  uint32_t total;                  // n_rows * hkv * (ck + cv), below 2^31
  float k_scale, v_scale;
};

constexpr int kReadUnroll = 4;

__global__ void __launch_bounds__(kFp4Threads) get_kv_buffer_fp4_kernel(const Fp4ReadArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t stride = gridDim.x * kFp4Threads;
  const uint32_t per_row = a.ck + a.cv;
  for (uint64_t base = blockIdx.x * kFp4Threads + threadIdx.x; base < a.total;
       base += (uint64_t)stride * kReadUnroll) {
    uint32_t code[kReadUnroll];
    uint32_t sc[kReadUnroll];
    uint4 *dst[kReadUnroll];
    float ts[kReadUnroll];
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      const uint64_t i64 = base + (uint64_t)u * stride;
      dst[u] = nullptr;
      code[u] = sc[u] = 0u;
      if (i64 < a.total) {
        const uint32_t i = (uint32_t)i64;
        const uint32_t row = i / per_row;
        uint32_t c = i - row * per_row;
        const uint32_t t = row / a.hkv, h = row - t * a.hkv;
        const int64_t slot = __ldg(a.kv_indices + t);
        const bool is_k = c < a.ck;
        if (!is_k) c -= a.ck;
        ts[u] = is_k ? a.k_scale : a.v_scale;
        dst[u] = is_k ? a.k + (int64_t)t * a.k_ts + (int64_t)h * a.k_hs + c
                      : a.v + (int64_t)t * a.v_ts + (int64_t)h * a.v_hs + c;
        if (slot >= 0 && slot < a.pool.num_slots) {  // else the row reads zero
          const uint8_t *pc = is_k ? a.pool.k + slot * a.pool.k_ss + (int64_t)h * a.pool.k_sh
                                   : a.pool.v + slot * a.pool.v_ss + (int64_t)h * a.pool.v_sh;
          const uint8_t *ps = is_k ? a.pool.ks + slot * a.pool.ks_ss + (int64_t)h * a.pool.ks_sh
                                   : a.pool.vs + slot * a.pool.vs_ss + (int64_t)h * a.pool.vs_sh;
          code[u] = __ldg(reinterpret_cast<const uint32_t *>(pc) + c);
          sc[u] = __ldg(ps + (c >> 1));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kReadUnroll; ++u) {
      if (!dst[u]) continue;
      const float s = __low2float(e4m3x2_to_f16x2(sc[u]));
      uint32_t h[4];
      e2m1x8_to_f16(code[u], h);
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        x[2 * i] = f.x * s * ts[u];  // the first product is exact
        x[2 * i + 1] = f.y * s * ts[u];
      }
      *dst[u] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                           pack_bf16(x[6], x[7]));
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
  a.hkv = (uint32_t)hkv;
  a.ck = (uint32_t)(lk / 8);
  a.cv = v ? (uint32_t)(lv / 8) : 0u;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const uint64_t per_row = (uint64_t)a.hkv * (a.ck + a.cv);
  if ((uint64_t)n_rows >= (1ull << 31) / per_row)
    return set_error(PKX_EUNSUPPORTED, "get_kv_buffer_fp4: 2^31 or more chunks in one call");
  a.total = (uint32_t)(n_rows * per_row);
  const uint64_t need = (a.total + kFp4Threads * kReadUnroll - 1) / (kFp4Threads * kReadUnroll);
  cudaError_t e = launch_pdl(get_kv_buffer_fp4_kernel, dim3(wave_grid(get_kv_buffer_fp4_kernel, need)),
                             dim3(kFp4Threads), 0, st, a);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "get_kv_buffer_fp4 launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
