// rope.cu -- what stands between the projection and the attention call: the RMS
// norm of every query and key head, the position rotation, and the KV write, in
// one pass over the rows.
//
// A row x (one token, one head, d elements) becomes
//   y = x * rsqrt(mean(x^2) + eps) * (w + w_offset)         (with weights)
//   (y[a], y[b]) -> (y[a] c - y[b] s, y[b] c + y[a] s)      for its pairs
// with pair i = (i, i + r / 2), or (2i, 2i + 1) interleaved, and c = table[p][i],
// s = table[p][r / 2 + i] for the token's position p on the pair's axis.  All
// in fp32, rounded once to bf16; the pool gets that bf16 row (or its fp8
// codes, as the KV write of an fp8 pool makes them), so that the pool and the
// returned keys agree.
//
// What bounds it: memory.  Each q, k and v row is read once and written once
// (k and v once more into the pool), the table row once a token.  A row lies
// in the smallest power of two of lanes that holds it 8 elements a lane, so a
// warp holds two rows of 128 dims.  Of half-split pairs a lane takes four pairs,
// as two runs of four elements (8 bytes) half the rotated dims apart, so that a
// pair never crosses lanes; only the sum of squares goes through shuffles.  A
// warp belongs to one token and walks its rows, kRows steps at a time and the
// next ones on their way: the cosines and sines, with the weights multiplied
// in, are made once for all heads.  A token's rows are shared by as many warps as
// fill the GPU (a decode step has few tokens), by one warp when there are many.
// Measured on 16384 tokens of 32 + 8 + 8 heads of 128 (436 MB): 171 us with one
// run of eight elements a lane and the partners shuffled, 107 without the
// shuffles, 85 with the weights folded in, 78.7 with the next rows loaded early,
// 80 with every row's mean square looked at (5.45 TB/s, 0.80 of the copy bandwidth).
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

constexpr int kRopeThreads = 128;
constexpr int kRows = 4;  // row steps in flight
// Mean squares whose sums are far inside fp32's range.
constexpr float kLeast = 0x1p-100f, kMost = 0x1p118f;

struct RopeParams {
  RopeArgs a;
  int64_t warps;  // tokens * parts
  int parts;      // warps that share a token's rows
  int chunks;     // d / 8: lanes that hold elements
  int turned;     // rotary / 8: lanes whose elements are rotated
  int q_steps, k_steps;  // row steps of q and of k (v has k's)
  float inv_d;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// A lane's eight elements of a row: two runs of four, `second` elements apart
// (one run of eight for neighbouring pairs).
template <bool LEAVED>
__device__ __forceinline__ uint4 load_row(const uint16_t *p, int second) {
  if constexpr (LEAVED) return *reinterpret_cast<const uint4 *>(p);
  const uint2 a = *reinterpret_cast<const uint2 *>(p);
  const uint2 b = *reinterpret_cast<const uint2 *>(p + second);
  return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool LEAVED>
__device__ __forceinline__ void store_row(uint16_t *p, int second, uint4 v) {
  if constexpr (LEAVED) {
    *reinterpret_cast<uint4 *>(p) = v;
  } else {
    *reinterpret_cast<uint2 *>(p) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2 *>(p + second) = make_uint2(v.z, v.w);
  }
}
template <bool LEAVED, int FMT>
__device__ __forceinline__ void store_codes(uint8_t *p, int second, uint4 v, float scale) {
  const uint2 c = bf16x8_to_fp8x8<FMT>(v, scale);
  if constexpr (LEAVED) {
    *reinterpret_cast<uint2 *>(p) = c;
  } else {
    *reinterpret_cast<uint32_t *>(p) = c.x;
    *reinterpret_cast<uint32_t *>(p + second) = c.y;
  }
}

// What a lane does to the rows of q or of k, for its four pairs: with e, f a
// pair's elements, (e A - f B, f C + e D), where the norm's weights are
// multiplied into the cosines and sines; without rotation (e A, f C).
struct Turn {
  float A[4], B[4], C[4], D[4];
};

template <bool LEAVED>
__device__ __forceinline__ Turn make_turn(uint4 weight, bool weighted, float offset, bool turned,
                                          const float (&cs)[4], const float (&sn)[4]) {
  float w[8];
  unpack8(weight, w);
  Turn r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = LEAVED ? 2 * i : i, n = LEAVED ? 2 * i + 1 : i + 4;
    const float we = weighted ? w[m] + offset : 1.0f, wf = weighted ? w[n] + offset : 1.0f;
    r.A[i] = turned ? we * cs[i] : we;
    r.B[i] = wf * sn[i];
    r.C[i] = turned ? wf * cs[i] : wf;
    r.D[i] = we * sn[i];
  }
  return r;
}

// FMT: the pool's element format (0 bf16, 1 e4m3, 2 e5m2).  LEAVED: pairs of
// neighbouring elements.  LOG: a row takes 1 << LOG lanes.
template <int FMT, bool LEAVED, int LOG>
__global__ void __launch_bounds__(kRopeThreads, 5) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int LANES = 1 << LOG, ROWS = 32 / LANES;  // rows of a warp's step
  constexpr int BYTES = FMT == 0 ? 2 : 1;
  grid_dep_wait();
  grid_dep_launch();
  const RopeArgs &a = p.a;
  const int lane = threadIdx.x & 31, c = lane % LANES, sub = lane / LANES;
  const bool in_row = c < p.chunks, turned = c < p.turned;
  const int half = a.rotary >> 1;
  // this lane's elements: run of four at `at`, the other `second` further on
  const int at = !LEAVED && turned ? 4 * c : 8 * c;
  const int second = turned ? half : 4;
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (a.q_weight && in_row) wq = load_row<LEAVED>(a.q_weight + at, second);
  if (a.k_weight && in_row) wk = load_row<LEAVED>(a.k_weight + at, second);

  int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  for (; w < p.warps; w += (int64_t)gridDim.x * (kRopeThreads / 32)) {
    const int64_t tok = p.parts == 1 ? w : w / p.parts;
    const int part = (int)(w - tok * p.parts);
    // rows of q are taken from step `part` on, those of k and v where q's end
    const int k_part = (part + p.parts - p.q_steps % p.parts) % p.parts;
    const int v_part = (k_part + p.parts - p.k_steps % p.parts) % p.parts;
    const int stride = p.parts * ROWS;  // rows between a warp's steps
    uint4 val[kRows], next[kRows];
    auto load = [&](uint4 (&to)[kRows], const uint16_t *x, int64_t hs, int heads, int h0) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int h = h0 + u * stride + sub;
        to[u] = make_uint4(0, 0, 0, 0);
        if (in_row && h < heads) to[u] = load_row<LEAVED>(x + h * hs, second);
      }
    };
    auto advance = [&] {
#pragma unroll
      for (int u = 0; u < kRows; ++u) val[u] = next[u];
    };
    const uint16_t *qp = a.q + tok * a.q_ts + at, *kp = a.k + tok * a.k_ts + at;
    const uint16_t *vp = a.v + tok * a.v_ts + at;
    load(val, qp, a.q_hs, a.hq, part * ROWS);
    int64_t slot = -1;
    if (a.cache_loc) {
      slot = __ldg(a.cache_loc + tok);
      if (slot >= a.num_slots) slot = -1;
    }
    // the four pairs' cosines and sines; NaN for a position outside the table
    // or no such axis
    float cs[4] = {0.f, 0.f, 0.f, 0.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (turned) {
      const float nan = __int_as_float(0x7fffffff);
      if (!a.pair_axis) {
        const int64_t pos = __ldg(a.positions + tok);
        const bool ok = pos >= 0 && pos < a.max_position;
        const float *row = a.cos_sin + (ok ? pos : 0) * a.rotary + 4 * c;
        const float4 x = __ldg(reinterpret_cast<const float4 *>(row));
        const float4 y = __ldg(reinterpret_cast<const float4 *>(row + half));
        cs[0] = ok ? x.x : nan; cs[1] = ok ? x.y : nan;
        cs[2] = ok ? x.z : nan; cs[3] = ok ? x.w : nan;
        sn[0] = y.x; sn[1] = y.y; sn[2] = y.z; sn[3] = y.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int axis = __ldg(a.pair_axis + 4 * c + i);
          const int64_t pos = axis < a.axes ? __ldg(a.positions + axis * a.n_tokens + tok) : -1;
          cs[i] = sn[i] = nan;
          if (pos >= 0 && pos < a.max_position) {
            cs[i] = __ldg(a.cos_sin + pos * a.rotary + 4 * c + i);
            sn[i] = __ldg(a.cos_sin + pos * a.rotary + half + 4 * c + i);
          }
        }
      }
    }
    // one row: norm and rotation (all lanes of the warp)
    auto turn_row = [&](uint4 in, bool norm, const Turn &T) {
      float x[8];
      unpack8(in, x);
      if (norm) {
        auto mean_square = [&](float eps) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
          for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          return ss * p.inv_d + eps;
        };
        float ms = mean_square(a.eps);
        // rows whose squares leave fp32 (elements above 1.8e19, or all of them tiny
        // and eps with them) once more, times a power of two
        if (__any_sync(0xffffffffu, !(ms > kLeast && ms < kMost))) {
          const float s = ms <= kLeast ? 0x1p100f : ms < kMost ? 1.0f : 0x1p-80f;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= s;
          ms = mean_square(a.eps * s * s);
        }
        const float inv = rsqrtf(ms);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = LEAVED ? 2 * i : i, n = LEAVED ? 2 * i + 1 : i + 4;
        const float e = x[m], f = x[n];
        x[m] = e * T.A[i];
        x[n] = f * T.C[i];
        if (turned) {
          x[m] -= f * T.B[i];
          x[n] += e * T.D[i];
        }
      }
      return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                        pack_bf16(x[6], x[7]));
    };
    auto store_pool = [&](void *pool, int64_t row, uint4 v, float scale) {
      uint8_t *dst = static_cast<uint8_t *>(pool) + (row + at) * BYTES;
      if constexpr (FMT == 0) store_row<LEAVED>(reinterpret_cast<uint16_t *>(dst), second, v);
      else store_codes<LEAVED, FMT>(dst, second, v, scale);
    };
    {
      const bool norm = a.q_weight != nullptr;
      const Turn T = make_turn<LEAVED>(wq, norm, a.weight_offset, turned, cs, sn);
      uint16_t *out = a.q_out + tok * a.qo_ts + at;
      for (int h0 = part * ROWS;; h0 += kRows * stride) {
        // the rows after these: of q, or the first of k
        const int h1 = h0 + kRows * stride;
        if (h1 < a.hq) load(next, qp, a.q_hs, a.hq, h1);
        else load(next, kp, a.k_hs, a.hkv, k_part * ROWS);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (h0 + u * stride >= a.hq) break;  // (the same for the whole warp)
          const int h = h0 + u * stride + sub;
          const uint4 r = turn_row(val[u], norm, T);
          if (in_row && h < a.hq) store_row<LEAVED>(out + h * a.qo_hs, second, r);
        }
        advance();
        if (h1 >= a.hq) break;
      }
    }
    {
      const bool norm = a.k_weight != nullptr;
      const Turn T = make_turn<LEAVED>(wk, norm, a.weight_offset, turned, cs, sn);
      uint16_t *out = a.k_out + tok * a.ko_ts + at;
      for (int h0 = k_part * ROWS;; h0 += kRows * stride) {
        const int h1 = h0 + kRows * stride;
        if (h1 < a.hkv) load(next, kp, a.k_hs, a.hkv, h1);
        else if (a.v && slot >= 0) load(next, vp, a.v_hs, a.hkv, v_part * ROWS);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (h0 + u * stride >= a.hkv) break;
          const int h = h0 + u * stride + sub;
          const uint4 r = turn_row(val[u], norm, T);
          if (!in_row || h >= a.hkv) continue;
          store_row<LEAVED>(out + h * a.ko_hs, second, r);
          if (slot >= 0) store_pool(a.k_buffer, slot * a.kb_ss + h * a.kb_hs, r, a.k_scale);
        }
        advance();
        if (h1 >= a.hkv) break;
      }
    }
    if (a.v && slot >= 0) {
      for (int h0 = v_part * ROWS; h0 < a.hkv; h0 += kRows * stride) {
        if (h0 != v_part * ROWS) load(val, vp, a.v_hs, a.hkv, h0);
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const int h = h0 + u * stride + sub;
          if (in_row && h < a.hkv)
            store_pool(a.v_buffer, slot * a.vb_ss + h * a.vb_hs, val[u], a.v_scale);
        }
      }
    }
  }
}

template <bool LEAVED, int LOG>
static void (*rope_kernel(int fmt))(const RopeParams) {
  return fmt == kKvBf16      ? qk_norm_rope_kernel<0, LEAVED, LOG>
         : fmt == kKvFp8E4M3 ? qk_norm_rope_kernel<1, LEAVED, LOG>
                             : qk_norm_rope_kernel<2, LEAVED, LOG>;
}
template <bool LEAVED>
static void (*rope_kernel(int fmt, int log))(const RopeParams) {
  switch (log) {
    case 3: return rope_kernel<LEAVED, 3>(fmt);
    case 4: return rope_kernel<LEAVED, 4>(fmt);
    case 5: return rope_kernel<LEAVED, 5>(fmt);
    default: return rope_kernel<LEAVED, 2>(fmt);  // d <= 32 (lanes may be idle)
  }
}

int launch_qk_norm_rope(const RopeArgs &a, cudaStream_t st) {
  if (a.n_tokens == 0) return PKX_OK;
  RopeParams p;
  p.a = a;
  p.chunks = a.d / 8;
  int log = 2;
  while ((1 << log) < p.chunks) ++log;
  p.turned = a.rotary / 8;
  p.inv_d = 1.0f / (float)a.d;
  const int nsm = num_sms_current_device();
  if (nsm <= 0) return set_error(PKX_ECUDA, "cannot query the current device");
  // Warps that share a token's rows: enough that the GPU holds about 16 warps
  // an SM, at most one a row step.
  const int rows = 32 >> log;
  p.q_steps = (a.hq + rows - 1) / rows;
  p.k_steps = (a.hkv + rows - 1) / rows;
  const int steps = p.q_steps + p.k_steps * (a.v ? 2 : 1);
  const int64_t want = ((int64_t)nsm * 16 + a.n_tokens - 1) / a.n_tokens;
  p.parts = (int)(want < steps ? want : steps);
  p.warps = a.n_tokens * p.parts;
  const int64_t need = (p.warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const unsigned grid = (unsigned)(need < (1 << 30) ? need : (1 << 30));
  auto kernel = a.interleaved ? rope_kernel<true>(a.kv_fmt, log) : rope_kernel<false>(a.kv_fmt, log);
  cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kRopeThreads), 0, st, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "qk_norm_rope launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
