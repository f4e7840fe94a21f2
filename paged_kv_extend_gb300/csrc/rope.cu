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
// in the smallest power of two of lanes that holds it 8 elements a lane (16
// bytes), so a warp holds two rows of 128 dims; the sum of squares and, for
// half-split pairs, the partners' elements go through shuffles.  A warp
// belongs to one token and walks its rows, kRows steps loaded before the first
// is used: the lane's cosines and sines are fetched once for all heads.  A
// token's rows are shared by as many warps as fill the GPU (a decode step has
// few tokens), by one warp when there are many tokens.
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

constexpr int kRopeThreads = 256;
constexpr int kRows = 4;  // row steps in flight

struct RopeParams {
  RopeArgs a;
  int64_t warps;        // tokens * parts
  int parts;            // warps that share a token's rows
  int lanes;            // lanes of a row (a power of two)
  int chunks;           // d / 8
  int half_chunks;      // rotary / 16: chunks of one half of the rotated dims
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

// FMT: the pool's element format (0 bf16, 1 e4m3, 2 e5m2).  LEAVED: pairs of
// neighbouring elements.
template <int FMT, bool LEAVED>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const RopeArgs &a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t w0 = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int c = lane & (p.lanes - 1);               // chunk of the row
  const int sub = lane / p.lanes, rows = 32 / p.lanes;  // row within a warp's step
  const bool in_row = c < p.chunks;
  const int n_rows = a.hq + a.hkv + (a.v ? a.hkv : 0);
  const int n_steps = (n_rows + rows - 1) / rows;
  const int half = a.rotary >> 1;
  // this chunk's pairs: first pair, and which side of them it holds
  const bool rot = c < 2 * p.half_chunks;
  const bool second = !LEAVED && c >= p.half_chunks;
  const int pair0 = LEAVED ? 4 * c : 8 * (second ? c - p.half_chunks : c);
  // lane of the chunk that holds the partners (half-split pairs)
  const int partner = !rot ? lane : second ? lane - p.half_chunks : lane + p.half_chunks;
  constexpr int NP = LEAVED ? 4 : 8;

  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (a.q_weight && in_row) wq = __ldg(reinterpret_cast<const uint4 *>(a.q_weight) + c);
  if (a.k_weight && in_row) wk = __ldg(reinterpret_cast<const uint4 *>(a.k_weight) + c);

  for (int64_t w = w0; w < p.warps; w += (int64_t)gridDim.x * (kRopeThreads / 32)) {
    const int64_t tok = w / p.parts;
    const int part = (int)(w - tok * p.parts);
    // this lane's cosines and sines; NaN for a position outside the table or
    // an axis that does not exist
    float cs[NP], sn[NP];
    if (rot) {
      if (!a.pair_axis) {
        const int64_t pos = __ldg(a.positions + tok);
        const bool ok = pos >= 0 && pos < a.max_position;
        const float *row = a.cos_sin + (ok ? pos : 0) * a.rotary + pair0;
#pragma unroll
        for (int i = 0; i < NP; i += 4) {
          const float4 x = __ldg(reinterpret_cast<const float4 *>(row + i));
          const float4 y = __ldg(reinterpret_cast<const float4 *>(row + half + i));
          cs[i] = x.x; cs[i + 1] = x.y; cs[i + 2] = x.z; cs[i + 3] = x.w;
          sn[i] = y.x; sn[i + 1] = y.y; sn[i + 2] = y.z; sn[i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (!ok) cs[i] = sn[i] = __int_as_float(0x7fffffff);
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int axis = __ldg(a.pair_axis + pair0 + i);
          const int64_t pos = axis < a.axes ? __ldg(a.positions + axis * a.n_tokens + tok) : -1;
          cs[i] = sn[i] = __int_as_float(0x7fffffff);
          if (pos >= 0 && pos < a.max_position) {
            cs[i] = __ldg(a.cos_sin + pos * a.rotary + pair0 + i);
            sn[i] = __ldg(a.cos_sin + pos * a.rotary + half + pair0 + i);
          }
        }
      }
    }
    int64_t slot = -1;
    if (a.cache_loc) {
      slot = __ldg(a.cache_loc + tok);
      if (slot >= a.num_slots) slot = -1;
    }
    for (int s0 = part; s0 < n_steps; s0 += p.parts * kRows) {
      uint4 val[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int r = (s0 + u * p.parts) * rows + sub;
        val[u] = make_uint4(0, 0, 0, 0);
        if (r < n_rows && in_row) {
          const uint16_t *src =
              r < a.hq ? a.q + tok * a.q_ts + r * a.q_hs
              : r < a.hq + a.hkv ? a.k + tok * a.k_ts + (r - a.hq) * a.k_hs
                                 : a.v + tok * a.v_ts + (r - a.hq - a.hkv) * a.v_hs;
          val[u] = *(reinterpret_cast<const uint4 *>(src) + c);
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int step = s0 + u * p.parts;
        if (step >= n_steps) break;  // (the same for the whole warp)
        const int r = step * rows + sub;
        const bool is_q = r < a.hq, is_k = !is_q && r < a.hq + a.hkv;
        uint4 out = val[u];
        float x[8];
        unpack8(out, x);
        if (a.q_weight || a.k_weight) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
          for (int o = p.lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
            const float inv = rsqrtf(ss * p.inv_d + a.eps);
            float wt[8];
            unpack8(is_q ? wq : wk, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= inv * (wt[i] + a.weight_offset);
          }
        }
        if (LEAVED) {
          if (rot) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e = x[2 * i], o = x[2 * i + 1];
              x[2 * i] = e * cs[i] - o * sn[i];
              x[2 * i + 1] = o * cs[i] + e * sn[i];
            }
          }
        } else if (p.half_chunks > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = __shfl_sync(0xffffffffu, x[i], partner);
            if (rot) x[i] = second ? x[i] * cs[i] + y * sn[i] : x[i] * cs[i] - y * sn[i];
          }
        }
        if (is_q || is_k)
          out = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                           pack_bf16(x[6], x[7]));
        if (r >= n_rows || !in_row) continue;
        if (is_q) {
          *(reinterpret_cast<uint4 *>(a.q_out + tok * a.qo_ts + r * a.qo_hs) + c) = out;
          continue;
        }
        const int h = is_k ? r - a.hq : r - a.hq - a.hkv;
        if (is_k) *(reinterpret_cast<uint4 *>(a.k_out + tok * a.ko_ts + h * a.ko_hs) + c) = out;
        if (slot >= 0) {
          const int64_t at = is_k ? slot * a.kb_ss + h * a.kb_hs : slot * a.vb_ss + h * a.vb_hs;
          uint8_t *pool = static_cast<uint8_t *>(is_k ? a.k_buffer : a.v_buffer);
          if constexpr (FMT == 0)
            *(reinterpret_cast<uint4 *>(pool + 2 * at) + c) = out;
          else
            *(reinterpret_cast<uint2 *>(pool + at) + c) =
                bf16x8_to_fp8x8<FMT>(out, is_k ? a.k_scale : a.v_scale);
        }
      }
    }
  }
}

int launch_qk_norm_rope(const RopeArgs &a, cudaStream_t st) {
  if (a.n_tokens == 0) return PKX_OK;
  RopeParams p;
  p.a = a;
  p.chunks = a.d / 8;
  p.lanes = 1;
  while (p.lanes < p.chunks) p.lanes *= 2;
  p.half_chunks = a.rotary / 16;
  p.inv_d = 1.0f / (float)a.d;
  const int nsm = num_sms_current_device();
  if (nsm <= 0) return set_error(PKX_ECUDA, "cannot query the current device");
  // Warps that share a token's rows: enough that the GPU holds about 16 warps
  // an SM, at most one a row step.
  const int rows = 32 / p.lanes;
  const int n_steps = (a.hq + a.hkv + (a.v ? a.hkv : 0) + rows - 1) / rows;
  const int64_t want = ((int64_t)nsm * 16 + a.n_tokens - 1) / a.n_tokens;
  p.parts = (int)(want < n_steps ? want : n_steps);
  p.warps = a.n_tokens * p.parts;
  const int64_t need = (p.warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const unsigned grid = (unsigned)(need < (1 << 30) ? need : (1 << 30));
  auto kernel = a.interleaved
                    ? (a.kv_fmt == kKvBf16      ? qk_norm_rope_kernel<0, true>
                       : a.kv_fmt == kKvFp8E4M3 ? qk_norm_rope_kernel<1, true>
                                                : qk_norm_rope_kernel<2, true>)
                    : (a.kv_fmt == kKvBf16      ? qk_norm_rope_kernel<0, false>
                       : a.kv_fmt == kKvFp8E4M3 ? qk_norm_rope_kernel<1, false>
                                                : qk_norm_rope_kernel<2, false>);
  cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kRopeThreads), 0, st, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "qk_norm_rope launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
