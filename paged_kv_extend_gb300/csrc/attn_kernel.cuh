// attn_kernel.cuh -- the attention kernel of attention.cu (which describes its
// design) and its launch, for the translation units that instantiate it:
// attention.cu (work listed by sched_kernel) and listed_attention.cu (work
// listed by schedulers of its own).
#pragma once

#include <climits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "fp8.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ void record_status(int32_t *status, int code) {
  atomicCAS(status, 0, code);
}

// First tokens that stay visible.  A query block whose first query sits at
// qpos0 sees the keys [0, first) and those from qpos0 - window on; the keys
// between them, block_gap() of them, are left out, and the block's keys are
// numbered without them: number v is key v below `first`, key v + gap from
// there on.
__device__ __forceinline__ int block_gap(int qpos0, int window, int first) {
  if (first <= 0 || window <= 0) return 0;
  return (int)max((long long)qpos0 - window - first, 0ll);
}
// The number of key j (for a key in the gap: of the next one that is not).
__device__ __forceinline__ int key_number(int j, int first, int gap) {
  return j <= first ? j : max(first, j - gap);
}

struct KParams {
  const bf16 *q;  // read directly by the MLA kernel (the GQA kernel uses the TMA map)
  bf16 *o;
  float *lse;
  const bf16 *k_pool, *v_pool, *k_ext, *v_ext;
  int64_t kb_ss, vb_ss, ke_st, ve_st;  // row strides (elements): slot / token
  int64_t kb_sh, vb_sh, ke_sh, ve_sh;  // head strides (elements)
  int64_t num_slots;
  const int32_t *qo_indptr, *kv_indptr;
  const void *kv_indices;
  int hq, group, tok, q_box_tok, window, use_cap, rows_per_slot;
  int first;  // FIRST instantiations: first tokens that stay visible before the window
  // 4-bit pool: block scales of K and V rows (byte strides)
  const uint8_t *k_bs, *v_bs;
  int64_t kbs_ss, kbs_sh, vbs_ss, vbs_sh;
  float scale_log2;  // sm_scale * log2(e)           (no cap)
  float cap_pre;     // sm_scale / cap                (cap)
  float cap_log2;    // cap * log2(e)                 (cap)
  const uint8_t *custom_mask;   // nullable: byte per (extend row, key); replaces causal
  const int32_t *mask_indptr;   // [batch+1] offsets of each sequence's mask rows
  const float *sinks;           // nullable [hq] sink logits (natural log)
  // fp8 pool: a key reads code * k_scale, a value code * v_scale.  The codes
  // go to shared memory as exact bf16; k_scale is folded into the logit
  // scale of pool tiles, v_scale into their P through the exponent
  // (2^(s - m + log2 v_scale)), and the tile's row sum is divided back
  float scale_log2_k, cap_pre_k, log2_v_scale, inv_v_scale, v_scale;
  int dec_two;  // decode units run two key streams (else one)
  const int32_t *prefix_lens;   // unified form: prefix length per sequence
  const WorkUnit *units;
  const int32_t *uorder;  // units by cost, largest first
  const WsHeader *hdr;
  int32_t *next_unit;     // claim counter over uorder (zeroed by the scheduler)
  const int32_t *part_first;  // MLA pairs: each pair's claim positions (stream partition), or null
  int32_t *status;
  float *plse, *po;
  // two-stage form with the fused KV write: the pool slot of each extend
  // token (nullable), and the pools as writable pointers
  const int64_t *cache_loc;
  bf16 *k_pool_w, *v_pool_w;
  uint64_t wait_ns;       // time limit of every bounded wait
  int stall;              // test hook: the softmax warps first wait on a barrier
                          // no thread arrives at, so that the limit runs out
};

// TMA descriptor of q (3-D: dim, head, token).
struct TMaps {
  CUtensorMap q;
};
// Listed units: besides it, one with a box of a single token.
struct ListedMaps : TMaps {
  CUtensorMap one;
};
template <int MODE> struct MapsOf { using T = TMaps; };
template <> struct MapsOf<kListed> { using T = ListedMaps; };
// The map over q [n, hq, lq]: box = 64 dims x G heads x tok tokens.
int make_q_map(CUtensorMap *m, const void *q, int64_t n, int hq, int lq, int G, int tok);

// Head configuration HD: 64 and 128 are Lq = Lv = HD (two Q tiles per unit);
// 192 and 288 are the split head dims Lq = 192 / Lv = 128 and Lq = 288 /
// Lv = 256 (sglang extend_attention.py, _get_block_sizes_for_extend_attention:
// 192 = 128 + 64 rope, 288 = 256 + 32 rope), run with one Q tile per unit and
// one key stream: S (128 columns) and O (Lv columns) of the one tile fit TMEM,
// and a K stage of 128 keys fits shared memory next to the larger Q tile.
template <int HD>
struct Cfg {
  static constexpr bool SPLIT = HD == 192 || HD == 288;
  static constexpr int BM = kBlockM, BN = kBlockN;
  static constexpr int LQ = HD;
  static constexpr int HDV = HD == 192 ? 128 : HD == 288 ? 256 : HD;
  static constexpr int QA = (LQ + 63) / 64;  // 64-dim swizzle atoms of a Q / K row
  static constexpr int VA = HDV / 64;        // ... of a V row
  static constexpr int NQT = SPLIT ? 1 : 2;  // Q tiles per unit
  static constexpr bool TWO_OK = !SPLIT;     // two key streams for one-tile units
  static constexpr int NK = HD == 128 ? 3 : HD == 64 ? 5 : HD == 192 ? 2 : 1;  // K ring stages
  static constexpr int NV = HD == 128 ? 2 : HD == 64 ? 5 : HD == 192 ? 2 : 1;  // V ring stages
  static constexpr int NI = HD == 64 ? 4 : 3;     // row-index ring stages
  static constexpr int Q_BYTES = BM * QA * 128;   // one Q tile (a 288-dim row fills 4.5 atoms)
  static constexpr int K_BYTES = BN * QA * 128;
  static constexpr int V_BYTES = BN * VA * 128;
  static constexpr int I_BYTES = BN * 4;        // int32 row of each key
  static constexpr int OFF_Q = 0;               // NQT Q tiles
  static constexpr int OFF_K = OFF_Q + NQT * Q_BYTES;
  static constexpr int OFF_V = OFF_K + NK * K_BYTES;
  static constexpr int OFF_I = OFF_V + NV * V_BYTES;
  static constexpr int OFF_BAR = OFF_I + NI * I_BYTES;
  // decode over an fp8 pool: the codes land in a ring of NRAW slots (the
  // unused second Q tile and K stage 0) and are converted from there
  static constexpr int NRAW = 4;
  static constexpr int RAW_BYTES = BN * LQ;  // the fp8 codes of one K or V tile
  static constexpr int OFF_RAW = OFF_Q + Q_BYTES;
  // (extend over a 4-bit pool: the raw barriers are one per K and V stage)
  static constexpr int N_RAW_BARS = 2 * NRAW > NK + NV ? 2 * NRAW : NK + NV;
  static constexpr int N_BARS = 17 + 2 * NK + 2 * NV + 2 * NI + N_RAW_BARS;
  static constexpr int SMEM = OFF_BAR + N_BARS * 8 + 1024;  // + alignment slack
  // S0 | S1 | O0 | O1, 128 columns each (split dims: S0 | unused | O0 of Lv)
  static constexpr int TMEM_COLS = 512;
  static_assert(2 * BN + NQT * HDV <= TMEM_COLS, "TMEM budget");
  static constexpr uint32_t IDESC_QK = idesc_bf16_f32(BM, BN, 0);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(BM, HDV, 1);
  // warps 0-7: two softmax warpgroups; 8: MMA; 9: row indices + Q;
  // 10-13: copies; 14-15: idle
  static constexpr int THREADS = 512;
  static constexpr int COPY_WARP0 = 10;
  static constexpr int COPY_THREADS = 128;
  // keys per copy pass: whole rows per thread group for 64 / 128 dims; by
  // swizzle atom (chunk t % 8 of every atom, keys t / 8 + 16 i) for the
  // split dims, whose 24 or 36 chunks per row do not divide 128 threads
  static constexpr int KPP = SPLIT ? 16 : COPY_THREADS / (HD / 8);
  // Registers: the kernel launches with REGS_LAUNCH per thread (checked at
  // build time); the softmax warpgroups take REGS_SOFTMAX, the other two
  // give back down to REGS_OTHER.  The split must add up exactly.
  static constexpr int REGS_LAUNCH = 128, REGS_SOFTMAX = 168, REGS_OTHER = 88;
  static_assert(256 * REGS_SOFTMAX + 256 * REGS_OTHER == THREADS * REGS_LAUNCH,
                "register split must match the launch allocation");
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(SPLIT || NRAW * RAW_BYTES == Q_BYTES + K_BYTES,
                "the raw ring fills the second Q tile and K stage 0");
};

// barrier indices
enum {
  B_Q_FULL = 0,
  B_Q_EMPTY = 1,
  B_S_FULL = 2,  // + Q tile
  B_P_FULL = 4,  // + Q tile
  B_O_DONE = 6,  // + Q tile
  B_FINAL = 8,
  B_U_FULL = 9,    // + unit ring slot (kUnitRing)
  B_U_EMPTY = 12,  // + unit ring slot
  B_Q_CONV = 15,   // decode over fp8: the query rows converted to f16
  B_NEVER = 16,    // no thread ever arrives (the stall hook waits on it)
  B_RING = 17,  // K full[NK], K empty[NK], V full[NV], V empty[NV],
                // I full[NI], I empty[NI], raw full[NRAW], raw empty[NRAW]
};

// Key range [kb, ke) of tile j of a unit (tiles never straddle k_split).
template <int BN = kBlockN>
__device__ __forceinline__ void tile_keys(const WorkUnit &w, int j, int &kb, int &ke) {
  const int pe = min(w.k_end, w.k_split);
  const int n_pre = pe > w.k_begin ? (pe - w.k_begin + BN - 1) / BN : 0;
  if (j < n_pre) {
    kb = w.k_begin + j * BN;
    ke = min(kb + BN, pe);
  } else {
    kb = max(w.k_begin, w.k_split) + (j - n_pre) * BN;
    ke = min(kb + BN, w.k_end);
  }
}

// The bits [from, from + n) of a word (those below 32; none for n <= 0).
__device__ __forceinline__ uint32_t bit_range(int from, int n) {
  uint32_t r;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(r) : "r"(from), "r"(max(n, 0)));
  return r;
}

__device__ __forceinline__ void abort_cta(volatile int *abort_flag, int32_t *status, int code) {
  *abort_flag = 1;
  record_status(status, code);
}

// Units are claimed at run time: the index warp takes the next position of
// the cost order (largest first) from a global counter and passes the unit
// to the CTA's other warps through a small ring in shared memory (-1 ends
// the stream).  A CTA that finishes early simply claims more, so the work
// evens out without a cost model.
constexpr int kUnitRing = 3;
// Consumer side: the uc-th unit of this CTA, or -1 at the end or on a
// timeout (then *ok is cleared).  The slot is released as soon as it is
// read: by every lane of a warp (lane 0 arrives) or by a lone thread.
__device__ __forceinline__ int ring_unit(uint64_t *u_full, uint64_t *u_empty,
                                         const volatile int *ring, uint32_t uc,
                                         volatile int *abort_flag, bool whole_warp, bool &ok,
                                         uint64_t limit_ns) {
  const int slot = uc % kUnitRing;
  if (!mbar_wait(&u_full[slot], (uc / kUnitRing) & 1u, abort_flag, limit_ns)) {
    ok = false;
    return -1;
  }
  const int u = ring[slot];
  if (whole_warp) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&u_empty[slot]);
  } else {
    mbar_arrive(&u_empty[slot]);
  }
  return u;
}

// Eight fp8 codes as eight f16 of the same values (exact), element order
// kept: an e5m2 code is the top byte of its f16; e4m3 goes through the
// converter.
template <int FMT>
__device__ __forceinline__ uint4 fp8x8_to_f16x8(uint2 raw) {
  uint32_t out[4];
  if constexpr (FMT == 2) {
    out[0] = __byte_perm(raw.x, 0u, 0x1404);
    out[1] = __byte_perm(raw.x, 0u, 0x3424);
    out[2] = __byte_perm(raw.y, 0u, 0x1404);
    out[3] = __byte_perm(raw.y, 0u, 0x3424);
  } else {
    const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      out[i] = (uint32_t)h.x | ((uint32_t)h.y << 16);
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Eight bf16 times 2^-8 as eight f16 (round to nearest): the power of two
// keeps any bf16 of magnitude below 2^24 inside the f16 range; the logit
// scale takes the 2^8 back.
constexpr float kQF16Down = 0x1p-8f, kQF16Up = 256.0f;
// 4-bit pool: P is in f16, whose normal range ends at 2^-14, so a key some 12
// nats below its row's largest would lose bits, and one at 17 nats all of them
// (they are the output when the largest is a first token with a small value).
// P is therefore taken 2^11 times too large (the sum takes the same factor,
// which cancels) and the running maximum may lag by 2^4 at most: P stays below
// 2^15, and a key keeps bf16's 8 bits down to 2^-28 of the largest.
constexpr float kF4Shift = 11.0f, kF4Lag = 4.0f;
__device__ __forceinline__ uint4 bf16x8_to_f16x8_scaled(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16) * kQF16Down;
    const float hi = __uint_as_float(w[i] & 0xFFFF0000u) * kQF16Down;
    const __half2 h = __floats2half2_rn(lo, hi);
    out[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// Eight e2m1 codes times their block scale (a pair of f16) as eight f16 or
// bf16: exact in both, since the product has six significant bits and lies in
// [2^-10, 2688].  On a quarter SM a word takes 13.5 clocks to f16 and 27 to
// bf16 (37 by shifting the f16 bits to bf16's exponent).
template <bool BF16>
__device__ __forceinline__ uint4 fp4x8_to_16bit(uint32_t codes, __half2 s2) {
  uint32_t h[4];
  e2m1x8_to_f16(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&h[i]), s2);
    const float2 f = __half22float2(x);
    h[i] = BF16 ? pack_bf16(f.x, f.y) : *reinterpret_cast<const uint32_t *>(&x);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// MASK: a custom mask replaces the causal mask (its own instantiation, so
// the unmasked kernel carries none of the mask code).
// FMT: the pool's element format (0 bf16; 1 fp8 e4m3, 2 fp8 e5m2 with
// k_scale / v_scale; 3 the 4-bit pool, extend only).  Extend rows of the
// two-stage form are always bf16.  FIRST: first tokens stay visible before the
// window, and key ranges are key numbers (block_gap); its own instantiation,
// so that the others carry none of it.
template <int HD, int MODE, bool MASK, int FMT = 0, bool FIRST = false>
__global__ void __launch_bounds__(Cfg<HD>::THREADS, 1)
    attn_kernel(const __grid_constant__ typename MapsOf<MODE>::T tm, const KParams p) {
  using C = Cfg<HD>;
  static_assert(!(FIRST && MASK) && !(FMT == 3 && MODE == kDecode), "not built");
  // Decode over an fp8 pool runs its products in f16: a code becomes f16 in
  // one step (exact), the unit's query rows are converted once (times 2^-8),
  // P is written as f16 and v_scale is applied to the output.
  constexpr bool F16 = FMT != 0 && MODE == kDecode;
  constexpr uint32_t IDQK = F16 ? idesc_f16_f32(C::BM, C::BN, 0) : C::IDESC_QK;
  constexpr uint32_t IDPV = F16 ? idesc_f16_f32(C::BM, C::HDV, 1) : C::IDESC_PV;
  // K ring: decode over fp8 gives stage 0 to the raw-code ring
  constexpr int NK_ = F16 ? C::NK - 1 : C::NK;
  constexpr uint32_t K0 = C::OFF_K + (F16 ? C::K_BYTES : 0);
  // decode over fp8: warps 10-11 copy the codes, warps 12-13 convert the K
  // tiles and 14-15 the V tiles; extend over a 4-bit pool: warp 10 copies K,
  // warp 11 V, warps 12-13 convert K and 14-15 V
  constexpr bool F4 = FMT == 3;
  constexpr bool BITS = FIRST || F4;  // masked tiles by words of bits
  constexpr int RAW_THREADS = 64, CONV_THREADS = 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_unit[kUnitRing];

  const uint32_t raw = smem_u32(smem_raw);
  uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *k_full = bars + B_RING;
  uint64_t *k_empty = k_full + C::NK;
  uint64_t *v_full = k_empty + C::NK;
  uint64_t *v_empty = v_full + C::NV;
  uint64_t *i_full = v_empty + C::NV;
  uint64_t *i_empty = i_full + C::NI;
  uint64_t *raw_full = i_empty + C::NI;
  uint64_t *raw_empty = raw_full + C::NRAW;
  volatile int *abort_flag = &s_abort;

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const bool kv_write = MODE == kTwoStage && p.cache_loc != nullptr;

  if (tid == 0) {
    mbar_init(&bars[B_Q_FULL], 1);
    mbar_init(&bars[B_Q_CONV], C::COPY_THREADS);  // decode over fp8: warps 12-15
    mbar_init(&bars[B_Q_EMPTY], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[B_S_FULL + i], 1);
      mbar_init(&bars[B_P_FULL + i], 4);  // one arrival per softmax warp
      mbar_init(&bars[B_O_DONE + i], 1);
    }
    mbar_init(&bars[B_FINAL], 1);
    mbar_init(&bars[B_NEVER], 1);
    for (int i = 0; i < kUnitRing; ++i) {
      mbar_init(&bars[B_U_FULL + i], 1);
      // softmax, MMA and copy warps (+ the two writer warps with the fused
      // KV write)
      mbar_init(&bars[B_U_EMPTY + i],
                8 + 1 + C::COPY_THREADS / 32 + (kv_write || F16 || F4 ? 2 : 0));
    }
    // stages are filled by the copy warps, or by the converting warps in
    // decode over fp8
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(&k_full[s], F16 || F4 ? CONV_THREADS : C::COPY_THREADS);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(&v_full[s], F16 || F4 ? CONV_THREADS : C::COPY_THREADS);
      mbar_init(&v_empty[s], 1);
    }
    if constexpr (F4) {  // codes of a K or V stage landed: the copying warp's lanes
      for (int s = 0; s < C::NK + C::NV; ++s) mbar_init(&raw_full[s], 32);
    } else {
      for (int s = 0; s < C::NRAW; ++s) {
        mbar_init(&raw_full[s], RAW_THREADS);
        mbar_init(&raw_empty[s], CONV_THREADS);
      }
    }
    for (int s = 0; s < C::NI; ++s) {
      mbar_init(&i_full[s], 32);
      mbar_init(&i_empty[s], (F16 || F4 ? RAW_THREADS : C::COPY_THREADS) / 32);
    }
    s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&s_tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the prologue above reads no global memory; the work list, indices and
  // Q come from the kernels before this one on the stream
  grid_dep_wait();
  grid_dep_launch();  // the combine may be scheduled (it waits for this grid)
  const uint32_t tmem = s_tmem;
  const int n_units = p.hdr->n_units;
  const int G = p.group, TOK = p.tok;

  if (warp < 8) {
    regs_increase<C::REGS_SOFTMAX>();
    // ------------------------------------------- softmax + epilogue (x2)
    const int wg = warp >> 2;  // Q tile of this warpgroup
    const int wq = warp & 3;   // TMEM lane quarter
    const int r = tid & 127;   // tile row == TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t s_col = wg * C::BN;
    const uint32_t o_col = 2 * C::BN + wg * C::HDV;
    uint32_t s_cnt = 0, o_cnt = 0;
    bool ring_ok = true;
    // test hook: a wait that cannot succeed, so that the time limit runs out
    // and the abort path (flag, drain, TMEM release, return) runs
    if (p.stall && !mbar_wait(&bars[B_NEVER], 0, abort_flag, p.wait_ns))
      abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
    for (uint32_t uc = 0; !*abort_flag; ++uc) {
      const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ring_ok, p.wait_ns);
      if (u < 0) {
        if (!ring_ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
        break;
      }
      const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
      // decode: warpgroup wg takes the unit's tiles wg, wg + 2, ... of the
      // one query tile (two key streams, merged by the combine)
      // Two key streams (decode units; split units of one query tile):
      // warpgroup wg takes the unit's tiles wg, wg + 2, ... of the one query
      // tile and writes its own partial, which the combine merges.
      const bool two = C::TWO_OK && (MODE == kDecode ? p.dec_two != 0 : (w.slot >= 0 && w.n_tok <= TOK));
      // this warpgroup's tiles: j0, j0 + jstep, ... below the unit's n_tiles
      const int j0 = two ? wg : 0, jstep = two ? 2 : 1;
      const int nt = w.n_tiles - j0;  // > 0 when the warpgroup has a tile
      const int tok0 = two ? 0 : wg * TOK;  // first token of this warpgroup's Q rows
      if (!two && wg == 1 && w.n_tok <= TOK) continue;
      const int n_tok_i = min(TOK, w.n_tok - tok0);
      const int rows_valid = n_tok_i * G;
      const bool valid = r < rows_valid;
      const bool warp_active = wq * 32 < rows_valid;
      const int t = tok0 + r / G, g = r - (r / G) * G;
      const int qpos = w.qpos0 + t;
      const int qmin = w.qpos0 + tok0, qmax = w.qpos0 + tok0 + n_tok_i - 1;
      const int gap = FIRST ? block_gap(w.qpos0, p.window, p.first) : 0;
      const int64_t orow_idx = (int64_t)(w.q_tok0 + t) * p.hq + w.kvh * G + g;
      const int64_t prow_idx =
          MODE == kDecode ? (int64_t)(w.slot + wg) * p.rows_per_slot + r
          : MODE == kListed
              // a stream's rows follow the other's (rows_per_slot: one token's)
              ? (int64_t)w.slot * p.rows_per_slot + wg * (two ? w.n_tok : TOK) * G + r
              : (int64_t)w.slot * p.rows_per_slot + wg * TOK * G + r;
      // custom mask rows: a byte per key of the sequence for each extend
      // token; mbase is the row of this Q tile's first token
      const uint8_t *mbase = nullptr;
      int64_t mstride = 0;
      if (MASK) {
        const int qo0 = p.qo_indptr[w.b];
        mstride = MODE == kTwoStage ? (int64_t)(p.kv_indptr[w.b + 1] - p.kv_indptr[w.b]) +
                                          (p.qo_indptr[w.b + 1] - qo0)
                                    : (int64_t)(p.kv_indptr[w.b + 1] - p.kv_indptr[w.b]);
        mbase = p.custom_mask + p.mask_indptr[w.b] + (int64_t)(w.q_tok0 + tok0 - qo0) * mstride;
      }
      if (nt <= 0) {
        if (valid) {
          if (w.slot < 0) {
            bf16 *orow = p.o + orow_idx * C::HDV;
            for (int c = 0; c < C::HDV; c += 8)
              *reinterpret_cast<uint4 *>(orow + c) = make_uint4(0, 0, 0, 0);
            if (p.lse) p.lse[orow_idx] = -INFINITY;
          } else {
            float *prow = p.po + prow_idx * C::HDV;
            for (int c = 0; c < C::HDV; c += 4)
              *reinterpret_cast<float4 *>(prow + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            p.plse[prow_idx] = -INFINITY;
          }
        }
        continue;
      }
      float m = -INFINITY, l = 0.f;
      for (int j = j0; j < w.n_tiles; j += jstep) {
        int kb, ke;
        tile_keys(w, j, kb, ke);
        // Mask bits of this thread's row for keys kb + 32 q + bit (q < 4).
        // The G heads of a token share its mask row, so the warp walks its
        // rows' tokens: all lanes read 32 consecutive bytes of the token's
        // row (one sector per load), a ballot turns them into a word, and
        // the lanes of that token keep it.  Issued before the S wait.
        uint32_t mb[4] = {0u, 0u, 0u, 0u};
        if constexpr (MASK) {
          if (warp_active) {
            const int t_lo = (wq * 32) / G, t_hi = min((wq * 32 + 31) / G, n_tok_i - 1);
            const int my_t = r / G;
            // eight tokens at a time: all loads first, so their latencies overlap
            for (int tc = t_lo; tc <= t_hi; tc += 8) {
              uint8_t by[8][4];
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                const uint8_t *rowp = mbase + (int64_t)(tc + u) * mstride;
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                  const int kpos = kb + 32 * q4 + lane;
                  by[u][q4] = (tc + u <= t_hi && kpos < ke) ? __ldg(rowp + kpos) : (uint8_t)0;
                }
              }
#pragma unroll
              for (int u = 0; u < 8; ++u) {
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                  const uint32_t word = __ballot_sync(0xffffffffu, by[u][q4] != 0);
                  if (my_t == tc + u) mb[q4] = word;
                }
              }
            }
          }
        }
        if (!mbar_wait(&bars[B_S_FULL + wg], s_cnt & 1u, abort_flag, p.wait_ns)) {
          abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
          break;
        }
        ++s_cnt;
        tc_fence_after();
        if (warp_active) {
          float x[C::BN];
          {
            uint32_t v0[32], v1[32], v2[32], v3[32];
            tmem_ld32(lane_base + s_col + 0, v0);
            tmem_ld32(lane_base + s_col + 32, v1);
            tmem_ld32(lane_base + s_col + 64, v2);
            tmem_ld32(lane_base + s_col + 96, v3);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              x[i] = __uint_as_float(v0[i]);
              x[32 + i] = __uint_as_float(v1[i]);
              x[64 + i] = __uint_as_float(v2[i]);
              x[96 + i] = __uint_as_float(v3[i]);
            }
          }
          // Logits in the log2 domain are sc * x.  The plain path keeps the
          // raw dot products and folds sc into the exponent's FMA; a capped
          // or masked tile is first mapped into the log2 domain (sc = 1).
          // A tile of an fp8 pool holds the codes: its logits take k_scale
          // in the scale, its P takes v_scale.
          const bool pool8 = FMT != 0 && !(MODE == kTwoStage && kb >= w.k_split);
          float sc = pool8 ? p.scale_log2_k * (F16 ? kQF16Up : 1.0f) : p.scale_log2;
          if (p.use_cap) {
            const float pre = pool8 ? p.cap_pre_k * (F16 ? kQF16Up : 1.0f) : p.cap_pre;
#pragma unroll
            for (int i = 0; i < C::BN; ++i) x[i] = p.cap_log2 * tanh_approx(x[i] * pre);
            sc = 1.0f;
          }
          bool need_mask = MASK || (ke - 1 > qmin) || (ke - kb < C::BN) ||
                           (p.window > 0 && kb < qmax - p.window);
          if constexpr (FIRST) {
            // the last key is past the first query, or a key behind the first
            // tokens is before the last query's window
            const int last = ke - 1 >= p.first ? ke - 1 + gap : ke - 1;
            need_mask = last > qmin || ke - kb < C::BN ||
                        (ke > p.first && max(kb, p.first) + gap < qmax - p.window);
          }
          if constexpr (MASK) {
            // the custom mask replaces the causal term; the window stays.
            // A row that sees every key of the tile (all bits set, the
            // window does not cut) keeps the plain path.
            const bool every = (mb[0] & mb[1] & mb[2] & mb[3]) == 0xffffffffu &&
                               (p.window <= 0 || qpos - kb <= p.window);
            if (!every) {
#pragma unroll
              for (int i = 0; i < C::BN; ++i) {
                const int kpos = kb + i;
                const bool vis = ((mb[i >> 5] >> (i & 31)) & 1u) &&
                                 (p.window <= 0 || qpos - kpos <= p.window);
                x[i] = vis ? x[i] * sc : -INFINITY;
              }
              sc = 1.0f;
            }
          } else if (BITS && need_mask) {
            // numbers of the row's last key (causal, end of the tile) and of
            // the first one in its window; a word of bits for every 32 keys of
            // the tile, tested one by one.  The logits keep their scale (it is
            // positive), so a hidden one is -inf before it.  Three comparisons
            // and a product a key took 45 of 179 us on 16 sequences of up to
            // (4096 + 1024) tokens with a window of 1024.
            int vhi = qpos, vlo = p.window > 0 ? qpos - p.window : 0;
            uint32_t bits[4];
            if constexpr (FIRST) {
              vhi = qpos - gap >= p.first ? qpos - gap : min(qpos, p.first - 1);
              vlo -= gap;
            }
            vhi = min(vhi, ke - 1);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int k0 = kb + 32 * q, lo = max(vlo - k0, 0);
              bits[q] = bit_range(lo, vhi + 1 - k0 - lo);
              if constexpr (FIRST) bits[q] |= bit_range(0, min(p.first, vhi + 1) - k0);
            }
#pragma unroll
            for (int i = 0; i < C::BN; ++i)
              if (!((bits[i >> 5] >> (i & 31)) & 1u)) x[i] = -INFINITY;
          } else if (need_mask) {
#pragma unroll
            for (int i = 0; i < C::BN; ++i) {
              const int kpos = kb + i;
              const bool vis =
                  kpos < ke && kpos <= qpos && (p.window <= 0 || qpos - kpos <= p.window);
              x[i] = vis ? x[i] * sc : -INFINITY;
            }
            sc = 1.0f;
          }
          // row max of sc * x: sc * max(x), or sc * min(x) for a negative sc
          float mt;
          if (sc >= 0.f) {
            float mt0 = x[0], mt1 = x[1], mt2 = x[2], mt3 = x[3];
#pragma unroll
            for (int i = 4; i < C::BN; i += 4) {
              mt0 = fmaxf(mt0, x[i]);
              mt1 = fmaxf(mt1, x[i + 1]);
              mt2 = fmaxf(mt2, x[i + 2]);
              mt3 = fmaxf(mt3, x[i + 3]);
            }
            mt = fmaxf(fmaxf(mt0, mt1), fmaxf(mt2, mt3)) * sc;
          } else {
            float mt0 = x[0], mt1 = x[1], mt2 = x[2], mt3 = x[3];
#pragma unroll
            for (int i = 4; i < C::BN; i += 4) {
              mt0 = fminf(mt0, x[i]);
              mt1 = fminf(mt1, x[i + 1]);
              mt2 = fminf(mt2, x[i + 2]);
              mt3 = fminf(mt3, x[i + 3]);
            }
            mt = fminf(fminf(mt0, mt1), fminf(mt2, mt3)) * sc;
          }
          const float m_new = fmaxf(m, mt);
          // Rescale only when the max grows by more than 2^8: exponents of
          // the stale max stay below 256, which fp32 sums and bf16 P hold.
          // (S_full of this tile completes after the previous PV, so O is
          // quiescent here.  A 4-bit pool: kF4Lag.)
          const bool grow = m_new > m + (F4 ? kF4Lag : 8.0f);
          const float alpha = grow ? ex2_approx(m - m_new) : 1.0f;
          const bool o_needs = grow && j > j0 && l > 0.f;
          if (grow) {
            l *= alpha;
            m = m_new;
          }
          const float mref = m == -INFINITY ? 0.f : m;
          // p = 2^(sc * x - m): one FMA into each exp2
          float nm = -mref;
          float lscale = 1.0f;
          if constexpr (FMT != 0 && !F16) {
            if constexpr (F4) {
              nm += kF4Shift;
              // the output takes v_scale; P of a tile of extend rows is
              // divided by it (bf16 has the range, the f16 P of a pool tile
              // has not)
              if (!pool8) {
                nm -= p.log2_v_scale;
                lscale = p.v_scale;
              }
            } else if (pool8) {
              nm += p.log2_v_scale;
              lscale = p.inv_v_scale;
            }
          }
          float l0 = 0.f, l1 = 0.f;
          uint32_t pk[C::BN / 2];
#pragma unroll
          for (int i = 0; i < C::BN; i += 2) {
            const float e0 = ex2_approx(fmaf(x[i], sc, nm));
            const float e1 = ex2_approx(fmaf(x[i + 1], sc, nm));
            l0 += e0;
            l1 += e1;
            const __half2 h = __floats2half2_rn(e0, e1);
            const uint32_t h2 = *reinterpret_cast<const uint32_t *>(&h);
            if constexpr (F16) pk[i / 2] = h2;
            else if constexpr (F4) pk[i / 2] = pool8 ? h2 : pack_bf16(e0, e1);
            else pk[i / 2] = pack_bf16(e0, e1);
          }
          if constexpr (FMT != 0) l += (l0 + l1) * lscale;
          else l += l0 + l1;
          // P (bf16 pairs) over the first 64 columns of this tile's S.
          {
            uint32_t a[32], b[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              a[i] = pk[i];
              b[i] = pk[32 + i];
            }
            tmem_st32(lane_base + s_col + 0, a);
            tmem_st32(lane_base + s_col + 32, b);
          }
          if (__any_sync(0xffffffffu, o_needs)) {
            const float a = o_needs ? alpha : 1.0f;
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < C::HDV / 32; ++c) {
              const uint32_t ta = lane_base + o_col + c * 32;
              tmem_ld32(ta, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * a);
              tmem_st32(ta, v);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_P_FULL + wg]);
      }
      if (*abort_flag) break;
      // epilogue: wait for the last PV of this tile, normalise, store
      if (!mbar_wait(&bars[B_O_DONE + wg], o_cnt & 1u, abort_flag, p.wait_ns)) {
        abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
        break;
      }
      ++o_cnt;
      tc_fence_after();
      if (warp_active) {
        if constexpr (F4) m -= kF4Shift;  // l and O are 2^kF4Shift times too large
        // a sum of 0: no visible key; a NaN sum (a NaN query or key) stays NaN
        float inv = l == 0.f ? 0.f : 1.0f / l;
        float lse_v = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
        if (p.sinks && w.slot < 0) {
          // the head's sink joins the denominator (a split row gets it in
          // the combine): with M = max(m, sink), l' = l 2^(m-M) + 2^(sink-M)
          const float s2 = __ldg(p.sinks + w.kvh * G + g) * 1.4426950408889634f;
          const float M = fmaxf(m, s2);
          const float a_m = m == -INFINITY ? 0.f : ex2_approx(m - M);
          const float lt = l * a_m + ex2_approx(s2 - M);
          inv = a_m / lt;
          lse_v = (M + __log2f(lt)) * 0.69314718055994531f;
        }
        if constexpr (F16 || F4) inv *= p.v_scale;  // V was read as its codes
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < C::HDV / 32; ++c) {
          tmem_ld32(lane_base + o_col + c * 32, v);
          tmem_wait_ld();
          if (valid) {
            if (w.slot < 0) {
              bf16 *orow = p.o + orow_idx * C::HDV + c * 32;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint4 q4;
                q4.x = pack_bf16(__uint_as_float(v[i + 0]) * inv, __uint_as_float(v[i + 1]) * inv);
                q4.y = pack_bf16(__uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv);
                q4.z = pack_bf16(__uint_as_float(v[i + 4]) * inv, __uint_as_float(v[i + 5]) * inv);
                q4.w = pack_bf16(__uint_as_float(v[i + 6]) * inv, __uint_as_float(v[i + 7]) * inv);
                *reinterpret_cast<uint4 *>(orow + i) = q4;
              }
            } else {
              float *prow = p.po + prow_idx * C::HDV + c * 32;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4 *>(prow + i) =
                    make_float4(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv,
                                __uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv);
            }
          }
        }
        if (valid) {
          if (w.slot < 0) {
            if (p.lse) p.lse[orow_idx] = lse_v;
          } else {
            p.plse[prow_idx] = lse_v;
          }
        }
      }
      tc_fence_before();
    }
  } else {
  regs_decrease<C::REGS_OTHER>();
  if (warp == 8) {
    // ------------------------------------------------ MMA issue (one warp)
    // All 32 lanes run the loop (and its waits), so the descriptors and
    // counters stay warp-uniform; one elected lane issues each tcgen05
    // operation.  The same loop run by lane 0 alone issued about 25 %
    // slower.
    {
      const bool leader = elect_one();
      uint32_t q_cnt = 0, kc = 0, vc = 0, p_cnt0 = 0, p_cnt1 = 0;
      const uint32_t sQ0 = sbase + C::OFF_Q, sQ1 = sQ0 + C::Q_BYTES;
      bool ok = true;
      // Descriptors are built once per tile and stepped by constants: the
      // issue path is a single thread, and a per-MMA dependent chain of
      // address arithmetic starves the tensor pipe.
      constexpr uint32_t K_LO = sw128_desc_lo(0), K_HI = sw128_desc_hi(1024);
      constexpr uint32_t V_LO = sw128_desc_lo(C::BN * 128), V_HI = sw128_desc_hi(1024);
      auto issue_s = [&](int qt, uint32_t sK) {
        const uint32_t a_lo = K_LO | desc_addr(qt ? sQ1 : sQ0), b_lo = K_LO | desc_addr(sK);
        const uint32_t d = tmem + qt * C::BN;
        static_for<0, C::LQ / 16>([&](auto kk_c) {
          constexpr int kk = decltype(kk_c)::value;
          constexpr uint32_t ao = ((kk / 4) * (C::BM * 128) + (kk % 4) * 32) / 16;
          constexpr uint32_t bo = ((kk / 4) * (C::BN * 128) + (kk % 4) * 32) / 16;
          if (leader) tc_mma_ss_step<ao, bo>(d, a_lo, b_lo, K_HI, IDQK, kk > 0 ? 1u : 0u);
        });
        if (leader) tc_commit(&bars[B_S_FULL + qt]);
      };
      // S of query tile 0 into S/P buffer `buf` (the decode streams)
      auto issue_s_q0 = [&](int buf, uint32_t sK) {
        const uint32_t a_lo = K_LO | desc_addr(sQ0), b_lo = K_LO | desc_addr(sK);
        const uint32_t d = tmem + buf * C::BN;
        static_for<0, C::LQ / 16>([&](auto kk_c) {
          constexpr int kk = decltype(kk_c)::value;
          constexpr uint32_t ao = ((kk / 4) * (C::BM * 128) + (kk % 4) * 32) / 16;
          constexpr uint32_t bo = ((kk / 4) * (C::BN * 128) + (kk % 4) * 32) / 16;
          if (leader) tc_mma_ss_step<ao, bo>(d, a_lo, b_lo, K_HI, IDQK, kk > 0 ? 1u : 0u);
        });
        if (leader) tc_commit(&bars[B_S_FULL + buf]);
      };
      // (4-bit pool: the first n_pool tiles of a unit have f16 V and P, the
      // tiles of extend rows bf16)
      [[maybe_unused]] int n_pool = 0;
      auto issue_pv = [&](int qt, uint32_t sV, bool acc_first, [[maybe_unused]] int tile) {
        uint32_t idpv = IDPV;
        if constexpr (F4) idpv = tile < n_pool ? idesc_f16_f32(C::BM, C::HDV, 1) : IDPV;
        const uint32_t b_lo = V_LO | desc_addr(sV);
        const uint32_t d = tmem + 2 * C::BN + qt * C::HDV, a = tmem + qt * C::BN;
        const uint32_t acc0 = acc_first ? 1u : 0u;
        static_for<0, C::BN / 16>([&](auto kk_c) {
          constexpr int kk = decltype(kk_c)::value;
          if (leader) tc_mma_ts_step<kk * 8, kk * 128>(d, a, b_lo, V_HI, idpv, kk > 0 ? 1u : acc0);
        });
      };
      for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
        const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ok, p.wait_ns);
        if (u < 0) break;
        const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
        const int nt = w.n_tiles;
        if (nt == 0) continue;
        if constexpr (F4) {  // tile_keys()'s count of tiles before k_split
          const int pe = min(w.k_end, w.k_split);
          n_pool = pe > w.k_begin ? (pe - w.k_begin + C::BN - 1) / C::BN : 0;
        }
        const bool q1 = w.n_tok > TOK;
        if (!mbar_wait(&bars[F16 ? B_Q_CONV : B_Q_FULL], q_cnt & 1u, abort_flag, p.wait_ns)) {
          ok = false;
          break;
        }
        ++q_cnt;
        tc_fence_after();
        if (C::TWO_OK && (MODE == kDecode ? p.dec_two != 0 : (w.slot >= 0 && !q1))) {
          // Two key streams over the one query tile: even tiles into S/P
          // buffer 0 (softmax warpgroup 0, O 0), odd tiles into buffer 1
          // (warpgroup 1, O 1).  S(j) waits only for PV(j-2), which reads
          // the P it overwrites, so one stream's softmax runs while the
          // other's products do.
          for (int j = 0; j < nt && ok; ++j) {
            const int b = j & 1;
            if (j >= 2) {
              const int vs = vc % C::NV;
              uint32_t &pc = b ? p_cnt1 : p_cnt0;
              if (!mbar_wait(&v_full[vs], (vc / C::NV) & 1u, abort_flag, p.wait_ns) ||
                  !mbar_wait(&bars[B_P_FULL + b], pc & 1u, abort_flag, p.wait_ns)) {
                ok = false;
                break;
              }
              ++pc;
              fence_proxy_async_smem();
              tc_fence_after();
              issue_pv(b, sbase + C::OFF_V + vs * C::V_BYTES, j >= 4, j - 2);
              if (leader) tc_commit(&v_empty[vs]);
              ++vc;
            }
            const int ks = kc % NK_;
            if (!mbar_wait(&k_full[ks], (kc / NK_) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
            fence_proxy_async_smem();
            tc_fence_after();
            issue_s_q0(b, sbase + K0 + ks * C::K_BYTES);
            if (leader) tc_commit(&k_empty[ks]);
            ++kc;
            if (j == nt - 1 && leader) tc_commit(&bars[B_Q_EMPTY]);
          }
          // the last PV of each stream, in tile order
          for (int j = nt >= 2 ? nt - 2 : 0; j < nt && ok; ++j) {
            const int b = j & 1;
            const int vs = vc % C::NV;
            uint32_t &pc = b ? p_cnt1 : p_cnt0;
            if (!mbar_wait(&v_full[vs], (vc / C::NV) & 1u, abort_flag, p.wait_ns) ||
                !mbar_wait(&bars[B_P_FULL + b], pc & 1u, abort_flag, p.wait_ns)) {
              ok = false;
              break;
            }
            ++pc;
            fence_proxy_async_smem();
            tc_fence_after();
            issue_pv(b, sbase + C::OFF_V + vs * C::V_BYTES, j >= 2, j);
            if (leader) tc_commit(&bars[B_O_DONE + b]);
            if (leader) tc_commit(&v_empty[vs]);
            ++vc;
          }
          continue;
        }
        // tile 0: S of both Q tiles
        {
          const int ks = kc % NK_;
          if (!mbar_wait(&k_full[ks], (kc / NK_) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          fence_proxy_async_smem();  // cp.async (generic proxy) -> tcgen05.mma reads
          tc_fence_after();
          const uint32_t sK = sbase + K0 + ks * C::K_BYTES;
          issue_s(0, sK);
          if (q1) issue_s(1, sK);
          if (leader) tc_commit(&k_empty[ks]);
          ++kc;
          if (nt == 1 && leader) tc_commit(&bars[B_Q_EMPTY]);
        }
        for (int j = 1; j < nt && ok; ++j) {
          const int ks = kc % NK_, vs = vc % C::NV;
          if (!mbar_wait(&k_full[ks], (kc / NK_) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          if (!mbar_wait(&v_full[vs], (vc / C::NV) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          if (!mbar_wait(&bars[B_P_FULL + 0], p_cnt0 & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          ++p_cnt0;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t sK = sbase + K0 + ks * C::K_BYTES;
          const uint32_t sV = sbase + C::OFF_V + vs * C::V_BYTES;
          issue_pv(0, sV, j > 1, j - 1);
          issue_s(0, sK);
          if (q1) {
            if (!mbar_wait(&bars[B_P_FULL + 1], p_cnt1 & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
            ++p_cnt1;
            tc_fence_after();
            issue_pv(1, sV, j > 1, j - 1);
            issue_s(1, sK);
          }
          if (leader) tc_commit(&v_empty[vs]);
          ++vc;
          if (leader) tc_commit(&k_empty[ks]);
          ++kc;
          if (j == nt - 1 && leader) tc_commit(&bars[B_Q_EMPTY]);
        }
        if (!ok) break;
        // last PV of both Q tiles
        {
          const int vs = vc % C::NV;
          if (!mbar_wait(&v_full[vs], (vc / C::NV) & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          if (!mbar_wait(&bars[B_P_FULL + 0], p_cnt0 & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
          ++p_cnt0;
          fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t sV = sbase + C::OFF_V + vs * C::V_BYTES;
          issue_pv(0, sV, nt > 1, nt - 1);
          if (leader) tc_commit(&bars[B_O_DONE + 0]);
          if (q1) {
            if (!mbar_wait(&bars[B_P_FULL + 1], p_cnt1 & 1u, abort_flag, p.wait_ns)) { ok = false; break; }
            ++p_cnt1;
            tc_fence_after();
            issue_pv(1, sV, nt > 1, nt - 1);
            if (leader) tc_commit(&bars[B_O_DONE + 1]);
          }
          if (leader) tc_commit(&v_empty[vs]);
          ++vc;
        }
      }
      if (!ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
      // drain: every MMA issued above must finish before TMEM is freed
      if (leader) tc_commit(&bars[B_FINAL]);
      if (!mbar_wait_drain(&bars[B_FINAL], 0)) record_status(p.status, PKX_ETIMEOUT);
    }
  } else if (warp == 9) {
    // --------------------------------------- Q tiles and row indices
    // Lane 0 loads each unit's Q tiles (3-D TMA box: 64 dims, G heads,
    // q_box_tok tokens; rows t * G + g).  Every lane resolves 4 keys of each
    // tile to a pool slot (or extend row) into the index ring, ahead of the
    // copy warps; -1 marks a key to zero-fill (past the tile's end, or an
    // out-of-range slot, which is also recorded).
    uint32_t q_cnt = 0, ic = 0;
    if (lane == 0) prefetch_tensormap(&tm.q);
    const uint32_t tile_box_bytes = 64u * 2u * G * p.q_box_tok;
    bool ok = true;
    for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
      // claim the next unit and hand it to the other warps
      int u = -1;
      if (lane == 0) {
        if (p.part_first) {  // stream partition: this CTA's share, in order
          const int pos = p.part_first[blockIdx.x] + (int)uc;
          u = pos < p.part_first[blockIdx.x + 1] ? pos : -1;
        } else {
          // (listed units are claimed from the grid's size on: the first is the
          // CTA's own)
          const int pos = MODE != kListed ? atomicAdd(p.next_unit, 1)
                          : uc == 0       ? (int)blockIdx.x
                                          : (int)gridDim.x + atomicAdd(p.next_unit, 1);
          u = pos < n_units ? pos : -1;
        }
      }
      u = __shfl_sync(0xffffffffu, u, 0);
      {
        const int slot = uc % kUnitRing;
        if (uc >= (uint32_t)kUnitRing &&
            !mbar_wait(&bars[B_U_EMPTY + slot], ((uc / kUnitRing) - 1) & 1u, abort_flag, p.wait_ns)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          s_unit[slot] = u;
          mbar_arrive(&bars[B_U_FULL + slot]);
        }
      }
      if (u < 0) break;
      const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
      const int nt = w.n_tiles;
      if (nt == 0) continue;
      const bool q1 = w.n_tok > TOK;
      if (lane == 0) {
        if (q_cnt > 0 && !mbar_wait(&bars[B_Q_EMPTY], (q_cnt - 1) & 1u, abort_flag, p.wait_ns)) ok = false;
        if (ok) {
          const int nq = q1 ? 2 : 1;
          const CUtensorMap *map = &tm.q;
          uint32_t q_box_bytes = tile_box_bytes;
          if constexpr (MODE == kListed) {
            if (w.n_tok == 1) {  // only the one token's rows
              map = &tm.one;
              q_box_bytes = 64u * 2u * G;
            }
          }
          mbar_arrive_expect_tx(&bars[B_Q_FULL], q_box_bytes * C::QA * nq);
          for (int qt = 0; qt < nq; ++qt)
            for (int h = 0; h < C::QA; ++h)
              tma_load_3d(sbase + C::OFF_Q + qt * C::Q_BYTES + h * (C::BM * 128), map, h * 64,
                          w.kvh * G, w.q_tok0 + qt * TOK, &bars[B_Q_FULL]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ++q_cnt;
      const int64_t kv_base = p.kv_indptr[w.b];
      const int64_t ext_base = MODE == kTwoStage ? p.qo_indptr[w.b] : 0;
      const int gap = FIRST ? block_gap(w.qpos0, p.window, p.first) : 0;
      // position of the first extend key
      const int ext_pos = FIRST && MODE == kTwoStage ? (int)(p.kv_indptr[w.b + 1] - kv_base)
                                                     : w.k_split;
      for (int j = 0; j < nt; ++j) {
        int kb, ke;
        tile_keys(w, j, kb, ke);
        const bool from_ext = MODE == kTwoStage && kb >= w.k_split;
        int rows[4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int jpos = kb + 4 * lane + i;
          int64_t row = -1;
          if (jpos < ke) {
            if (FIRST && jpos >= p.first) jpos += gap;
            if (from_ext) {
              row = ext_base + (jpos - ext_pos);
            } else {
              row = MODE == kUnified
                        ? __ldg(static_cast<const int64_t *>(p.kv_indices) + kv_base + jpos)
                        : (int64_t)__ldg(static_cast<const int32_t *>(p.kv_indices) + kv_base + jpos);
              if (row < 0 || row >= p.num_slots) {
                bad = true;
                row = -1;
              }
            }
          }
          rows[i] = (int)row;
        }
        if (bad) record_status(p.status, PKX_EDEVICE);
        const int is = ic % C::NI;
        if (ic >= (uint32_t)C::NI &&
            !mbar_wait(&i_empty[is], ((ic / C::NI) - 1) & 1u, abort_flag, p.wait_ns)) {
          ok = false;
          break;
        }
        {
          // ring[key % KPP][key / KPP]: each copy thread's rows contiguous
          constexpr int KPP = C::KPP, NK_T = C::BN / KPP;
          int *ring = reinterpret_cast<int *>(smem + C::OFF_I + is * C::I_BYTES);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 4 * lane + i;
            ring[(key % KPP) * NK_T + key / KPP] = rows[i];
          }
        }
        mbar_arrive(&i_full[is]);
        ++ic;
      }
    }
    if (!ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
    // the last Q load this warp issued lands before the CTA may exit (after
    // an abort nobody else may have waited for it)
    if (lane == 0 && q_cnt > 0 && !mbar_wait_drain(&bars[B_Q_FULL], (q_cnt - 1) & 1u))
      record_status(p.status, PKX_ETIMEOUT);
    __syncwarp();
  } else if (F16 && warp >= 12) {
    // ------------------------------- fp8 codes -> f16 stages (warps 12-15)
    // Decode over an fp8 pool: each raw slot (K(j) and V(j) alternate, in
    // the order the copying warps issue them) is converted into the next
    // stage of its ring once its codes have landed and the stage is free;
    // warps 12-13 take the K slots and 14-15 the V slots, so that neither
    // ring waits behind the other.  Chunk c of a slot holds the eight codes
    // of key c / CPR, dims 8 (c % CPR) + [0, 8); thread cv of a group
    // converts chunks cv + 64 m, so a warp reads 256 contiguous bytes and
    // writes whole 128-byte rows of the swizzled stage.  Its chunk index
    // (c % CPR) and the key's swizzle phase are the same for every m, so
    // source and destination step by constants.  All four warps convert
    // each unit's query rows to f16 (Q_CONV).
    if constexpr (F16) {
    constexpr int CPR = HD / 8;
    constexpr int NCH = C::BN * CPR / CONV_THREADS;
    constexpr int KSTEP = CONV_THREADS / CPR;  // keys between a thread's chunks
    // swizzle phases (key % 8) a thread's keys cycle through
    constexpr int NPH = KSTEP % 8 == 0 ? 1 : 8 / KSTEP;
    static_assert(C::BN * CPR % CONV_THREADS == 0 && NCH % NPH == 0 &&
                      (KSTEP % 8 == 0 || 8 % KSTEP == 0),
                  "conversion geometry");
    const int grp = warp >= 14;                // 0: K slots, 1: V slots
    const int cq = tid - 12 * 32;              // 0 .. 127 for the query rows
    const int cv = cq - grp * CONV_THREADS;    // 0 .. 63 within the group
    const int ck = cv % CPR, key0 = cv / CPR;
    const uint32_t sthr = (uint32_t)cv * 8u;
    uint32_t dthr[NPH];  // chunk m = NPH mm + ph: key key0 + KSTEP m
#pragma unroll
    for (int ph = 0; ph < NPH; ++ph) {
      const int key = key0 + KSTEP * ph;
      dthr[ph] = (uint32_t)(ck >> 3) * (C::BN * 128) + (uint32_t)key * 128u +
                 ((uint32_t)((ck & 7) ^ (key & 7)) << 4);
    }
    uint32_t rc = grp, kc = 0, vc = 0, qc = 0;  // rc: slot use (K even, V odd)
    bool ok = true;
    // the group's next slot into `stage` once both are ready
    auto convert_slot = [&](uint64_t *st_empty, uint32_t n_used, int n_stages, uint32_t stage,
                            uint64_t *st_full) -> bool {
      const int s = rc % C::NRAW;
      if (!mbar_wait(&raw_full[s], (rc / C::NRAW) & 1u, abort_flag, p.wait_ns)) return false;
      if (n_used >= (uint32_t)n_stages &&
          !mbar_wait(st_empty, ((n_used / n_stages) - 1) & 1u, abort_flag, p.wait_ns))
        return false;
      const uint32_t src = sbase + C::OFF_RAW + s * C::RAW_BYTES + sthr;
#pragma unroll 2
      for (int mm = 0; mm < NCH / NPH; ++mm) {
#pragma unroll
        for (int ph = 0; ph < NPH; ++ph)
          st_shared_u4(stage + dthr[ph] + mm * (KSTEP * NPH * 128),
                       fp8x8_to_f16x8<FMT>(
                           ld_shared_u2(src + (mm * NPH + ph) * (CONV_THREADS * 8))));
      }
      fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
      mbar_arrive(st_full);
      mbar_arrive(&raw_empty[s]);
      rc += 2;
      return true;
    };
    for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
      const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ok, p.wait_ns);
      if (u < 0) break;
      const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
      const int nt = w.n_tiles;
      if (nt == 0) continue;
      // the unit's query rows (tokens x G heads of query tile 0) to f16 in
      // place once their load has landed, 16 bytes at a time (the swizzle
      // only permutes whole chunks within a row)
      if (!mbar_wait(&bars[B_Q_FULL], qc & 1u, abort_flag, p.wait_ns)) {
        ok = false;
        break;
      }
      ++qc;
      const int n_chunks = w.n_tok * G * (HD / 8);
      for (int c = cq; c < n_chunks; c += 2 * CONV_THREADS) {
        const int row = c / (HD / 8), k = c % (HD / 8);
        const uint32_t off = C::OFF_Q + (uint32_t)(k >> 3) * (C::BM * 128) + (uint32_t)row * 128u +
                             (uint32_t)(k & 7) * 16u;
        const uint4 v = *reinterpret_cast<const uint4 *>(smem + off);
        st_shared_u4(sbase + off, bf16x8_to_f16x8_scaled(v));
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars[B_Q_CONV]);
      for (int j = 0; j < nt; ++j) {
        const int ks = kc % NK_, vs = vc % C::NV;
        if (grp == 0 ? !convert_slot(&k_empty[ks], kc, NK_, sbase + K0 + ks * C::K_BYTES, &k_full[ks])
                     : !convert_slot(&v_empty[vs], vc, C::NV, sbase + C::OFF_V + vs * C::V_BYTES,
                                     &v_full[vs])) {
          ok = false;
          break;
        }
        if (grp == 0) ++kc;
        else ++vc;
      }
    }
    if (!ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
    }
  } else if (F16) {
    // ------------------------------------ fp8 codes into raw slots (warps 10-11)
    // Decode over an fp8 pool: the codes of each K and V tile go
    // fire-and-forget into the next slot of the raw ring (row-major, 8 bytes
    // per (key, chunk)) once the converting warps have read what it held;
    // each thread arrives (noinc) on the slot's barrier when its own copies
    // land.  Thread ct copies chunk ct % CPR of keys ct / CPR + KG i.
    if constexpr (F16) {
    constexpr int CPR = HD / 8, KG = RAW_THREADS / CPR, NKEYS = C::BN / KG;
    constexpr int KPP = C::KPP, NK_T = C::BN / KPP;  // the index ring's layout
    static_assert(KG * CPR == RAW_THREADS && C::BN % KG == 0, "copy geometry");
    const int ct = tid - C::COPY_WARP0 * 32;
    const int ch = ct % CPR, kg = ct / CPR;
    const uint32_t rthr = (uint32_t)(kg * CPR + ch) * 8u;
    uint32_t rc = 0, ic = 0;
    bool ok = true;
    for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
      const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ok, p.wait_ns);
      if (u < 0) break;
      const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
      const int nt = w.n_tiles;
      if (nt == 0) continue;
      const uint8_t *kp8 =
          reinterpret_cast<const uint8_t *>(p.k_pool) + (int64_t)w.kvh * p.kb_sh + ch * 8;
      const uint8_t *vp8 =
          reinterpret_cast<const uint8_t *>(p.v_pool) + (int64_t)w.kvh * p.vb_sh + ch * 8;
      for (int j = 0; j < nt && ok; ++j) {
        // this thread's rows (the index ring holds key's row at
        // [key % KPP][key / KPP])
        const int is = ic % C::NI;
        if (!mbar_wait(&i_full[is], (ic / C::NI) & 1u, abort_flag, p.wait_ns)) {
          ok = false;
          break;
        }
        int rows[NKEYS];
        {
          const int *ring = reinterpret_cast<const int *>(smem + C::OFF_I + is * C::I_BYTES);
#pragma unroll
          for (int i = 0; i < NKEYS; ++i) {
            const int key = kg + KG * i;
            rows[i] = ring[(key % KPP) * NK_T + key / KPP];
          }
        }
        __syncwarp();  // the warp is done with the ring slot
        if (lane == 0) mbar_arrive(&i_empty[is]);
        ++ic;
        for (int t = 0; t < 2; ++t) {  // K(j), then V(j)
          const int s = rc % C::NRAW;
          if (rc >= (uint32_t)C::NRAW &&
              !mbar_wait(&raw_empty[s], ((rc / C::NRAW) - 1) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          const uint8_t *base = t == 0 ? kp8 : vp8;
          const int64_t stride = t == 0 ? p.kb_ss : p.vb_ss;
          const uint32_t slot = sbase + C::OFF_RAW + s * C::RAW_BYTES + rthr;
          static_for<0, NKEYS>([&](auto i_c) {
            constexpr int i = decltype(i_c)::value;
            const int r = rows[i];
            const uint8_t *src = base + (int64_t)max(r, 0) * stride;
            cp_async_8_at<i * KG * CPR * 8>(slot, src, r >= 0 ? 8u : 0u);
          });
          cp_async_arrive_noinc(&raw_full[s]);
          ++rc;
        }
      }
    }
    if (!ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
    cp_async_wait_all();
    }
  } else if (F4) {
    // ---------------------- extend over a 4-bit pool (warps 10-15)
    // Warp 10 copies the K tiles into their stages and warp 11 the V tiles;
    // warps 12-13 convert K in place to bf16 (Q's type) and 14-15 V to f16,
    // which takes half the time: P of a pool tile is f16 too, and the output
    // takes v_scale.  Copies and conversions of
    // K and of V thus wait for nothing of each other: with four warps that
    // copied and converted both in turn, a tile was a chain of two conversions,
    // two landings and the product that frees V's stage (678 us on
    // 64 x (8192 + 16), 32 and 8 heads of 128; 453 now, as over a bf16 pool).
    // A lane takes chunk q4 (16 code bytes, 32 elements) of its keys: the codes
    // land in the first of the four 16-byte chunks that their bf16 fill, and a
    // key's block scales in the second chunk of its row, so that only lanes of
    // the converting warp that holds all of a key overwrite what it still
    // reads (they load first).  Neighbouring lanes hold consecutive keys of one
    // chunk: their stores lie in different banks.  Every tile's landing is one
    // phase of its stage's raw barrier; a tile of extend rows (bf16) passes
    // through the converting warps untouched.
    if constexpr (F4) {
    static_assert(!C::SPLIT, "4-bit pools are built for Lq = Lv");
    constexpr int Q4 = HD / 32, KPW = 32 / Q4;  // chunks of a row; keys of a warp's pass
    static_assert(KPW == C::KPP, "the index ring's layout");
    const int q4 = lane / KPW, kl = lane % KPW;
    // sub-chunk s of the lane's four: chunk c4 ^ s of its row's swizzled atom
    const uint32_t c4 = (uint32_t)((4 * (q4 & 1)) ^ (kl & 7));
    const uint32_t d4 = (uint32_t)(q4 >> 1) * (C::BN * 128) + (uint32_t)kl * 128u;
    const uint32_t sc4 = (uint32_t)kl * 128u + (((uint32_t)(kl & 7) ^ 1u) << 4);  // block scales
    static_assert(C::K_BYTES == C::V_BYTES, "one stage size");
    const bool is_v = warp == 11 || warp >= 14;
    uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
    uint64_t *landed = is_v ? raw_full + C::NK : raw_full;
    const uint32_t n_stages = is_v ? C::NV : C::NK;
    const uint32_t stages = sbase + (is_v ? C::OFF_V : K0);
    constexpr uint32_t STAGE_BYTES = C::K_BYTES;
    // key groups [g0, g1) (KPW keys each) of the tile in `stage`, two at a time.
    // A loop, not unrolled: unrolled over a tile the code of the warps' roles
    // outgrew the instruction cache, and a word took 140 clocks.
    auto convert = [&](uint32_t stage, int g0, int g1, auto bf16_c) {
      constexpr bool BF16 = decltype(bf16_c)::value;
      constexpr int U = 2;
#pragma unroll 1
      for (uint32_t at = stage + g0 * (KPW * 128); at < stage + g1 * (KPW * 128);
           at += U * KPW * 128) {
        uint4 codes[U];
        __half2 sc[U][2];  // the chunk's two block scales, each twice
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint32_t key = at + i * (KPW * 128);
          codes[i] = ld_shared_u4(key + d4 + (c4 << 4));
          const uint2 sw = ld_shared_u2(key + sc4);
          const uint32_t two = (q4 & 2 ? sw.y : sw.x) >> (16 * (q4 & 1));
          const __half2 s = e4m3x2_to_f16x2(two & 0xFFFFu);
          sc[i][0] = __low2half2(s);
          sc[i][1] = __high2half2(s);
        }
        __syncwarp();  // every lane has read before any writes
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint32_t dst = at + d4 + i * (KPW * 128);
          const uint32_t x[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
          uint4 out[4];  // all four before a store, for the chains to overlap
#pragma unroll
          for (int sub = 0; sub < 4; ++sub) out[sub] = fp4x8_to_16bit<BF16>(x[sub], sc[i][sub >> 1]);
#pragma unroll
          for (int sub = 0; sub < 4; ++sub) st_shared_u4(dst + ((c4 ^ sub) << 4), out[sub]);
        }
      }
    };
    uint32_t c = 0, ic = 0;  // tiles of this warp's kind, so far
    bool ok = true;
    for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
      const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ok, p.wait_ns);
      if (u < 0) break;
      const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
      const int nt = w.n_tiles;
      auto from_ext = [&](int j) {
        int kb, ke;
        tile_keys(w, j, kb, ke);
        return MODE == kTwoStage && kb >= w.k_split;
      };
      if (warp < 12) {
        const uint8_t *pool = reinterpret_cast<const uint8_t *>(is_v ? p.v_pool : p.k_pool) +
                              (int64_t)w.kvh * (is_v ? p.vb_sh : p.kb_sh) + q4 * 16;
        const uint8_t *scales = (is_v ? p.v_bs : p.k_bs) +
                                (int64_t)w.kvh * (is_v ? p.vbs_sh : p.kbs_sh);
        const bf16 *ext = (is_v ? p.v_ext : p.k_ext) + (int64_t)w.kvh * (is_v ? p.ve_sh : p.ke_sh) +
                          q4 * 32;
        const int64_t ss = is_v ? p.vb_ss : p.kb_ss, sss = is_v ? p.vbs_ss : p.kbs_ss;
        const int64_t es = is_v ? p.ve_st : p.ke_st;
        constexpr int N = C::BN / KPW;  // keys of a lane
        for (int j = 0; j < nt; ++j) {
          const int is = ic % C::NI;
          if (!mbar_wait(&i_full[is], (ic / C::NI) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t st = c % n_stages;
          if (c >= n_stages && !mbar_wait(&empty[st], ((c / n_stages) - 1) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          // the lane's rows are contiguous in the ring, four to a load; loops
          // that are short in code, for the same reason as the conversion's
          const int4 *ring =
              reinterpret_cast<const int4 *>(smem + C::OFF_I + is * C::I_BYTES) + kl * (N / 4);
          const uint32_t stage = stages + st * STAGE_BYTES;
          const bool is_ext = from_ext(j);
#pragma unroll 1
          for (int i0 = 0; i0 < N; i0 += 4) {
            const int4 v = ring[i0 / 4];
            const int rows[4] = {v.x, v.y, v.z, v.w};
            const uint32_t dst = stage + d4 + i0 * (KPW * 128);
            if (is_ext) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const bf16 *src = ext + (int64_t)max(rows[i], 0) * es;
#pragma unroll
                for (int sub = 0; sub < 4; ++sub)
                  cp_async_16(dst + i * (KPW * 128) + ((c4 ^ sub) << 4), src + sub * 8,
                              rows[i] >= 0 ? 16u : 0u);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                cp_async_16(dst + i * (KPW * 128) + (c4 << 4), pool + (int64_t)max(rows[i], 0) * ss,
                            rows[i] >= 0 ? 16u : 0u);
              // block scales, one copy a key: chunk q4's lanes take every Q4-th key
#pragma unroll
              for (int i = 0; i < 4; i += Q4) {
                int row = rows[i];
#pragma unroll
                for (int k = 1; k < Q4; ++k)
                  if (q4 == k) row = rows[i + k];
                const uint32_t at = stage + sc4 + (i0 + i + q4) * (KPW * 128);
                const uint8_t *src = scales + (int64_t)max(row, 0) * sss;
                if constexpr (HD == 128) cp_async_8_at<0>(at, src, row >= 0 ? 8u : 0u);
                else cp_async_4_at<0>(at, src, row >= 0 ? 4u : 0u);
              }
            }
          }
          __syncwarp();  // the warp is done with the ring slot
          if (lane == 0) mbar_arrive(&i_empty[is]);
          ++ic;
          cp_async_arrive_noinc(&landed[st]);
          ++c;
        }
      } else {
        constexpr int HALF = C::BN / KPW / 2;  // key groups of each of the two warps
        const int g0 = (warp & 1) * HALF;
        for (int j = 0; j < nt; ++j) {
          const uint32_t st = c % n_stages;
          if (!mbar_wait(&landed[st], (c / n_stages) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          if (!from_ext(j)) {  // (rows of the new tokens are bf16 already)
            const uint32_t stage = stages + st * STAGE_BYTES;
            if (is_v) convert(stage, g0, g0 + HALF, std::false_type{});
            else convert(stage, g0, g0 + HALF, std::true_type{});
          }
          fence_proxy_async_smem();  // copies' and this warp's writes -> tensor-core reads
          mbar_arrive(&full[st]);
          ++c;
        }
      }
    }
    if (!ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
    cp_async_wait_all();
    }
  } else if (warp < C::COPY_WARP0 + C::COPY_THREADS / 32) {
    // ------------------------------------------------ K/V copies (4 warps)
    // Thread ct copies 16-byte chunk ch = ct % CPR of keys key0 + KPP * i
    // (key0 = ct / CPR): every copy instruction of a warp reads whole rows.
    // KPP is a multiple of 8, so the swizzle term (ch ^ key % 8) is fixed
    // per thread and key i lands at a constant offset from the thread's
    // destination base.  The index warp stores each thread's rows
    // contiguously (ring[key0][i]).  A thread arrives (noinc) on the stage
    // barrier when its own copies have landed.
    // Split head dims: thread ct copies chunk ct % 8 of every 64-dim atom of
    // keys ct / 8 + 16 i (KPP = 16), so the swizzle term is again fixed per
    // thread; a warp instruction reads four rows' 128-byte segments.
    const int ct = tid - C::COPY_WARP0 * 32;
    constexpr int CPR = C::SPLIT ? 8 : C::LQ / 8;  // chunk lanes of a key
    constexpr int KPP = C::KPP;                    // keys per pass
    constexpr int NKEYS = C::BN / KPP;             // keys per thread
    static_assert(KPP * CPR == C::COPY_THREADS, "copy geometry");
    static_assert(KPP % 8 == 0 && C::BN % KPP == 0, "constant swizzle per thread");
    const int ch = ct % CPR, key0 = ct / CPR;
    const uint32_t dthr = (uint32_t)(ch >> 3) * (C::BN * 128) + (uint32_t)key0 * 128u +
                          ((uint32_t)((ch & 7) ^ (key0 & 7)) << 4);
    // the thread's chunks of its NKEYS rows (of L elements) into a stage
    auto copy_rows = [&](uint32_t stage, const bf16 *base, int64_t stride, const int *rows,
                         auto l_c) {
      constexpr int L = decltype(l_c)::value;
      static_for<0, NKEYS>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
        const int r = rows[i];
        const uint32_t bytes = r >= 0 ? 16u : 0u;
        const bf16 *src = base + (int64_t)max(r, 0) * stride;
        if constexpr (!C::SPLIT) {
          static_assert(L == C::LQ || L == C::HDV, "row length");
          cp_async_16_at<i * KPP * 128, 0>(stage + dthr, src, bytes);
        } else {
          static_for<0, (L + 63) / 64>([&](auto a_c) {
            constexpr int a = decltype(a_c)::value;
            if (a * 8 + ch < L / 8)  // the last atom of a 288-dim row holds 4 chunks
              cp_async_16_at<a * C::BN * 128 + i * KPP * 128, a * 128>(stage + dthr, src, bytes);
          });
        }
      });
    };
    constexpr std::integral_constant<int, C::LQ> K_LEN{};
    constexpr std::integral_constant<int, C::HDV> V_LEN{};
    uint32_t kc = 0, vc = 0, ic = 0;
    [[maybe_unused]] uint32_t qc = 0;
    bool ok = true;
    if constexpr (FMT == 0 || F4) {  // (F4 has its own warps, above)
      for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
        const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ok, p.wait_ns);
        if (u < 0) break;
        const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
        const int nt = w.n_tiles;
        if (nt == 0) continue;
        const bf16 *kp = p.k_pool + (int64_t)w.kvh * p.kb_sh + ch * 8;
        const bf16 *vp = p.v_pool + (int64_t)w.kvh * p.vb_sh + ch * 8;
        const bf16 *kx = p.k_ext + (int64_t)w.kvh * p.ke_sh + ch * 8;
        const bf16 *vx = p.v_ext + (int64_t)w.kvh * p.ve_sh + ch * 8;
        for (int j = 0; j < nt; ++j) {
          int kb, ke;
          tile_keys(w, j, kb, ke);
          const bool from_ext = MODE == kTwoStage && kb >= w.k_split;
          // this thread's rows from the index ring
          const int is = ic % C::NI;
          if (!mbar_wait(&i_full[is], (ic / C::NI) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          int rows[NKEYS];
          {
            const int4 *ring =
                reinterpret_cast<const int4 *>(smem + C::OFF_I + is * C::I_BYTES) + key0 * (NKEYS / 4);
  #pragma unroll
            for (int q = 0; q < NKEYS / 4; ++q) {
              const int4 v = ring[q];
              rows[4 * q] = v.x;
              rows[4 * q + 1] = v.y;
              rows[4 * q + 2] = v.z;
              rows[4 * q + 3] = v.w;
            }
          }
          __syncwarp();  // the warp is done with the ring slot
          if (lane == 0) mbar_arrive(&i_empty[is]);
          ++ic;
          // K tile
          const int ks = kc % NK_;
          if (kc >= (uint32_t)NK_ &&
              !mbar_wait(&k_empty[ks], ((kc / NK_) - 1) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          copy_rows(sbase + K0 + ks * C::K_BYTES, from_ext ? kx : kp,
                    from_ext ? p.ke_st : p.kb_ss, rows, K_LEN);
          cp_async_arrive_noinc(&k_full[ks]);
          ++kc;
          // V tile
          const int vs = vc % C::NV;
          if (vc >= (uint32_t)C::NV &&
              !mbar_wait(&v_empty[vs], ((vc / C::NV) - 1) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          copy_rows(sbase + C::OFF_V + vs * C::V_BYTES, from_ext ? vx : vp,
                    from_ext ? p.ve_st : p.vb_ss, rows, V_LEN);
          cp_async_arrive_noinc(&v_full[vs]);
          ++vc;
        }
      }
    } else {
    // extend over an fp8 pool.  A pool tile's codes are copied 8 bytes per (thread, key)
    // into the first half of the 16-byte chunk the same thread later
    // writes, and converted there in place to bf16 once they have landed, so no thread overwrites another's codes.  The copies
    // of tile j+1 go out before tile j is converted, in the order
    // K(j+1), convert K(j), V(j+1), convert V(j): V(j+1) reuses the stage of
    // V(j-1), which the tensor core frees only after K(j) is full.  Extend
    // tiles (bf16 rows of the two-stage form) take the plain copy.  One
    // cp.async group is committed per issued tile.
    // (split head dims: by 64-dim atom, as copy_rows does; a row of L codes)
    auto issue_raw = [&](uint32_t stage, const uint8_t *base, int64_t stride, const int *rows,
                         auto l_c) {
      constexpr int L = decltype(l_c)::value;
      static_for<0, NKEYS>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
        const int r = rows[i];
        const uint8_t *src = base + (int64_t)max(r, 0) * stride;
        if constexpr (!C::SPLIT) {
          static_assert(L == C::LQ || L == C::HDV, "row length");
          cp_async_8_at<i * KPP * 128>(stage + dthr, src, r >= 0 ? 8u : 0u);
        } else {
          static_for<0, (L + 63) / 64>([&](auto a_c) {
            constexpr int a = decltype(a_c)::value;
            if (a * 8 + ch < L / 8)
              cp_async_8_at<a * C::BN * 128 + i * KPP * 128>(stage + dthr, src + a * 64,
                                                             r >= 0 ? 8u : 0u);
          });
        }
      });
    };
    auto convert = [&](uint32_t stage, auto l_c) {
      constexpr int L = decltype(l_c)::value;
      static_for<0, NKEYS>([&](auto i_c) {
        constexpr int i = decltype(i_c)::value;
        if constexpr (!C::SPLIT) {
          const uint32_t a = stage + dthr + i * KPP * 128;
          st_shared_u4(a, fp8x8_to_bf16x8<FMT>(ld_shared_u2(a)));
        } else {
          static_for<0, (L + 63) / 64>([&](auto a_c) {
            constexpr int a = decltype(a_c)::value;
            if (a * 8 + ch < L / 8) {
              const uint32_t at = stage + dthr + a * C::BN * 128 + i * KPP * 128;
              st_shared_u4(at, fp8x8_to_bf16x8<FMT>(ld_shared_u2(at)));
            }
          });
        }
      });
      fence_proxy_async_smem();  // generic-proxy writes -> tensor-core reads
    };
    for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
      const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ok, p.wait_ns);
      if (u < 0) break;
      const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
      const int nt = w.n_tiles;
      if (nt == 0) continue;
      const uint8_t *kp8 =
          reinterpret_cast<const uint8_t *>(p.k_pool) + (int64_t)w.kvh * p.kb_sh + ch * 8;
      const uint8_t *vp8 =
          reinterpret_cast<const uint8_t *>(p.v_pool) + (int64_t)w.kvh * p.vb_sh + ch * 8;
      const bf16 *kx = p.k_ext + (int64_t)w.kvh * p.ke_sh + ch * 8;
      const bf16 *vx = p.v_ext + (int64_t)w.kvh * p.ve_sh + ch * 8;
      int rows[NKEYS];
      auto tile_from_ext = [&](int j) {
        int kb, ke;
        tile_keys(w, j, kb, ke);
        return MODE == kTwoStage && kb >= w.k_split;
      };
      auto fetch = [&]() -> bool {
        const int is = ic % C::NI;
        if (!mbar_wait(&i_full[is], (ic / C::NI) & 1u, abort_flag, p.wait_ns)) return false;
        const int4 *ring =
            reinterpret_cast<const int4 *>(smem + C::OFF_I + is * C::I_BYTES) + key0 * (NKEYS / 4);
#pragma unroll
        for (int q = 0; q < NKEYS / 4; ++q) {
          const int4 v = ring[q];
          rows[4 * q] = v.x;
          rows[4 * q + 1] = v.y;
          rows[4 * q + 2] = v.z;
          rows[4 * q + 3] = v.w;
        }
        __syncwarp();  // the warp is done with the ring slot
        if (lane == 0) mbar_arrive(&i_empty[is]);
        ++ic;
        return true;
      };
      auto issue_k = [&](bool from_ext) -> bool {
        const int ks = kc % NK_;
        if (kc >= (uint32_t)NK_ &&
            !mbar_wait(&k_empty[ks], ((kc / NK_) - 1) & 1u, abort_flag, p.wait_ns))
          return false;
        const uint32_t stage = sbase + K0 + ks * C::K_BYTES;
        if (from_ext) {
          copy_rows(stage, kx, p.ke_st, rows, K_LEN);
          cp_async_arrive_noinc(&k_full[ks]);
        } else {
          issue_raw(stage, kp8, p.kb_ss, rows, K_LEN);
        }
        cp_async_commit();
        ++kc;
        return true;
      };
      auto issue_v = [&](bool from_ext) -> bool {
        const int vs = vc % C::NV;
        if (vc >= (uint32_t)C::NV &&
            !mbar_wait(&v_empty[vs], ((vc / C::NV) - 1) & 1u, abort_flag, p.wait_ns))
          return false;
        const uint32_t stage = sbase + C::OFF_V + vs * C::V_BYTES;
        if (from_ext) {
          copy_rows(stage, vx, p.ve_st, rows, V_LEN);
          cp_async_arrive_noinc(&v_full[vs]);
        } else {
          issue_raw(stage, vp8, p.vb_ss, rows, V_LEN);
        }
        cp_async_commit();
        ++vc;
        return true;
      };
      if constexpr (NK_ < 2 || C::NV < 2) {
        // one K or one V stage (the 288 / 256 layout): the next tile's codes
        // could only go into the stage this tile holds, so each tile's codes
        // are converted as soon as they land
        for (int j = 0; j < nt; ++j) {
          const bool ext = tile_from_ext(j);
          if (!fetch() || !issue_k(ext)) {
            ok = false;
            break;
          }
          if (!ext) {
            cp_async_wait_group<0>();
            const int ks = (kc - 1) % NK_;
            convert(sbase + K0 + ks * C::K_BYTES, K_LEN);
            mbar_arrive(&k_full[ks]);
          }
          if (!issue_v(ext)) {
            ok = false;
            break;
          }
          if (!ext) {
            cp_async_wait_group<0>();
            const int vs = (vc - 1) % C::NV;
            convert(sbase + C::OFF_V + vs * C::V_BYTES, V_LEN);
            mbar_arrive(&v_full[vs]);
          }
        }
        continue;
      }
      bool ext_j = tile_from_ext(0);
      if (!fetch() || !issue_k(ext_j) || !issue_v(ext_j)) {
        ok = false;
        break;
      }
      for (int j = 0; j < nt; ++j) {
        const int ks_j = (kc - 1) % NK_, vs_j = (vc - 1) % C::NV;
        const bool more = j + 1 < nt;
        const bool ext_n = more && tile_from_ext(j + 1);
        if (more && (!fetch() || !issue_k(ext_n))) {
          ok = false;
          break;
        }
        if (!ext_j) {
          // groups issued after K(j): V(j), and K(j+1) if there is one
          if (more) cp_async_wait_group<2>();
          else cp_async_wait_group<1>();
          convert(sbase + K0 + ks_j * C::K_BYTES, K_LEN);
          mbar_arrive(&k_full[ks_j]);
        }
        if (more && !issue_v(ext_n)) {
          ok = false;
          break;
        }
        if (!ext_j) {
          // groups issued after V(j): K(j+1) and V(j+1) if there are
          if (more) cp_async_wait_group<2>();
          else cp_async_wait_group<0>();
          convert(sbase + C::OFF_V + vs_j * C::V_BYTES, V_LEN);
          mbar_arrive(&v_full[vs_j]);
        }
        ext_j = ext_n;
      }
    }
    }
    if (!ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
    cp_async_wait_all();
  } else if (kv_write) {
    // ------------------------------------------ fused KV write (warps 14-15)
    // The pages store the new tokens' K/V rows in the pool before attending
    // (set_kv_buffer(layer, cache_loc, k, v)).  The two-stage form reads the
    // extend keys from k_extend / v_extend, so the store can run beside the
    // attention: each unit copies the rows of its own tokens whose key
    // positions lie in its key range (split-KV units of one block cover
    // disjoint ranges, so every (token, KV head) row is written once).  A
    // slot outside the pool is skipped.
    constexpr int CK = C::LQ / 8, CV = C::HDV / 8;  // 16-byte chunks of a K / V row
    const int wt = tid - 14 * 32;                    // 0 .. 63
    bool ok = true;
    for (uint32_t uc = 0; ok && !*abort_flag; ++uc) {
      const int u = ring_unit(&bars[B_U_FULL], &bars[B_U_EMPTY], s_unit, uc, abort_flag, true, ok, p.wait_ns);
      if (u < 0) break;
      const WorkUnit w = p.units[MODE == kListed ? u : p.uorder[u]];
      const int t0 = max(w.k_begin, w.qpos0) - w.qpos0;
      const int t1 = min(w.k_end, w.qpos0 + w.n_tok) - w.qpos0;
      const int n = (t1 - t0) * (CK + CV);
      const bf16 *kx = p.k_ext + (int64_t)w.kvh * p.ke_sh;
      const bf16 *vx = p.v_ext + (int64_t)w.kvh * p.ve_sh;
      bf16 *kp = p.k_pool_w + (int64_t)w.kvh * p.kb_sh;
      bf16 *vp = p.v_pool_w + (int64_t)w.kvh * p.vb_sh;
      // four chunks in flight per thread: loads first, then the stores
      for (int c0 = wt; c0 < n; c0 += 4 * 64) {
        uint4 v[4];
        bf16 *dst[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + k * 64;
          dst[k] = nullptr;
          if (c < n) {
            const int t = t0 + c / (CK + CV), ch = c % (CK + CV);
            const int64_t row = w.q_tok0 + t;
            const int64_t slot = __ldg(p.cache_loc + row);
            if (slot >= 0 && slot < p.num_slots) {
              const bool is_k = ch < CK;
              const int e = (is_k ? ch : ch - CK) * 8;
              v[k] = __ldg(reinterpret_cast<const uint4 *>(
                  (is_k ? kx + row * p.ke_st : vx + row * p.ve_st) + e));
              dst[k] = (is_k ? kp + slot * p.kb_ss : vp + slot * p.vb_ss) + e;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (dst[k]) *reinterpret_cast<uint4 *>(dst[k]) = v[k];
      }
    }
    if (!ok) abort_cta(abort_flag, p.status, PKX_ETIMEOUT);
  }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------- launch (host)
// Whether a kernel's dynamic shared-memory limit has been raised on the
// current device (the attribute is per device; one set of flags per kernel).
inline bool needs_config(PerDevice &done) {
  std::atomic<int> *here = done.here();
  return !here || here->load(std::memory_order_acquire) == 0;
}
inline void mark_configured(PerDevice &done) {
  if (std::atomic<int> *here = done.here()) here->store(1, std::memory_order_release);
}

template <int HD, int MODE, bool MASK = false, int FMT = 0, bool FIRST = false>
static int launch_attn_kernel(const typename MapsOf<MODE>::T &tmaps, const KParams &kp, int grid,
                              cudaStream_t s) {
  using C = Cfg<HD>;
  static PerDevice configured;  // per instantiation
  if (needs_config(configured)) {
    cudaError_t e = cudaFuncSetAttribute(attn_kernel<HD, MODE, MASK, FMT, FIRST>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess)
      return set_error(PKX_ECUDA, "cudaFuncSetAttribute(attn_kernel): %s", cudaGetErrorString(e));
    mark_configured(configured);
  }
  cudaError_t e = launch_pdl(attn_kernel<HD, MODE, MASK, FMT, FIRST>, dim3(grid), dim3(C::THREADS),
                             C::SMEM, s, tmaps, kp);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "attn_kernel launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
