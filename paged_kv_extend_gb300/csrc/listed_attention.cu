// listed_attention.cu -- decode attention whose work is listed by schedulers of
// its own and done by the kernel of attn_kernel.cuh (mode kListed), with a
// combine that joins any number of partials of a row:
//
//  * shared prefixes: the sequences of a group have their first S keys in
//    common.  Softmax over a sequence's keys splits over key sets, so a group's
//    prefix is one block of query rows (its sequences' heads, 128 rows a tile,
//    two tiles a unit) against S keys, and each sequence's own keys are a block
//    of one token; the partials (o, lse) of both meet in the combine.  K and V
//    of the prefix are read once for 256 query rows instead of once for each
//    sequence, and the tensor core works on full tiles instead of on
//    Hq / Hkv rows of 128.
//  * selected pages: each (sequence, KV head) attends to pages of its own; the
//    units follow from the batch alone (equal shares of top_k pages), so no scan
//    is needed.
//
// One-token units (own keys, selected pages) of groups of at most 16 query
// heads run in rows_kernel, a warp a unit: 128 rows of the tensor core would be
// padding for them, and a unit's way through the pipeline of the tile kernel
// (claim, query load, two tiles in flight, epilogue) takes an SM some us however
// short it is: 3 with 4 heads (256 sequences of 32 own keys behind a shared prefix:
// 2048 units, 40 us), 5.8 with 17 heads and one key (1672 units, 71 us; 152 units, one
// an SM: 13 us).  Larger groups and the prefixes run in the tile kernel; for selected
// pages of larger groups a first kernel writes each list of pool slots, where
// rows_kernel's warps look their pages up themselves.
//
// Partials are fp32 (o normalised, lse in natural logs) and merged as
//   lse = log sum_i exp(lse_i),  o = sum_i exp(lse_i - lse) o_i.
// A unit's partial rows lie in granules of Hq / Hkv rows (one token's heads of
// one KV head): n_tok granules a key stream, so that a one-token unit takes one
// (rows_kernel) or two (the tile kernel's two streams) and not two whole tiles.
//
// Roundings.  Both kernels round the softmax weights P to bf16 for the product
// with V, as decode_attention_fwd does: the tensor core's bf16 form takes both
// factors in it, and V of a bf16 pool has no other 16-bit form that holds it (an
// fp8 pool's codes would fit f16, and P three more bits with them; not built).  Sums of
// P are of the fp32 values before that rounding; logits, maxima, sums, O and the
// partials are fp32.  Independent roundings of the weights (2^-9 each at most) move
// o by 0.0017 of its norm, as much as o's own rounding to bf16 does; measured
// against 64 bits (o, lse) are off by 0.0017 to 0.0022, a plain fp32 form rounded once
// by 0.0017.
#include <algorithm>
#include <climits>
#include <cstring>
#include <cuda_runtime.h>

#include "attn_kernel.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

// Position of the first of a listed unit's at most 256 query tokens: past every
// key, so that no causal mask applies.
constexpr int kPastAll = kMaxListedKeys;
static_assert(kPastAll <= INT_MAX - 256, "positions of a unit's tokens");

// Groups of at most this many query heads take one-token units to rows_kernel.
constexpr int kRowsGroup = 16;
// Keys that a one-token unit of rows_kernel is cut at, and the fewest such runs
// it holds.
constexpr int kRowRun = 64, kMinRuns = 2;
constexpr int kRowsWarps = 8;  // of a CTA, one CTA an SM

// Where a token's partials lie: granule a + kvh * a_head + i * a_step + s *
// a_stream for its prefix (i < a_n splits, s < a_streams), likewise b + kvh *
// b_head + i * b_step + s for its own keys (the launch's b_head, b_step).
struct __align__(16) ListedRow {
  int32_t a, a_n, a_head, a_step, a_streams, a_stream, b, b_n;
};

struct ListedLayout {
  size_t seq_off, grp_off, units_off, rows_off, idx_off, ptr_off, err_off, plse_off,
      po_off, total;
  int unit_max;
  int64_t gran_max;
};

// First key of piece i when n runs of `run` keys, `keys` in all, are cut into S
// pieces (sizes differ by one run).
__device__ __forceinline__ int piece_at(int i, int n, int S, int run, int keys) {
  const int q = n / S;
  return (int)min((int64_t)(i * q + min(i, n - q * S)) * run, (int64_t)keys);
}

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// ------------------------------------------------------------------ combine
// WPR warps a (token, head) row: they take its partials in turn, 32 weights in a
// warp's lanes, the row's dims split over the lanes (float4 each), four partials'
// loads in flight, and meet in shared memory.
template <int D, int WPR>
__global__ void __launch_bounds__(256, 4) listed_combine_kernel(
    const ListedRow *__restrict__ rows, const float *__restrict__ plse,
    const float *__restrict__ po, bf16 *__restrict__ o, float *__restrict__ lse, int batch, int hq,
    int group, int b_head, int b_step, int b_streams, int b_n, const int32_t *__restrict__ err,
    int n_err, int32_t *status) {
  constexpr int ROWS = 8 / WPR;  // rows of a CTA
  __shared__ float4 s_acc[WPR > 1 ? 8 : 1][32];
  __shared__ float2 s_mw[8];  // maximum and sum of weights
  grid_dep_wait();
  grid_dep_launch();
  constexpr float kLog2e = 1.4426950408889634f;
  if (err && blockIdx.x == 0)  // errors that the listing kernel's CTAs found
    for (int i = threadIdx.x; i < n_err; i += blockDim.x)
      if (err[i]) record_status(status, PKX_EDEVICE);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WPR;
  const int64_t n_rows = (int64_t)batch * hq;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < n_rows; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t r = min(r0 + warp / WPR, n_rows - 1);
    const bool own_row = r0 + warp / WPR < n_rows;
    const int t = (int)(r / hq), head = (int)(r - (int64_t)t * hq);
    const int kvh = head / group, g = head - kvh * group;
    // (without a table: b_n pieces of each of the token's KV heads in turn)
    ListedRow R{};
    if (rows) {
      R = rows[t];
    } else {
      R.b = t * (hq / group) * b_head;
      R.b_n = b_n;
    }
    const int na = R.a_n * R.a_streams, n = na + b_streams * R.b_n;
    auto row_of = [&](int i) -> int64_t {
      int64_t gr;
      if (i < na) {
        const int sp = R.a_streams == 2 ? i >> 1 : i, s = i - sp * R.a_streams;
        gr = (int64_t)R.a + (int64_t)kvh * R.a_head + (int64_t)sp * R.a_step + s * R.a_stream;
      } else {
        const int j = i - na, sp = b_streams == 2 ? j >> 1 : j;
        gr = (int64_t)R.b + (int64_t)kvh * b_head + (int64_t)sp * b_step + (j - sp * b_streams);
      }
      return gr * group + g;
    };
    // this warp's partials: part, part + WPR, ...
    const int mine = n > part ? (n - part + WPR - 1) / WPR : 0;
    // maximum of their log sums (fmaxf drops a NaN one, which comes back as a
    // NaN weight below)
    float mx = -INFINITY;
    bool any = false;
    for (int i0 = 0; i0 < mine; i0 += 32) {
      const float x = i0 + lane < mine ? plse[row_of((i0 + lane) * WPR + part)] : -INFINITY;
      any |= !(x == -INFINITY);
      mx = fmaxf(mx, x);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    any = __any_sync(0xffffffffu, any);
    float wsum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; any && i0 < mine; i0 += 32) {
      const bool have = i0 + lane < mine;
      const int64_t row = have ? row_of((i0 + lane) * WPR + part) : 0;
      const float w = have ? exp2f((plse[row] - mx) * kLog2e) : 0.f;
      wsum += w;
      const int m = min(32, mine - i0);
      for (int i = 0; i < m; i += 4) {
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t at = __shfl_sync(0xffffffffu, row, (i + u) & 31);
          if (i + u < m && lane * 4 < D)
            v[u] = *reinterpret_cast<const float4 *>(po + at * D + lane * 4);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float wi = __shfl_sync(0xffffffffu, w, (i + u) & 31);
          // (a stream without keys has weight 0 and a row of zeros)
          if (i + u < m && lane * 4 < D) {
            acc.x += wi * v[u].x;
            acc.y += wi * v[u].y;
            acc.z += wi * v[u].z;
            acc.w += wi * v[u].w;
          }
        }
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, s);
    if constexpr (WPR > 1) {
      // the warps' sums, each relative to its own maximum (one without partials,
      // or with empty ones alone, has the maximum -inf, weight 0 and zeros)
      s_acc[warp][lane] = acc;
      if (lane == 0) s_mw[warp] = make_float2(mx, wsum);
      __syncthreads();
      float all = -INFINITY, sum = 0.f;
      bool seen = false;
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        const float2 mw = s_mw[warp - part + w];
        seen |= !(mw.x == -INFINITY && mw.y == 0.f);
        all = fmaxf(all, mw.x);
      }
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        const float2 mw = s_mw[warp - part + w];
        if (mw.x == -INFINITY && mw.y == 0.f) continue;
        const float f = exp2f((mw.x - all) * kLog2e);
        const float4 x = s_acc[warp - part + w][lane];
        sum += f * mw.y;
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      mx = all;
      wsum = sum;
      any = seen;
      __syncthreads();
    }
    if (!own_row || part != 0) continue;
    bf16 *orow = o + r * D;
    const float inv = any ? 1.0f / wsum : 0.f;  // no visible key: 0 and -inf
    if (lane * 4 < D)
      *reinterpret_cast<uint2 *>(orow + lane * 4) =
          any ? make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv))
              : make_uint2(0, 0);
    if (lane == 0 && lse) lse[r] = any ? mx + logf(wsum) : -INFINITY;
  }
}

// Fields of the header's padding: first granule, units and claim counter of
// rows_kernel.
enum { kRowsGran = 0, kRowsCount = 1, kRowsNext = 2 };

// --------------------------------------------------------- one-token units
// A warp a unit: the 16 rows of mma.sync m16n8k16 are the query heads of one KV
// head (zero rows behind the group), 16 keys a step.
//  * S = Q K^T: Q's fragments stay in registers; K rows come from the warp's own
//    ring in shared memory (cp.async, 16-byte chunks in an order that spreads
//    eight rows over the banks) as ldmatrix pairs.
//  * The online softmax keeps one maximum a row, moved only when a logit passes it
//    by kRowsLag (in log2), which a vote finds; P (bf16) is S's accumulator
//    packed, already the A fragment of P V.
//  * An fp8 row's codes become bf16 (exact) on the way into the fragments.  A lane
//    holds four neighbouring codes of a key for K, so a step's 16 dims run in the
//    order (4 t, 4 t + 1 | 4 t + 2, 4 t + 3) for both factors; for V two
//    neighbouring dims of two keys, which are regrouped by bytes into the two
//    tiles of even and of odd dims.
// Nothing is shared between the warps: no barriers, no waits but cp.async's.
// What bounds it: the rows' bytes; the ring holds 192 KB an SM.  A step of 8 KB
// takes about 230 instructions, a sixth of the issue slots of the time that
// its bytes need.
constexpr float kRowsLag = 8.0f;

template <int D, int FMT>
struct RowsCfg {
  static constexpr int ROW = D * (FMT == 0 ? 2 : 1);  // bytes of a K or V row
  static constexpr int CPR = ROW / 16;                // chunks of a row
  static constexpr int STAGE = 2 * 16 * ROW;          // 16 K rows, 16 V rows
  static constexpr int STAGES = STAGE == 8192 ? 3 : STAGE == 4096 ? 6 : 8;
  static constexpr int SMEM = kRowsWarps * STAGES * STAGE;
};

struct RowsParams {
  const bf16 *q;
  const uint8_t *k, *v;
  int64_t k_ss, k_sh, v_ss, v_sh;  // bytes
  int64_t num_slots;
  const int32_t *kv_indptr, *kv_indices;
  WsHeader *hdr;
  float *plse, *po;
  int batch, hq, hkv, group;
  float scale_log2, cap_pre, cap_log2, v_scale;
  int use_cap;
  // own keys [batch + 1]: first key, and first piece of each sequence; its keys
  // below alias_len are listed by sequence alias_of
  const int32_t *own_begin, *own_first, *alias_len, *alias_of;
  // selected pages
  const int32_t *selected, *last_page_len;
  int64_t n_indices;
  int top_k, page_size, pieces;
  int32_t *err;  // [units]
  bf16 *o;       // one unit a (sequence, KV head): the outputs themselves, or null
  float *lse;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two fp8 codes (the low 16 bits) as two bf16.
template <int FMT>
__device__ __forceinline__ uint32_t fp8x2_to_bf16x2(uint32_t codes) {
  constexpr __nv_fp8_interpretation_t kind = FMT == 1 ? __NV_E4M3 : __NV_E5M2;
  const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), kind));
  const float2 f = __half22float2(h);
  return pack_bf16(f.x, f.y);
}

// The unit's keys: own keys (units are pieces of the sequences, KV heads
// innermost), or (PAGES) top_k * page_size places for keys of selected pages, of
// which an entry below 0 or a part of the last page leaves some empty.
template <int D, int FMT, bool PAGES>
__global__ void __launch_bounds__(kRowsWarps * 32, 1) rows_kernel(const RowsParams p) {
  using C = RowsCfg<D, FMT>;
  constexpr int RP = 32 / C::CPR;  // rows of one copy instruction
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_empty[kRowsWarps][C::STAGES];  // places without a key, a bit each
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::STAGE);
  // chunk c of row r in a stage: c ^ r % 8 (rows of 64 bytes: two to a line)
  auto spread = [](int r, int c) { return C::CPR == 4 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); };
  const int count = PAGES ? p.batch * p.hkv * p.pieces : p.hdr->pad[kRowsCount];
  const int gran0 = PAGES ? 0 : p.hdr->pad[kRowsGran];
  if (PAGES && blockIdx.x == 0 && threadIdx.x == 0) set_status_in_units(p.hdr, p.err, count);
  const int warps = gridDim.x * kRowsWarps;
  // the first unit by the warp's number (neighbouring units, which share a
  // sequence's slots, on different SMs); then own keys are claimed (ragged), and
  // pages, of equal sizes, taken in turn
  for (int u = warp * gridDim.x + blockIdx.x; u < count;) {
    int b, kvh, k_begin, k_end, at, n_pages = 0, last_len = 0, alias = 0, alias_at = 0;
    bool bad = false;
    const int32_t *sel = nullptr;
    if constexpr (PAGES) {
      const int pair = u / p.pieces, sp = u - pair * p.pieces;
      b = pair / p.hkv;
      kvh = pair - b * p.hkv;
      const int places = p.top_k * p.page_size, runs = (places + kRowRun - 1) / kRowRun;
      k_begin = piece_at(sp, runs, p.pieces, kRowRun, places);
      k_end = piece_at(sp + 1, runs, p.pieces, kRowRun, places);
      sel = p.selected + (int64_t)pair * p.top_k;
      at = __ldg(p.kv_indptr + b);
      n_pages = __ldg(p.kv_indptr + b + 1) - at;
      if (at < 0 || n_pages < 0 || (int64_t)at + n_pages > p.n_indices) {
        bad = true;
        n_pages = 0;
      }
      if (n_pages > 0) {
        last_len = __ldg(p.last_page_len + b);
        bad |= last_len < 0 || last_len > p.page_size;
        last_len = min(max(last_len, 0), p.page_size);
      }
    } else {
      const int x = u / p.hkv;
      kvh = u - x * p.hkv;
      b = 0;  // the last sequence whose first piece is at most x, by 32 probes at a time
      for (int span = p.batch; span > 1;) {
        const int step = (span + 31) / 32, i = lane * step;
        const bool before = i < span && (i == 0 || __ldg(p.own_first + b + i) <= x);
        const int top = 31 - __clz(__ballot_sync(0xffffffffu, before));
        b += top * step;
        span = min(step, span - top * step);
      }
      const int first = __ldg(p.own_first + b), S = __ldg(p.own_first + b + 1) - first;
      at = __ldg(p.kv_indptr + b);
      const int begin = __ldg(p.own_begin + b), keys = __ldg(p.kv_indptr + b + 1) - at - begin;
      const int runs = keys / kRowRun + (keys % kRowRun != 0);
      alias = __ldg(p.alias_len + b);
      if (alias > 0) alias_at = __ldg(p.kv_indptr + __ldg(p.alias_of + b));
      k_begin = begin + piece_at(x - first, runs, S, kRowRun, keys);
      k_end = begin + piece_at(x - first + 1, runs, S, kRowRun, keys);
    }
    const int n = k_end - k_begin, steps = (n + 15) / 16;
    const int row = lane / C::CPR, chunk = lane % C::CPR;  // of this lane's copies
    const uint8_t *kp = p.k + kvh * p.k_sh + chunk * 16, *vp = p.v + kvh * p.v_sh + chunk * 16;
    // slots of 32 keys at a time, one block ahead: `slots` of the block that the
    // copies are in, `coming` of the next; kNone: no key, kOutside: outside the pool
    constexpr int kNone = -1, kOutside = -2;
    auto fetch = [&](int block) {
      const int i = block * 32 + lane;
      if (i >= n) return kNone;
      if constexpr (PAGES) {
        const int e = (k_begin + i) / p.page_size, off = k_begin + i - e * p.page_size;
        const int s = __ldg(sel + e);
        bad |= s >= n_pages;
        if (s < 0 || s >= n_pages || (s == n_pages - 1 && off >= last_len)) return kNone;
        const int page = __ldg(p.kv_indices + at + s);
        const int64_t slot = (int64_t)page * p.page_size + off;
        // (a page is inside the pool as a whole or not at all)
        return page < 0 || slot - off + p.page_size > p.num_slots ? kOutside : (int)slot;
      } else {
        const int j = k_begin + i;
        const int s = __ldg(p.kv_indices + (j < alias ? alias_at : at) + j);
        return (uint32_t)s < (uint64_t)p.num_slots ? s : kOutside;
      }
    };
    int slots = fetch(0), coming = fetch(1);
    bad |= slots == kOutside;
    auto issue = [&](int step) {
      if (step < steps) {
        if ((step & 1) == 0 && step > 0) {
          slots = coming;
          bad |= slots == kOutside;
          coming = fetch((step >> 1) + 1);
        }
        uint32_t none = 0;
        if constexpr (PAGES) {
          none = (__ballot_sync(0xffffffffu, slots == kNone) >> ((step & 1) * 16)) & 0xFFFFu;
          if (lane == 0) s_empty[warp][step % C::STAGES] = none;
        }
        const uint32_t stage = ring + (step % C::STAGES) * C::STAGE;
        // (a step of empty places is passed over)
#pragma unroll
        for (int i = 0; i < 16 / RP && none != 0xFFFFu; ++i) {
          const int r = i * RP + row;
          const int s = __shfl_sync(0xffffffffu, slots, (step & 1) * 16 + r);
          const uint32_t at = stage + r * C::ROW + spread(r, chunk) * 16;
          const int64_t s0 = max(s, 0);
          cp_async_16(at, kp + s0 * p.k_ss, s >= 0 ? 16u : 0u);
          cp_async_16(at + 16 * C::ROW, vp + s0 * p.v_ss, s >= 0 ? 16u : 0u);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) issue(s);
    // Q's fragments: rows g and g + 8
    uint32_t qa[D / 16][4];
    {
      const uint32_t *q0 = reinterpret_cast<const uint32_t *>(
          p.q + ((int64_t)b * p.hq + (int64_t)kvh * p.group + g) * D);
      const uint32_t *q1 = q0 + 8 * (D / 2);
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const int lo = s * 8 + (FMT == 0 ? t : 2 * t), hi = s * 8 + (FMT == 0 ? t + 4 : 2 * t + 1);
        qa[s][0] = g < p.group ? __ldg(q0 + lo) : 0u;
        qa[s][1] = g + 8 < p.group ? __ldg(q1 + lo) : 0u;
        qa[s][2] = g < p.group ? __ldg(q0 + hi) : 0u;
        qa[s][3] = g + 8 < p.group ? __ldg(q1 + hi) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const int mr = lane & 7, mi = lane >> 3;  // row and matrix of this lane's ldmatrix address
    for (int step = 0; step < steps; ++step) {
      cp_async_wait_group<C::STAGES - 2>();
      __syncwarp();  // the step's rows are here, and all lanes are done with the step before
      uint32_t empty = 0;
      if constexpr (PAGES) empty = s_empty[warp][step % C::STAGES];
      issue(step + C::STAGES - 1);
      if (PAGES && empty == 0xFFFFu) continue;
      const uint32_t sk = ring + (step % C::STAGES) * C::STAGE, sv = sk + 16 * C::ROW;
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};  // keys 0-7, 8-15
      if constexpr (FMT == 0) {
        const int r = (mi >> 1) * 8 + mr;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          uint32_t b[4];
          ldmatrix4(b, sk + r * C::ROW + spread(r, 2 * s + (mi & 1)) * 16);
          mma_bf16(s0, qa[s], b[0], b[1]);
          mma_bf16(s1, qa[s], b[2], b[3]);
        }
      } else {
        const int r = (mi & 1) * 8 + mr;
#pragma unroll
        for (int s = 0; s < D / 16; s += 2) {
          uint32_t b[4];
          ldmatrix4(b, sk + r * C::ROW + spread(r, s + (mi >> 1)) * 16);
          mma_bf16(s0, qa[s], fp8x2_to_bf16x2<FMT>(b[0] & 0xFFFFu), fp8x2_to_bf16x2<FMT>(b[0] >> 16));
          mma_bf16(s1, qa[s], fp8x2_to_bf16x2<FMT>(b[1] & 0xFFFFu), fp8x2_to_bf16x2<FMT>(b[1] >> 16));
          mma_bf16(s0, qa[s + 1], fp8x2_to_bf16x2<FMT>(b[2] & 0xFFFFu),
                   fp8x2_to_bf16x2<FMT>(b[2] >> 16));
          mma_bf16(s1, qa[s + 1], fp8x2_to_bf16x2<FMT>(b[3] & 0xFFFFu),
                   fp8x2_to_bf16x2<FMT>(b[3] >> 16));
        }
      }
      // logits in log2; places without a key are -inf
      float x[8] = {s0[0], s0[1], s1[0], s1[1], s0[2], s0[3], s1[2], s1[3]};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = p.use_cap ? p.cap_log2 * tanh_approx(x[i] * p.cap_pre) : x[i] * p.scale_log2;
      if constexpr (!PAGES) {
        const int left = n - step * 16;
        if (left < 16) empty = 0xFFFFu << left;
      }
      if (empty != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((empty >> (((i >> 1) & 1) * 8 + 2 * t + (i & 1))) & 1u) x[i] = -INFINITY;
      }
      float t0 = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      float t1 = fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]));
      if (__any_sync(0xffffffffu, t0 > m0 + kRowsLag || t1 > m1 + kRowsLag)) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
        const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
        // (an old maximum of -inf goes with sums of 0)
        const float a0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - n0);
        const float a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= a0;
          o[j][1] *= a0;
          o[j][2] *= a1;
          o[j][3] *= a1;
        }
      }
      const float c0 = m0 == -INFINITY ? 0.f : m0, c1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = ex2_approx(x[i] - c0);
        x[4 + i] = ex2_approx(x[4 + i] - c1);
        l0 += x[i];
        l1 += x[4 + i];
      }
      const uint32_t pa[4] = {pack_bf16(x[0], x[1]), pack_bf16(x[4], x[5]), pack_bf16(x[2], x[3]),
                              pack_bf16(x[6], x[7])};
      const int r = (mi & 1) * 8 + mr;
      if constexpr (FMT == 0) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t b[4];
          ldmatrix4_trans(b, sv + r * C::ROW + spread(r, 2 * j + (mi >> 1)) * 16);
          mma_bf16(o[2 * j], pa, b[0], b[1]);
          mma_bf16(o[2 * j + 1], pa, b[2], b[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < D / 16; j += 2) {
          uint32_t b[4];
          ldmatrix4_trans(b, sv + r * C::ROW + spread(r, j + (mi >> 1)) * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // bytes: (key, dims 2 g and 2 g + 1), (next key, the same dims)
            const uint32_t x0 = __byte_perm(b[2 * i], 0u, 0x3120);
            const uint32_t x1 = __byte_perm(b[2 * i + 1], 0u, 0x3120);
            mma_bf16(o[2 * (j + i)], pa, fp8x2_to_bf16x2<FMT>(x0 & 0xFFFFu),
                     fp8x2_to_bf16x2<FMT>(x1 & 0xFFFFu));
            mma_bf16(o[2 * (j + i) + 1], pa, fp8x2_to_bf16x2<FMT>(x0 >> 16),
                     fp8x2_to_bf16x2<FMT>(x1 >> 16));
          }
        }
      }
    }
    __syncwarp();  // the ring is free
    // the partial: o / l and lse of rows g and g + 8
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int head = g + 8 * half;
      if (head >= p.group) continue;
      const float l = half ? l1 : l0, m = half ? m1 : m0;
      const float inv = (l == 0.f ? 0.f : 1.0f / l) * p.v_scale;
      const float lse = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
      if (PAGES && p.o) {
        const int64_t out = (int64_t)b * p.hq + (int64_t)kvh * p.group + head;
        bf16 *dst = p.o + out * D;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const float e0 = o[2 * j][2 * half] * inv, e1 = o[2 * j][2 * half + 1] * inv;
          const float f0 = o[2 * j + 1][2 * half] * inv, f1 = o[2 * j + 1][2 * half + 1] * inv;
          if constexpr (FMT == 0) {
            *reinterpret_cast<uint32_t *>(dst + 16 * j + 2 * t) = pack_bf16(e0, e1);
            *reinterpret_cast<uint32_t *>(dst + 16 * j + 8 + 2 * t) = pack_bf16(f0, f1);
          } else {
            *reinterpret_cast<uint2 *>(dst + 16 * j + 4 * t) =
                make_uint2(pack_bf16(e0, f0), pack_bf16(e1, f1));
          }
        }
        if (t == 0 && p.lse) p.lse[out] = lse;
        continue;
      }
      const int64_t out = (int64_t)(gran0 + u) * p.group + head;
      float *dst = p.po + out * D;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const float e0 = o[2 * j][2 * half] * inv, e1 = o[2 * j][2 * half + 1] * inv;
        const float f0 = o[2 * j + 1][2 * half] * inv, f1 = o[2 * j + 1][2 * half + 1] * inv;
        if constexpr (FMT == 0) {
          *reinterpret_cast<float2 *>(dst + 16 * j + 2 * t) = make_float2(e0, e1);
          *reinterpret_cast<float2 *>(dst + 16 * j + 8 + 2 * t) = make_float2(f0, f1);
        } else {  // tiles of even and of odd dims
          *reinterpret_cast<float4 *>(dst + 16 * j + 4 * t) = make_float4(e0, f0, e1, f1);
        }
      }
      if (t == 0) p.plse[out] = lse;
    }
    bad = __any_sync(0xffffffffu, bad);
    if constexpr (PAGES) {
      if (lane == 0) p.err[u] = bad;
      u += warps;
    } else {
      int next = 0;
      if (lane == 0) {
        if (bad) record_status(&p.hdr->status, PKX_EDEVICE);
        next = atomicAdd(&p.hdr->pad[kRowsNext], 1);
      }
      u = warps + __shfl_sync(0xffffffffu, next, 0);
    }
  }
  cp_async_wait_all();
}

// --------------------------------------------------------- shared prefixes
struct SharedParams {
  const int32_t *kv_indptr, *group_indptr, *shared_lens;
  int batch, num_groups, hkv;
  int tok;          // tokens of a query tile
  int sms;
  int own_run;      // keys that own keys are cut at: 1 << own_shift
  int own_shift;
  int own_least;    // fewest such runs of a unit
  int own_target;   // units of own keys wanted
  int own_gran;     // granules of one
  int rows;         // own keys go to rows_kernel
  int tile_kernel;  // the tile kernel runs
  int64_t n_indices;
  int unit_max;
  int64_t gran_max;
  int32_t *seq;     // [kSeqArrays][batch + 1]
  // [batch + 1] first own key; first piece; keys that sequence alias_of lists
  int32_t *own_begin, *own_first, *alias_len, *alias_of;
  int key_elements;  // of a key's K and V rows, all KV heads
  int row_elements;  // of a token's outputs: hq * d
  int32_t *grp;     // [kGroupArrays][num_groups + 1]
  int in_smem;      // those arrays in dynamic shared memory instead
  WorkUnit *units;
  ListedRow *rows_out;
  WsHeader *hdr;
};

// Exclusive sums over a block of 1024 threads of two values in [0, kMany] each,
// and the totals; sums are held at kMany, far above any count that the
// workspace takes (an indptr that decreases can make them larger than 32 bits).
constexpr uint32_t kMany = 1u << 30;
__device__ __forceinline__ uint32_t add_held(uint32_t a, uint32_t b) { return min(a + b, kMany); }
__device__ __forceinline__ uint32_t mul_held(uint32_t a, uint32_t b) {
  return (uint32_t)min((uint64_t)a * b, (uint64_t)kMany);
}
struct Two {
  uint32_t x, y;
};
__device__ __forceinline__ Two add_held(Two a, Two b) { return {add_held(a.x, b.x), add_held(a.y, b.y)}; }
__device__ __forceinline__ Two block_sum_before(Two v, Two *sh, Two &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Two s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two y = {__shfl_up_sync(0xffffffffu, s.x, o), __shfl_up_sync(0xffffffffu, s.y, o)};
    if (lane >= o) s = add_held(s, y);
  }
  if (lane == 31) sh[warp] = s;
  const Two up = {__shfl_up_sync(0xffffffffu, s.x, 1), __shfl_up_sync(0xffffffffu, s.y, 1)};
  __syncthreads();
  Two t = sh[lane], before = lane < warp ? t : Two{0, 0};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t = add_held(t, Two{__shfl_xor_sync(0xffffffffu, t.x, o), __shfl_xor_sync(0xffffffffu, t.y, o)});
    before = add_held(before, Two{__shfl_xor_sync(0xffffffffu, before.x, o),
                                  __shfl_xor_sync(0xffffffffu, before.y, o)});
  }
  __syncthreads();
  total = t;
  return lane == 0 ? before : add_held(before, up);
}

// One CTA of 1024 threads: the units of every group's prefix and the pieces of
// every sequence's own keys.  A group has min(shared_lens, the shortest of its
// sequences) keys in common, which its first sequence lists for all.  They are
// shared unless each sequence reads them as own keys: less than a tile of them, a
// group of one, or (kShareElements) too little to save.  A prefix is cut into
// equal pieces of at most C tiles.  The units are few and long, so C is the one of
// up to 64 candidates (the longest prefix in 1, 2, ... pieces) that takes least:
// its rounds over the SMs, a unit counting C + kUnitTiles tiles (its query load,
// pipeline fill and partials), and for each piece a partial of every row that
// goes out and comes back (256 sequences and 32768 shared keys in 4 pieces
// instead of 9: combine 15 -> 11.5 us, the tile kernel 112 -> 116.5, half the
// partials' traffic).  Own keys are cut for a given number of units.
//
// The whole call waits for this one CTA, so it is a chain of few barriers with
// no 64-bit division (a candidate in 64 bits took 2400 clocks); what a group
// or a sequence needs later stays in shared memory.
constexpr int kUnitTiles = 3;
// Elements of K and V that sharing has to save for the tile kernel to run, which
// takes 13 us with one short unit an SM and more than 20 with a few.  rows_kernel
// reads a prefix again for every sequence, from L2 where it fits.  A captured call
// from a cold cache, shared / read by each, us, one group of sequences with 64 keys
// of their own, 32 heads over 8 KV heads of 128 (16 over 16: the same within 7 us),
// by saved elements >> 20:
//                        44         66         88        110        176        352
//   bf16, 8 sequences   37 / 33    39 / 37    39 / 44    41 / 52    46 / 64    56 / 105
//   bf16, 64            43 / 29    48 / 36    43 / 39    46 / 41    48 / 56    48 / 82
//   e4m3, 8             46 / 37    48 / 39    48 / 46    48 / 56    52 / 68    64 / 111
//   e4m3, 64            51 / 31    56 / 37    52 / 44    52 / 46    54 / 64    54 / 95
//   bf16, 2             58 / 60    66 / 78    72 / 93    80 / 107  101 / 150  156 / 254
//   e4m3, 2             60 / 52    74 / 64    84 / 80    95 / 86   125 / 120  209 / 192
// The rule counts elements alone: for two sequences it is late in a bf16 pool, and
// in an fp8 pool, whose tiles are converted before the products, sharing between two
// never pays.
constexpr float kShareElements = 88 << 20;
constexpr int kSeqArrays = 3, kGroupArrays = 7;
__global__ void __launch_bounds__(1024, 1) shared_sched_kernel(const SharedParams p) {
  extern __shared__ int32_t s_dyn[];
  __shared__ Two sh[32];
  __shared__ float2 s_best[32];
  __shared__ int s_longest;
  __shared__ uint32_t s_saved;    // tiles of keys, over the sequences
  __shared__ uint32_t s_members;  // sequences in groups that share
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.batch, NG = p.num_groups, B1 = B + 1, G1 = NG + 1;
  int32_t *seq = p.in_smem ? s_dyn : p.seq, *grp = p.in_smem ? s_dyn + kSeqArrays * B1 : p.grp;
  // keys, shared keys, pieces of own keys
  int32_t *sT = seq, *sS = seq + B1, *sN = seq + 2 * B1;
  // shared keys, first sequence, blocks, granules and pieces; first unit, first granule
  int32_t *gS = grp, *gB = grp + G1, *gK = grp + 2 * G1, *gR = grp + 3 * G1, *gP = grp + 4 * G1;
  int32_t *gU = grp + 5 * G1, *gG = grp + 6 * G1;
  const int blk = 2 * p.tok;  // tokens of a prefix unit
  if (tid == 0) {
    s_longest = 0;
    s_saved = 0;
    s_members = 0;
  }
  grid_dep_wait();
  grid_dep_launch();
  // groups are consecutive runs of sequences, else nothing is shared
  bool bad = false, bad_groups = false;
  for (int g = tid; g <= NG && NG > 0; g += 1024) {
    const int lo = p.group_indptr[g], hi = g < NG ? p.group_indptr[g + 1] : lo;
    const int s = g < NG ? p.shared_lens[g] : 0;
    bad_groups |= lo < 0 || hi < lo || hi > B || s < 0;
    gB[g] = lo;
    gS[g] = s;
  }
  for (int b = tid; b < B; b += 1024) {
    const int k0 = p.kv_indptr[b], T = p.kv_indptr[b + 1] - k0;
    const bool ok = k0 >= 0 && T >= 0 && (int64_t)k0 + T <= p.n_indices;
    bad |= !ok;
    sT[b] = ok ? T : 0;
    sS[b] = 0;
    p.alias_len[b] = 0;
  }
  if (tid == 0) {
    p.hdr->status = 0;
    p.hdr->next_unit = 0;
    p.hdr->pad[kRowsNext] = 0;
  }
  const bool share = __syncthreads_or(bad_groups) == 0;
  if (bad || bad_groups) record_status(&p.hdr->status, PKX_EDEVICE);
  auto tiles = [](int keys) { return keys / kBlockN + (keys % kBlockN != 0); };
  // shared keys of each group (a warp each), its blocks of queries, and the
  // granules of one piece of all of them for one KV head (two streams of partials
  // where the block is one tile of rows)
  for (int g = warp; g < NG; g += 32) {
    int S = 0, lo = 0, hi = 0;
    if (share) {
      lo = gB[g];
      hi = gB[g + 1];
      int least = gS[g];
      for (int b = lo + lane; b < hi; b += 32) least = min(least, sT[b]);
      least = __reduce_min_sync(0xffffffffu, least);
      if (hi - lo < 2) least = 0;
      if (least >= kBlockN || !p.rows) S = least;
      for (int b = lo + lane; b < hi; b += 32) {
        sS[b] = S;
        p.alias_len[b] = least;
        p.alias_of[b] = lo;
      }
    }
    __syncwarp();
    if (lane == 0) {
      const int nb = S > 0 ? (hi - lo + blk - 1) / blk : 0, last = hi - lo - (nb - 1) * blk;
      gS[g] = S;
      gK[g] = nb;
      gR[g] = nb > 0 ? (nb - 1) * blk + (last <= p.tok ? 2 * last : last) : 0;
      if (S > 0) {
        atomicMax(&s_longest, tiles(S));
        atomicAdd(&s_saved, (uint32_t)(hi - lo - 1) * (uint32_t)tiles(S));
        atomicAdd(&s_members, (uint32_t)(hi - lo));
      }
    }
  }
  __syncthreads();
  if (p.rows &&
      (!p.tile_kernel || (float)s_saved * kBlockN * p.key_elements < kShareElements)) {  // every sequence reads its prefix
    __syncthreads();
    for (int b = tid; b < B; b += 1024) sS[b] = 0;
    for (int g = tid; g < NG; g += 1024) gS[g] = gK[g] = gR[g] = 0;
    if (tid == 0) s_longest = 0;
    __syncthreads();
  }
  // totals: tiles of the prefixes, runs of own keys
  auto runs = [&](int b) {
    const int n = sT[b] - sS[b];
    return (n >> p.own_shift) + ((n & (p.own_run - 1)) != 0);
  };
  const int bc = (B + 1023) / 1024, b0 = min(B, tid * bc), b1 = min(B, b0 + bc);
  Two sum = {0, 0}, all;
  for (int b = b0; b < b1; ++b) sum.y = add_held(sum.y, (uint32_t)runs(b));
  for (int g = tid; g < NG; g += 1024) sum.x = add_held(sum.x, mul_held(gK[g], tiles(gS[g])));
  block_sum_before(sum, sh, all);
  // pieces of R runs: about own_target of them and one more a sequence at most
  // (the quotient in fp32 is raised past its rounding)
  const float own_each = (float)all.y * (float)p.hkv / (float)p.own_target * 1.000001f;
  const int R = max((int)ceilf(min(own_each, 1e9f)), p.own_least);
  Two units = {0, 0};  // of own keys
  for (int b = b0; b < b1; ++b) {
    sN[b] = (runs(b) + R - 1) / R;
    units.x = add_held(units.x, (uint32_t)sN[b]);
  }
  Two own_all, pre = {0, 0};  // pre: prefix units, their granules
  const Two own_before = block_sum_before(units, sh, own_all);
  if (s_longest > 0) {
    // at most four units an SM and one more a block
    const float each = (float)all.x * (float)p.hkv / (4.0f * p.sms) * 1.000001f;
    const int least = max((int)ceilf(min(each, 1e9f)), kMinSplitTiles);
    // (estimates, in fp32: any C of at least `least` does; a piece's partials in
    // the 1.7 us that a tile takes, at 4 TB/s)
    const float piece_cost = (float)s_members * (float)p.row_elements * (1.0f / 832000.0f);
    const float per_sm = (float)p.hkv / (float)p.sms;
    float2 best = make_float2(INFINITY, 0.f);  // (tiles, C)
    for (int j = warp + 1; j <= 64; j += 32) {
      const float c = fmaxf(ceilf((float)s_longest / (float)j), (float)least), inv = 1.0f / c;
      float n = 0.f;
      for (int g = lane; g < NG; g += 32) n += (float)gK[g] * ceilf((float)tiles(gS[g]) * inv);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      const float t = ceilf(n * per_sm) * (c + kUnitTiles) + ceilf((float)s_longest * inv) * piece_cost;
      if (t < best.x) best = make_float2(t, c);
    }
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
    best = s_best[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float2 x = {__shfl_xor_sync(0xffffffffu, best.x, o), __shfl_xor_sync(0xffffffffu, best.y, o)};
      if (x.x < best.x || (x.x == best.x && x.y < best.y)) best = x;
    }
    const int C = max((int)best.y, least);
    // first unit and granule of each group
    const int gc = (NG + 1023) / 1024, g0 = min(NG, tid * gc), g1 = min(NG, g0 + gc);
    auto size = [&](int g) {  // units and granules
      return Two{mul_held(mul_held(gP[g], gK[g]), p.hkv), mul_held(mul_held(gP[g], gR[g]), p.hkv)};
    };
    Two n = {0, 0};
    for (int g = g0; g < g1; ++g) {
      gP[g] = (tiles(gS[g]) + C - 1) / C;
      n = add_held(n, size(g));
    }
    n = block_sum_before(n, sh, pre);
    for (int g = g0; g < g1; ++g) {
      gU[g] = (int)n.x;
      gG[g] = (int)n.y;
      n = add_held(n, size(g));
    }
  }
  const int64_t own_units = (int64_t)own_all.x * p.hkv;
  // (false only for an indptr that decreases: the workspace is sized for the
  // largest counts)
  const bool fits = pre.x + own_units <= p.unit_max &&
                    pre.y + p.own_gran * own_units <= p.gran_max;
  if (!fits) {
    if (tid == 0) {
      record_status(&p.hdr->status, PKX_EDEVICE);
      p.hdr->n_units = 0;
      p.hdr->pad[kRowsCount] = 0;
    }
    for (int b = tid; b < B; b += 1024) p.rows_out[b] = ListedRow{};
    return;
  }
  const int pre_units = (int)pre.x, pre_gran = (int)pre.y;
  __syncthreads();  // the groups' first units and granules
  int first_piece = (int)own_before.x;
  for (int b = b0; b < b1; ++b) {
    p.own_first[b] = first_piece;
    p.own_begin[b] = sS[b];
    // where the token's partials lie
    ListedRow r{};
    r.b = pre_gran + p.own_gran * first_piece * p.hkv;
    r.b_n = sN[b];
    first_piece += sN[b];
    if (sS[b] > 0) {
      int lo = 0, hi = NG - 1;  // last g with gB[g] <= b
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (gB[mid] <= b) lo = mid;
        else hi = mid - 1;
      }
      const int g = lo, i = b - gB[g], k = i / blk;
      const int n_tok = min(blk, gB[g + 1] - gB[g] - k * blk);
      r.a = gG[g] + i;
      r.a_n = gP[g];
      r.a_head = gR[g];
      r.a_step = p.hkv * gR[g];
      r.a_streams = n_tok <= p.tok ? 2 : 1;
      r.a_stream = n_tok;
    }
    p.rows_out[b] = r;
  }
  if (tid == 0) {
    p.own_first[B] = (int)own_all.x;
    p.hdr->n_units = (int)(p.rows ? pre_units : pre_units + own_units);
    p.hdr->pad[kRowsGran] = pre_gran;
    p.hdr->pad[kRowsCount] = (int)(p.rows ? own_units : 0);
  }
  // units of the prefixes: group, piece, KV head, block (blocks of one piece
  // and head next to each other: they read the same keys)
  for (int u = tid; u < pre_units; u += 1024) {
    int lo = 0, hi = NG - 1;  // last g with gU[g] <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (gU[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    const int g = lo, nb = gK[g], nt = tiles(gS[g]), S = gP[g];
    const int r = u - gU[g], r2 = r / nb, k = r - r2 * nb, sp = r2 / p.hkv, kvh = r2 - sp * p.hkv;
    const int first = gB[g], n = gB[g + 1] - first;
    WorkUnit w;
    w.q_tok0 = first + k * blk;
    w.n_tok = min(blk, n - k * blk);
    w.qpos0 = kPastAll;
    w.kvh = kvh;
    w.k_begin = piece_at(sp, nt, S, kBlockN, gS[g]);
    w.k_end = piece_at(sp + 1, nt, S, kBlockN, gS[g]);
    w.k_split = INT_MAX;
    w.n_tiles = tiles(w.k_end - w.k_begin);
    w.b = first;
    w.slot = gG[g] + (sp * p.hkv + kvh) * gR[g] + k * blk;
    w.dq = w.claim = 0;
    p.units[u] = w;
  }
  __syncthreads();  // (own_first, for the units below)
  if (p.rows) return;  // (rows_kernel finds its units itself)
  // units of the sequences' own keys: sequence, piece, KV head
  for (int i = tid; i < (int)own_units; i += 1024) {
    const int x = i / p.hkv, kvh = i - x * p.hkv;
    int lo = 0, hi = B - 1;  // last b with own_first[b] <= x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.own_first[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo, nr = runs(b), S = sN[b], sp = x - p.own_first[b];
    WorkUnit w;
    w.q_tok0 = b;
    w.n_tok = 1;
    w.qpos0 = kPastAll;
    w.kvh = kvh;
    w.k_begin = sS[b] + piece_at(sp, nr, S, p.own_run, sT[b] - sS[b]);
    w.k_end = sS[b] + piece_at(sp + 1, nr, S, p.own_run, sT[b] - sS[b]);
    w.k_split = INT_MAX;
    w.n_tiles = tiles(w.k_end - w.k_begin);
    w.b = b;
    w.slot = pre_gran + p.own_gran * i;
    w.dq = w.claim = 0;
    p.units[pre_units + i] = w;
  }
}

// Units of own keys wanted, the keys they are cut at, the fewest of those runs,
// and granules of a unit: three for each warp of rows_kernel, or three tile
// units an SM.
struct OwnUnits {
  int target, run, least, gran;
};
static OwnUnits own_units(int group, int num_sms) {
  const int n = num_sms > 0 ? num_sms : 160;
  return group <= kRowsGroup ? OwnUnits{3 * kRowsWarps * n, kRowRun, kMinRuns, 1}
                             : OwnUnits{3 * n, kBlockN, kMinSplitTiles, 2};
}

static ListedLayout shared_layout(int batch, int num_groups, int hkv, int group, int d,
                                  int num_sms) {
  ListedLayout L{};
  const int tok = tokens_per_block(group), blk = 2 * tok;
  const int n = num_sms > 0 ? num_sms : 160;
  const OwnUnits own = own_units(group, num_sms);
  // blocks: at most one partly filled a group (of two sequences or more)
  const int64_t blocks = batch / blk + std::min(num_groups, batch / 2);
  const int64_t units = 4ll * n + own.target + (int64_t)hkv * (blocks + batch);
  L.unit_max = (int)std::min<int64_t>(units, INT_MAX / 4);
  // four prefix units an SM of blk granules, or twice the batch's tokens, and,
  // a block's first piece, twice its tokens; the units of own keys
  const int64_t prefix = num_groups > 0 ? 4ll * n * std::min<int64_t>(blk, 2ll * batch) +
                                              2ll * hkv * batch
                                        : 0;
  L.gran_max = prefix + own.gran * (own.target + (int64_t)hkv * batch);
  size_t off = up256(sizeof(WsHeader));
  L.seq_off = off;
  off = up256(off + sizeof(int32_t) * (kSeqArrays + 4) * (size_t)(batch + 1));
  L.grp_off = off;
  off = up256(off + sizeof(int32_t) * kGroupArrays * (size_t)(num_groups + 1));
  L.units_off = off;
  off = up256(off + sizeof(WorkUnit) * (size_t)L.unit_max);
  L.rows_off = off;
  off = up256(off + sizeof(ListedRow) * (size_t)batch);
  L.plse_off = off;
  off = up256(off + sizeof(float) * (size_t)L.gran_max * group);
  L.po_off = off;
  off = up256(off + sizeof(float) * (size_t)L.gran_max * group * d);
  L.total = off;
  return L;
}

size_t shared_decode_workspace(int batch, int num_groups, int hq, int hkv, int d, int num_sms) {
  return shared_layout(batch, num_groups, hkv, hq / hkv, d, num_sms).total;
}

// ------------------------------------------------------------ selected pages
struct PagesParams {
  const int32_t *kv_indptr, *kv_indices, *last_page_len, *selected;
  int64_t n_indices, num_slots;
  int batch, hkv, page_size, top_k;
  int pieces;      // units of a (sequence, KV head)
  int run;         // keys they are cut at
  int gran;        // granules of one
  int cap;         // keys of its list: top_k * page_size
  int32_t *slots;  // [batch * hkv][cap]
  int32_t *ptr;    // [batch * hkv] first key of each list
  int32_t *err;    // [batch * hkv]
  WorkUnit *units;
  ListedRow *rows_out;
  WsHeader *hdr;
};

// One CTA for each (sequence, KV head): the pool slots of its selected pages
// one after another, and its units (equal shares of the list).
__global__ void __launch_bounds__(256) list_pages_kernel(const PagesParams p) {
  extern __shared__ int s_first[];  // [top_k + 1] first key of each entry
  int *s_slot = s_first + p.top_k + 1;  // [top_k] its first pool slot, or -1
  __shared__ int s_warp[8];
  __shared__ int s_run, s_bad;
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = blockIdx.x, b = pair / p.hkv, kvh = pair - b * p.hkv;
  const int at = p.kv_indptr[b];
  int n = p.kv_indptr[b + 1] - at;
  bool bad = at < 0 || n < 0 || (int64_t)at + n > p.n_indices;
  if (bad) n = 0;
  const int last = n > 0 ? p.last_page_len[b] : 0;
  bad |= n > 0 && (last < 0 || last > p.page_size);
  const int32_t *sel = p.selected + (int64_t)pair * p.top_k;
  if (tid == 0) {
    s_run = 0;
    s_bad = 0;
  }
  __syncthreads();
  // first key of each entry (a running sum of the entries' lengths) and its
  // page's first slot
  const int64_t pages = p.num_slots / p.page_size;
  for (int e0 = 0; e0 < p.top_k; e0 += 256) {
    const int e = e0 + tid;
    int len = 0;
    if (e < p.top_k) {
      const int s = sel[e];
      bad |= s >= n;
      int slot = -1;
      if (s >= 0 && s < n) {
        const int page = __ldg(p.kv_indices + at + s);
        if (page >= 0 && page < pages) slot = page * p.page_size;
        len = s == n - 1 ? min(max(last, 0), p.page_size) : p.page_size;
      }
      s_slot[e] = slot;
    }
    int x = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int before = s_run;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    if (e < p.top_k) s_first[e] = before + x - len;
    __syncthreads();
    if (tid == 255) s_run = before + x;
    __syncthreads();
  }
  const int keys = s_run;
  if (tid == 0) s_first[p.top_k] = keys;
  if (bad) s_bad = 1;
  __syncthreads();
  if (tid == 0) {
    p.ptr[pair] = pair * p.cap;
    p.err[pair] = s_bad;
    if (pair == 0) {
      p.hdr->status = 0;
      p.hdr->next_unit = 0;
      p.hdr->n_units = gridDim.x * p.pieces;
    }
    if (kvh == 0) {
      ListedRow R{};
      R.b = pair * p.pieces * p.gran;
      R.b_n = p.pieces;
      p.rows_out[b] = R;
    }
  }
  const int nt = (keys + p.run - 1) / p.run;
  for (int s = tid; s < p.pieces; s += 256) {
    const int u = pair * p.pieces + s;
    WorkUnit w;
    w.q_tok0 = b;
    w.n_tok = 1;
    w.qpos0 = kPastAll;
    w.kvh = kvh;
    w.k_begin = piece_at(s, nt, p.pieces, p.run, keys);
    w.k_end = piece_at(s + 1, nt, p.pieces, p.run, keys);
    w.k_split = INT_MAX;
    w.n_tiles = (w.k_end - w.k_begin + kBlockN - 1) / kBlockN;
    w.b = pair;
    w.slot = p.gran * u;
    w.dq = w.claim = 0;
    p.units[u] = w;
  }
  // the slots, a warp an entry; a page outside the pool is listed as -1, which
  // the attention kernel reads as a zero row and reports
  int32_t *out = p.slots + (int64_t)pair * p.cap;
  for (int e = warp; e < p.top_k; e += 8) {
    const int first = s_first[e], len = s_first[e + 1] - first, slot = s_slot[e];
    for (int i = lane; i < len; i += 32) out[first + i] = slot < 0 ? -1 : slot + i;
  }
}

// Units of a (sequence, KV head): as many as own_units() wants, of at least its
// fewest runs.
static int pages_pieces(int batch, int hkv, int group, int page_size, int top_k, int num_sms) {
  const OwnUnits own = own_units(group, num_sms);
  const int64_t nr = ((int64_t)top_k * page_size + own.run - 1) / own.run;
  const int64_t pairs = std::max<int64_t>((int64_t)batch * hkv, 1);
  const int64_t want = (own.target + pairs - 1) / pairs;
  return (int)std::max<int64_t>(1, std::min(want, nr / own.least));
}

static ListedLayout pages_layout(int batch, int hkv, int group, int d, int page_size, int top_k,
                                 int num_sms) {
  ListedLayout L{};
  const bool rows = group <= kRowsGroup;  // (no units and no lists)
  const int64_t pairs = (int64_t)batch * hkv;
  const int64_t units = pairs * pages_pieces(batch, hkv, group, page_size, top_k, num_sms);
  L.unit_max = (int)std::min<int64_t>(units, INT_MAX / 4);
  L.gran_max = own_units(group, num_sms).gran * units;
  size_t off = up256(sizeof(WsHeader));
  L.err_off = off;
  off = up256(off + sizeof(int32_t) * (size_t)(rows ? units : pairs));
  if (!rows) {
    L.units_off = off;
    off = up256(off + sizeof(WorkUnit) * (size_t)units);
    L.rows_off = off;
    off = up256(off + sizeof(ListedRow) * (size_t)batch);
    L.ptr_off = off;
    off = up256(off + sizeof(int32_t) * (size_t)pairs);
    L.idx_off = off;
    off = up256(off + sizeof(int32_t) * (size_t)pairs * top_k * page_size);
  }
  L.plse_off = off;
  off = up256(off + sizeof(float) * (size_t)L.gran_max * group);
  L.po_off = off;
  off = up256(off + sizeof(float) * (size_t)L.gran_max * group * d);
  L.total = off;
  return L;
}

size_t pages_decode_workspace(int batch, int hq, int hkv, int d, int page_size, int top_k,
                              int num_sms) {
  return pages_layout(batch, hkv, hq / hkv, d, page_size, top_k, num_sms).total;
}

// -------------------------------------------------------------------- host
static int check_workspace(const ListedArgs &a, const ListedLayout &L) {
  if (!a.workspace || a.workspace_bytes < L.total)
    return set_error(PKX_EWORKSPACE, "workspace of %zu bytes given, %zu needed",
                     a.workspace_bytes, L.total);
  if (reinterpret_cast<uintptr_t>(a.workspace) & 255)
    return set_error(PKX_EINVAL, "workspace must be 256-byte aligned");
  return PKX_OK;
}

template <int D>
static int launch_listed(int fmt, const ListedMaps &tm, const KParams &kp, int grid,
                         cudaStream_t s) {
  if (fmt == kKvFp8E4M3) return launch_attn_kernel<D, kListed, false, 1>(tm, kp, grid, s);
  if (fmt == kKvFp8E5M2) return launch_attn_kernel<D, kListed, false, 2>(tm, kp, grid, s);
  return launch_attn_kernel<D, kListed>(tm, kp, grid, s);
}

template <int D, int FMT, bool PAGES>
static int launch_rows_as(const RowsParams &p, int nsm, cudaStream_t s) {
  static PerDevice configured;
  if (needs_config(configured)) {
    cudaError_t e = cudaFuncSetAttribute(rows_kernel<D, FMT, PAGES>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         RowsCfg<D, FMT>::SMEM);
    if (e != cudaSuccess)
      return set_error(PKX_ECUDA, "cudaFuncSetAttribute(rows_kernel): %s", cudaGetErrorString(e));
    mark_configured(configured);
  }
  cudaError_t e = launch_pdl(rows_kernel<D, FMT, PAGES>, dim3(nsm), dim3(kRowsWarps * 32),
                             RowsCfg<D, FMT>::SMEM, s, p);
  if (e != cudaSuccess) return set_error(PKX_ECUDA, "rows_kernel launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

// pieces > 0: selected pages, so many units a (sequence, KV head); 0: own keys.
template <int D>
static int launch_rows(const ListedArgs &a, const KParams &kp, const ListedLayout &L, int nsm,
                       int pieces) {
  const int size = a.kv_fmt == kKvBf16 ? 2 : 1;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  RowsParams p{};
  p.q = kp.q;
  p.k = static_cast<const uint8_t *>(a.k_buf);
  p.v = static_cast<const uint8_t *>(a.v_buf);
  p.k_ss = a.kb_ss * size;
  p.k_sh = a.kb_sh * size;
  p.v_ss = a.vb_ss * size;
  p.v_sh = a.vb_sh * size;
  p.num_slots = a.num_slots;
  p.kv_indptr = a.kv_indptr;
  p.kv_indices = a.kv_indices;
  p.hdr = reinterpret_cast<WsHeader *>(ws);
  p.plse = kp.plse;
  p.po = kp.po;
  p.batch = a.batch;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = kp.group;
  const bool fp8 = a.kv_fmt != kKvBf16;
  p.use_cap = kp.use_cap;
  p.scale_log2 = fp8 ? kp.scale_log2_k : kp.scale_log2;
  p.cap_pre = fp8 ? kp.cap_pre_k : kp.cap_pre;
  p.cap_log2 = kp.cap_log2;
  p.v_scale = fp8 ? a.v_scale : 1.0f;
  if (pieces > 0) {
    p.selected = a.selected;
    p.last_page_len = a.last_page_len;
    p.n_indices = a.n_indices;
    p.top_k = a.top_k;
    p.page_size = a.page_size;
    p.pieces = pieces;
    p.err = reinterpret_cast<int32_t *>(ws + L.err_off);
    p.o = pieces == 1 ? kp.o : nullptr;
    p.lse = a.lse;
    if (a.kv_fmt == kKvFp8E4M3) return launch_rows_as<D, 1, true>(p, nsm, a.stream);
    if (a.kv_fmt == kKvFp8E5M2) return launch_rows_as<D, 2, true>(p, nsm, a.stream);
    return launch_rows_as<D, 0, true>(p, nsm, a.stream);
  }
  p.own_begin = reinterpret_cast<int32_t *>(ws + L.seq_off) + kSeqArrays * (size_t)(a.batch + 1);
  p.own_first = p.own_begin + (a.batch + 1);
  p.alias_len = p.own_first + (a.batch + 1);
  p.alias_of = p.alias_len + (a.batch + 1);
  if (a.kv_fmt == kKvFp8E4M3) return launch_rows_as<D, 1, false>(p, nsm, a.stream);
  if (a.kv_fmt == kKvFp8E5M2) return launch_rows_as<D, 2, false>(p, nsm, a.stream);
  return launch_rows_as<D, 0, false>(p, nsm, a.stream);
}

// How the combine finds the partials of one-token units.
struct OwnPartials {
  const ListedRow *rows;  // or null: `pieces` a KV head, in order
  int head, step, pieces;
  const int32_t *err;  // errors of the listing kernel's CTAs (nullable)
  int n_err;
};

// One warp a row where the rows fill the GPU (32 warps an SM), else up to eight.
template <int D>
static int launch_combine(const ListedArgs &a, const KParams &kp, const OwnPartials &own, int nsm) {
  const int64_t rows = (int64_t)a.batch * a.hq, full = (int64_t)nsm * 32;
  const int wpr = rows * 8 <= full ? 8 : rows * 4 <= full ? 4 : rows * 2 <= full ? 2 : 1;
  auto kernel = wpr == 8   ? listed_combine_kernel<D, 8>
                : wpr == 4 ? listed_combine_kernel<D, 4>
                : wpr == 2 ? listed_combine_kernel<D, 2>
                           : listed_combine_kernel<D, 1>;
  const int64_t ctas = (rows * wpr + 7) / 8;
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, (int64_t)nsm * 8);
  WsHeader *hdr = static_cast<WsHeader *>(a.workspace);
  cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(256), 0, a.stream, own.rows,
                             (const float *)kp.plse, (const float *)kp.po, kp.o, a.lse, a.batch,
                             a.hq, kp.group, own.head, own.step, kp.group <= kRowsGroup ? 1 : 2,
                             own.pieces, own.err, own.n_err, &hdr->status);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "listed_combine launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

// The attention kernels and the combine: the tile kernel over the units in the
// workspace where there may be some, rows_kernel for groups of at most
// kRowsGroup heads.
static int run_listed(const ListedArgs &a, const ListedMaps *tm, const ListedLayout &L, int nsm,
                      const int32_t *kv_indptr, const int32_t *kv_indices, int pieces,
                      const OwnPartials &own) {
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  WsHeader *hdr = reinterpret_cast<WsHeader *>(ws);
  const int group = a.hq / a.hkv;
  KParams kp;
  memset(&kp, 0, sizeof kp);
  kp.q = static_cast<const bf16 *>(a.q);
  kp.o = static_cast<bf16 *>(a.o);
  kp.lse = a.lse;
  kp.k_pool = kp.k_ext = static_cast<const bf16 *>(a.k_buf);
  kp.v_pool = kp.v_ext = static_cast<const bf16 *>(a.v_buf);
  kp.kb_ss = a.kb_ss;
  kp.vb_ss = a.vb_ss;
  kp.kb_sh = a.kb_sh;
  kp.vb_sh = a.vb_sh;
  kp.num_slots = a.num_slots;
  kp.kv_indptr = kv_indptr;
  kp.kv_indices = kv_indices;
  kp.hq = a.hq;
  kp.group = group;
  kp.tok = kp.q_box_tok = tokens_per_block(group);
  kp.window = -1;
  kp.rows_per_slot = group;
  const float log2e = 1.4426950408889634f;
  const float sm_scale = a.sm_scale > 0.f ? a.sm_scale : 1.0f / sqrtf((float)a.d);
  kp.use_cap = a.logit_cap > 0.f;
  kp.scale_log2 = sm_scale * log2e;
  kp.cap_pre = kp.use_cap ? sm_scale / a.logit_cap : 0.f;
  kp.cap_log2 = kp.use_cap ? a.logit_cap * log2e : 0.f;
  kp.scale_log2_k = kp.scale_log2 * a.k_scale;
  kp.cap_pre_k = kp.cap_pre * a.k_scale;
  kp.log2_v_scale = log2f(a.v_scale);
  kp.v_scale = a.v_scale;
  kp.inv_v_scale = 1.0f / a.v_scale;
  kp.units = reinterpret_cast<WorkUnit *>(ws + L.units_off);
  kp.next_unit = &hdr->next_unit;
  kp.hdr = hdr;
  kp.status = &hdr->status;
  kp.plse = reinterpret_cast<float *>(ws + L.plse_off);
  kp.po = reinterpret_cast<float *>(ws + L.po_off);
  wait_settings(&kp.wait_ns, &kp.stall);
  cudaEvent_t ev_before = nullptr, ev_after = nullptr;
  attention_events(&ev_before, &ev_after);
  if (ev_before) cudaEventRecord(ev_before, a.stream);
  int rc = PKX_OK;
  if (tm)
    rc = a.d == 128 ? launch_listed<128>(a.kv_fmt, *tm, kp, nsm, a.stream)
                    : launch_listed<64>(a.kv_fmt, *tm, kp, nsm, a.stream);
  if (rc != PKX_OK) return rc;
  if (group <= kRowsGroup) {
    rc = a.d == 128 ? launch_rows<128>(a, kp, L, nsm, pieces) : launch_rows<64>(a, kp, L, nsm, pieces);
    if (rc != PKX_OK) return rc;
  }
  if (ev_after) cudaEventRecord(ev_after, a.stream);
  if (own.pieces == 1) return PKX_OK;  // rows_kernel has written the outputs
  return a.d == 128 ? launch_combine<128>(a, kp, own, nsm) : launch_combine<64>(a, kp, own, nsm);
}

static int make_maps(ListedMaps &tm, const ListedArgs &a) {
  const int group = a.hq / a.hkv;
  memset(&tm, 0, sizeof tm);
  const int rc = make_q_map(&tm.q, a.q, a.batch, a.hq, a.d, group, tokens_per_block(group));
  return rc != PKX_OK ? rc : make_q_map(&tm.one, a.q, a.batch, a.hq, a.d, group, 1);
}

int launch_decode_shared(const ListedArgs &a) {
  const int nsm = num_sms_current_device();
  if (nsm <= 0) return set_error(PKX_ECUDA, "cannot query the current device");
  const int group = a.hq / a.hkv;
  const ListedLayout L = shared_layout(a.batch, a.num_groups, a.hkv, group, a.d, nsm);
  int rc = check_workspace(a, L);
  if (rc != PKX_OK) return rc;
  if (L.unit_max >= INT_MAX / 4 || L.gran_max >= INT_MAX)
    return set_error(PKX_EUNSUPPORTED, "decode_shared: batch too large");
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  SharedParams p;
  p.kv_indptr = a.kv_indptr;
  p.group_indptr = a.group_indptr;
  p.shared_lens = a.shared_lens;
  p.batch = a.batch;
  p.num_groups = a.num_groups;
  p.hkv = a.hkv;
  p.tok = tokens_per_block(group);
  p.sms = nsm;
  const OwnUnits own = own_units(group, nsm);
  p.own_run = own.run;
  p.own_shift = own.run == kRowRun ? 6 : 7;
  static_assert(kRowRun == 64 && kBlockN == 128, "own_shift");
  p.own_least = own.least;
  p.own_target = own.target;
  p.own_gran = own.gran;
  p.rows = group <= kRowsGroup;
  // (the lists hold every prefix once a sequence: no more than all of them can be
  // saved)
  p.tile_kernel = !p.rows || (a.num_groups > 0 && (float)a.n_indices * 2 * a.d * a.hkv >=
                                                      kShareElements);
  p.n_indices = a.n_indices;
  p.unit_max = L.unit_max;
  p.gran_max = L.gran_max;
  p.seq = reinterpret_cast<int32_t *>(ws + L.seq_off);
  p.own_begin = p.seq + kSeqArrays * (size_t)(a.batch + 1);
  p.own_first = p.own_begin + (a.batch + 1);
  p.alias_len = p.own_first + (a.batch + 1);
  p.alias_of = p.alias_len + (a.batch + 1);
  p.key_elements = 2 * a.d * a.hkv;
  p.row_elements = a.d * a.hq;
  p.grp = reinterpret_cast<int32_t *>(ws + L.grp_off);
  ListedMaps tm;
  if (p.tile_kernel && (rc = make_maps(tm, a)) != PKX_OK) return rc;
  size_t smem = sizeof(int32_t) * (kSeqArrays * (size_t)(a.batch + 1) +
                                   kGroupArrays * (size_t)(a.num_groups + 1));
  p.in_smem = smem <= 40 * 1024;
  if (!p.in_smem) smem = 0;
  p.units = reinterpret_cast<WorkUnit *>(ws + L.units_off);
  p.rows_out = reinterpret_cast<ListedRow *>(ws + L.rows_off);
  p.hdr = reinterpret_cast<WsHeader *>(ws);
  cudaError_t e = launch_pdl(shared_sched_kernel, dim3(1), dim3(1024), smem, a.stream, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "shared_sched launch: %s", cudaGetErrorString(e));
  return run_listed(a, p.tile_kernel ? &tm : nullptr, L, nsm, a.kv_indptr, a.kv_indices, 0,
                    OwnPartials{p.rows_out, own.gran, own.gran * a.hkv, 0, nullptr, 0});
}

int launch_decode_pages(const ListedArgs &a) {
  const int group = a.hq / a.hkv;
  const int64_t pairs = (int64_t)a.batch * a.hkv;
  if (pairs * a.top_k * a.page_size > kMaxListedKeys)  // (units and granules are fewer)
    return set_error(PKX_EUNSUPPORTED,
                     "decode_pages: batch * hkv * top_k * page_size must be below 2^31 - 4096");
  const int nsm = num_sms_current_device();
  if (nsm <= 0) return set_error(PKX_ECUDA, "cannot query the current device");
  const ListedLayout L = pages_layout(a.batch, a.hkv, group, a.d, a.page_size, a.top_k, nsm);
  int rc = check_workspace(a, L);
  if (rc != PKX_OK) return rc;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  const OwnUnits own = own_units(group, nsm);
  const int pieces = pages_pieces(a.batch, a.hkv, group, a.page_size, a.top_k, nsm);
  int32_t *err = reinterpret_cast<int32_t *>(ws + L.err_off);
  if (group <= kRowsGroup)
    return run_listed(a, nullptr, L, nsm, nullptr, nullptr, pieces,
                      OwnPartials{nullptr, pieces, 1, pieces, nullptr, 0});
  ListedMaps tm;
  if ((rc = make_maps(tm, a)) != PKX_OK) return rc;
  PagesParams p;
  p.kv_indptr = a.kv_indptr;
  p.kv_indices = a.kv_indices;
  p.last_page_len = a.last_page_len;
  p.selected = a.selected;
  p.n_indices = a.n_indices;
  p.num_slots = a.num_slots;
  p.batch = a.batch;
  p.hkv = a.hkv;
  p.page_size = a.page_size;
  p.top_k = a.top_k;
  p.pieces = pieces;
  p.run = own.run;
  p.gran = own.gran;
  p.cap = a.top_k * a.page_size;
  p.slots = reinterpret_cast<int32_t *>(ws + L.idx_off);
  p.ptr = reinterpret_cast<int32_t *>(ws + L.ptr_off);
  p.err = err;
  p.units = reinterpret_cast<WorkUnit *>(ws + L.units_off);
  p.rows_out = reinterpret_cast<ListedRow *>(ws + L.rows_off);
  p.hdr = reinterpret_cast<WsHeader *>(ws);
  const size_t smem = sizeof(int) * (2 * (size_t)a.top_k + 1);
  cudaError_t e = launch_pdl(list_pages_kernel, dim3((unsigned)pairs), dim3(256), smem, a.stream, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "list_pages launch: %s", cudaGetErrorString(e));
  return run_listed(a, &tm, L, nsm, p.ptr, p.slots, 0,
                    OwnPartials{p.rows_out, own.gran * pieces, own.gran, 0, err, (int)pairs});
}

}  // namespace pkx
