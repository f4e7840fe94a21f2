// page_select.cu -- which pages of a paged KV cache a decode step reads: the
// bounds of every page's keys, and the selection by them.
//
// Bounds.  For page P and KV head h, per dim d: lo = min and hi = max of
// k[d] over the page's keys.  They are elements of K, so bf16 holds them
// exactly (an fp8 pool's codes too; its k_scale, a positive factor of every
// score, is left out).
//
// Score.  max over the box of <q, k> is sum_d max(q_d lo_d, q_d hi_d) =
// sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d, an upper bound of the logit of
// every key in the page.  Summed over the query heads of a KV head the q factors
// add up first:
//   score = sum_d qn_d lo_d + sum_d qp_d hi_d,  qp = sum_g max(q_g, 0), ...
// so that a page costs one product a bound whatever the group.  The order of the
// sums is part of the definition (each product and sum rounded to fp32, dims
// added pairwise: 0 + 1, 2 + 3, then those), so that the selection does not
// depend on how the work is split: a lane adds its 8 dims as a tree, and a
// butterfly over the lanes goes on with it.
//
// What bounds it: the bounds are read once, 4 d bytes a page and KV head (1/64
// of K and V at pages of 64 bf16 keys).  The scores are ordered 32-bit keys; the
// threshold of the top k is found by halving the key range two bits a round with
// counts over the CTA (a histogram by shared atomics would serialise: the scores
// share their exponents), and the pages are written in order, so equal scores go
// to the lower page and no atomic decides.  Where the (sequence, KV head) pairs
// fill the GPU one kernel does all of it for a pair; a few long sequences are
// scored by runs of pages first.
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

// ------------------------------------------------------------------ bounds
constexpr int kBoundThreads = 256;
constexpr int kBoundUnroll = 8;

struct BoundParams {
  const uint8_t *k;
  int64_t kb_ss, kb_hs;  // bytes
  const int32_t *page_ids, *page_lens;
  int64_t num_pages;
  int page_size, hkv, d;
  int slices;  // runs of 32 chunks of a slot's row (all heads)
  uint4 *bounds;  // [num_pages][hkv][2][d / 8]
};

template <int FMT>
__device__ __forceinline__ uint4 load_keys(const uint8_t *p) {
  if constexpr (FMT == 0) return __ldg(reinterpret_cast<const uint4 *>(p));
  else return fp8x8_to_bf16x8<FMT>(__ldg(reinterpret_cast<const uint2 *>(p)));
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // NaN if either is
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                       *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                       *reinterpret_cast<const __nv_bfloat162 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint4 min8(uint4 a, uint4 b) {
  return make_uint4(min2(a.x, b.x), min2(a.y, b.y), min2(a.z, b.z), min2(a.w, b.w));
}
__device__ __forceinline__ uint4 max8(uint4 a, uint4 b) {
  return make_uint4(max2(a.x, b.x), max2(a.y, b.y), max2(a.z, b.z), max2(a.w, b.w));
}

// One CTA: a page and 32 neighbouring 8-element chunks of its slots' rows (a
// lane each); the eight warps take slots in turn and meet in shared memory.
template <int FMT>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const BoundParams p) {
  constexpr int WARPS = kBoundThreads / 32;
  __shared__ uint4 s_lo[WARPS][32], s_hi[WARPS][32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = blockIdx.x / p.slices;
  const int chunk = (int)(blockIdx.x - item * p.slices) * 32 + lane;
  const int cph = p.d / 8;
  const int page = __ldg(p.page_ids + item);
  int len = p.page_lens ? min(__ldg(p.page_lens + item), p.page_size) : p.page_size;
  if (page < 0 || page >= p.num_pages || len <= 0) return;  // (the same for the whole CTA)
  const int h = chunk / cph, c = chunk - h * cph;
  const bool have = h < p.hkv;
  const uint8_t *src = p.k + (int64_t)page * p.page_size * p.kb_ss + (have ? h : 0) * p.kb_hs +
                       c * (FMT == 0 ? 16 : 8);
  const uint32_t inf2 = 0x7F807F80u, ninf2 = 0xFF80FF80u;
  uint4 lo = make_uint4(inf2, inf2, inf2, inf2), hi = make_uint4(ninf2, ninf2, ninf2, ninf2);
  for (int s0 = warp; s0 < len; s0 += WARPS * kBoundUnroll) {
    uint4 x[kBoundUnroll];
    // (a slot past the end repeats the first one)
#pragma unroll
    for (int u = 0; u < kBoundUnroll; ++u) {
      const int s = s0 + u * WARPS;
      if (have) x[u] = load_keys<FMT>(src + (int64_t)(s < len ? s : s0) * p.kb_ss);
    }
    if (have) {
#pragma unroll
      for (int u = 0; u < kBoundUnroll; ++u) {
        lo = min8(lo, x[u]);
        hi = max8(hi, x[u]);
      }
    }
  }
  s_lo[warp][lane] = lo;
  s_hi[warp][lane] = hi;
  __syncthreads();
  if (warp < 2 && have) {
    uint4 r = warp == 0 ? s_lo[0][lane] : s_hi[0][lane];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) r = warp == 0 ? min8(r, s_lo[w][lane]) : max8(r, s_hi[w][lane]);
    p.bounds[(((int64_t)page * p.hkv + h) * 2 + warp) * cph + c] = r;
  }
}

int launch_update_page_bounds(const void *k_buffer, int64_t kb_ss, int64_t kb_hs, int kv_fmt,
                              int page_size, int64_t num_pages, int hkv, int d,
                              const int32_t *page_ids, const int32_t *page_lens, int64_t n_pages,
                              void *bounds, cudaStream_t st) {
  if (n_pages == 0) return PKX_OK;
  const int size = kv_fmt == kKvBf16 ? 2 : 1;
  BoundParams p;
  p.k = static_cast<const uint8_t *>(k_buffer);
  p.kb_ss = kb_ss * size;
  p.kb_hs = kb_hs * size;
  p.page_ids = page_ids;
  p.page_lens = page_lens;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.hkv = hkv;
  p.d = d;
  p.slices = (hkv * (d / 8) + 31) / 32;
  p.bounds = static_cast<uint4 *>(bounds);
  if (n_pages * p.slices >= (1ll << 31))
    return set_error(PKX_EUNSUPPORTED, "update_page_bounds: too many pages in one call");
  auto kernel = kv_fmt == kKvBf16      ? page_bounds_kernel<0>
                : kv_fmt == kKvFp8E4M3 ? page_bounds_kernel<1>
                                       : page_bounds_kernel<2>;
  cudaError_t e = launch_pdl(kernel, dim3((unsigned)(n_pages * p.slices)), dim3(kBoundThreads), 0,
                             st, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "update_page_bounds launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

// ------------------------------------------------------------------- score
constexpr int kScoreThreads = 128;
constexpr int kScoreRun = 32;   // entries of a warp, at most

struct ScoreParams {
  const uint16_t *q;
  const uint4 *bounds;
  int64_t num_pages;
  const int32_t *kv_indptr, *kv_indices;
  int64_t n_indices;
  int batch, hq, hkv, group, top_k;
  int run;         // entries of a warp, at most 32
  int64_t runs;    // runs of a KV head
  uint32_t *keys;  // [hkv][n_indices]
  WsHeader *hdr;
};

// A score as an unsigned key of the same order: NaN above everything, equal
// zeros equal.  0 stands for a page outside the bounds (no score maps there).
__device__ __forceinline__ uint32_t score_key(float s) {
  if (s != s) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(s + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// A lane's part of the q sums of one (sequence, KV head): chunk c (8 dims) of qp
// (`is_hi`) or qn.
template <int D>
__device__ __forceinline__ void query_sums(const uint16_t *q, int64_t first_row, int group, int c,
                                           bool is_hi, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = 0.f;
  const uint4 *row = reinterpret_cast<const uint4 *>(q + first_row * D) + c;
#pragma unroll 4
  for (int g = 0; g < group; ++g) {
    const uint4 v = __ldg(row + g * (D / 8));
    const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float qv = __uint_as_float(k & 1 ? wd[k / 2] & 0xFFFF0000u : wd[k / 2] << 16);
      // (a NaN stays one)
      f[k] = __fadd_rn(f[k], is_hi ? (qv <= 0.f ? 0.f : qv) : (qv >= 0.f ? 0.f : qv));
    }
  }
}

// The scores of eight copies (a copy: 512 bytes, the bounds of 128 / D pages, 16
// bytes a lane): lane l ends with the score of copy l % 8 (and its own page of
// the copy).  The lanes' sums meet in a butterfly in which a lane passes on the
// half of its values that its partner keeps, so that eight sums take 4 + 2 + 1
// shuffles (and one a level from there on), each of them the sum of two
// neighbours of the tree.
template <int D, typename F>
__device__ __forceinline__ float eight_scores(const float (&f)[8], F &&copy) {
  constexpr int LP = D / 4;  // lanes of a page
  const int lane = threadIdx.x & 31;
  float v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint4 x = copy(u);
    const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      t[k] = __fmul_rn(__uint_as_float(k & 1 ? wd[k / 2] & 0xFFFF0000u : wd[k / 2] << 16), f[k]);
#pragma unroll
    for (int m = 4; m > 0; m >>= 1)
#pragma unroll
      for (int k = 0; k < m; ++k) t[k] = __fadd_rn(t[2 * k], t[2 * k + 1]);
    v[u] = t[0];
  }
#pragma unroll
  for (int o = 1, m = 4; o < 8; o <<= 1, m >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < m; ++k) {
      const float keep = up ? v[2 * k + 1] : v[2 * k], pass = up ? v[2 * k] : v[2 * k + 1];
      v[k] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, pass, o));
    }
  }
#pragma unroll
  for (int o = 8; o < LP; o <<= 1) v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}

// A warp: one KV head and a run of up to 32 consecutive entries of kv_indices,
// whose page ids its lanes fetch together; neighbouring warps take the heads
// of the same pages.  D / 4 lanes hold a page's two bounds, 8 dims each.  All of
// the run's bounds are on their way (cp.async, each lane its own 16 bytes, so
// nothing is shared) before the warp looks for its sequence and sums up its
// queries: with loads into registers, 8 pages at a time, that preparation stood
// between the loads (64 sequences of 512 pages, 8 KV heads of 128, 134 MB: this
// kernel took 65 us and takes 35).
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const ScoreParams p) {
  constexpr int LP = D / 4;        // lanes of a page
  constexpr int PPW = 32 / LP;     // pages of a warp's copy
  constexpr int CH = D / 8;        // lanes of one bound
  constexpr int COPIES = kScoreRun / PPW;
  extern __shared__ __align__(16) uint8_t smem[];
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) p.hdr->status = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t w = (int64_t)blockIdx.x * (kScoreThreads / 32) + warp;
  if (w >= p.runs * p.hkv) return;
  const int64_t r = w / p.hkv;
  const int h = (int)(w - r * p.hkv);
  const int64_t e0 = r * p.run;
  const int sub = lane / LP, l = lane - sub * LP;
  const bool is_hi = l >= CH;
  const int c = is_hi ? l - CH : l;
  const int n = (int)min((int64_t)p.run, p.n_indices - e0);
  int my_page = lane < n ? __ldg(p.kv_indices + e0 + lane) : -1;
  if (my_page >= p.num_pages) my_page = -1;
  const uint4 *box = p.bounds + (int64_t)h * LP + l;
  const uint32_t mine = smem_u32(smem) + warp * (COPIES * 512) + lane * 16;
#pragma unroll
  for (int u = 0; u < COPIES; ++u) {
    const int page = __shfl_sync(0xffffffffu, my_page, u * PPW + sub);
    if (page >= 0) cp_async_16(mine + u * 512, box + (int64_t)page * p.hkv * LP, 16u);
    if (u % 8 == 7) cp_async_commit();
  }
  uint32_t *keys = p.keys + (int64_t)h * p.n_indices + e0;
  int landed = 0;  // copies that have
  for (int i = 0; i < n;) {
    // the sequence of entry e0 + i: the last b with kv_indptr[b] <= it, by 32
    // probes at a time
    const int64_t e = e0 + i;
    int b = 0;
    for (int span = p.batch; span > 1;) {
      const int step = (span + 31) / 32;
      const int at = lane * step;
      const bool before = at < span && (at == 0 || __ldg(p.kv_indptr + b + at) <= e);
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
      b += last * step;
      span = min(step, span - last * step);
    }
    const int64_t first = __ldg(p.kv_indptr + b), end = __ldg(p.kv_indptr + b + 1);
    if (first > e) {  // in front of the first sequence
      i = (int)min(first - e0, (int64_t)n);
      continue;
    }
    if (end <= e) break;  // behind the last one
    const int seg = (int)min(end - e0, (int64_t)n);
    if (end - first <= p.top_k) {  // all of its pages are taken
      i = seg;
      continue;
    }
    float f[8];
    query_sums<D>(p.q, (int64_t)b * p.hq + (int64_t)h * p.group, p.group, c, is_hi, f);
    // eight copies at a time (entries of other sequences in a copy are left out)
    for (int u0 = i / PPW / 8 * 8; u0 * PPW < seg; u0 += 8) {
      if (u0 >= landed) {
        landed = u0 + 8;
        switch (COPIES / 8 - landed / 8) {
          case 3: cp_async_wait_group<3>(); break;
          case 2: cp_async_wait_group<2>(); break;
          case 1: cp_async_wait_group<1>(); break;
          default: cp_async_wait_group<0>();
        }
      }
      const float score =
          eight_scores<D>(f, [&](int u) { return ld_shared_u4(mine + (u0 + u) * 512); });
      const int at = (u0 + (lane & 7)) * PPW + sub;
      const int page = __shfl_sync(0xffffffffu, my_page, at & 31);
      if (l < 8 && at >= i && at < seg) keys[at] = page < 0 ? 0u : score_key(score);
    }
    i = seg;
  }
  cp_async_wait_all();
}

// ------------------------------------------------------------------ select
struct SelectParams {
  const int32_t *kv_indptr;
  int64_t n_indices;
  int batch, hkv, top_k, first_pages, last_pages;
  const uint32_t *keys;
  int32_t *selected;
  int32_t *err;  // [batch * hkv] (the fused kernel)
  WsHeader *hdr;
};

// The threshold of the `want` largest of the CTA's keys: the largest T with
// count(key >= T) >= want, two bits a round, and `above` = count(key > T).  HELD
// keys a thread in registers (an absent one is 0, below every bound tried);
// keys from HELD * THREADS on are read again each round.
template <int THREADS, int HELD>
__device__ __forceinline__ void threshold(const uint32_t *keys, int m, int want,
                                          const uint32_t (&held)[16], int (*s_cnt)[32][3],
                                          uint32_t &T, int &above) {
  constexpr int WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  T = 0;
  above = 0;
  int parity = 0;
  for (int shift = 30; shift >= 0; shift -= 2, parity ^= 1) {
    const uint32_t t1 = T + (1u << shift), t2 = T + (2u << shift), t3 = T + (3u << shift);
    int c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
    for (int r = 0; r < HELD; ++r) {
      c1 += held[r] >= t1;
      c2 += held[r] >= t2;
      c3 += held[r] >= t3;
    }
    if constexpr (HELD == 16)
      for (int i = HELD * THREADS + tid; i < m; i += THREADS) {
        const uint32_t k = keys[i];
        c1 += k >= t1;
        c2 += k >= t2;
        c3 += k >= t3;
      }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    if constexpr (WARPS > 1) {
      if (lane == 0) {
        s_cnt[parity][warp][0] = c1;
        s_cnt[parity][warp][1] = c2;
        s_cnt[parity][warp][2] = c3;
      }
      __syncthreads();
      c1 = __reduce_add_sync(0xffffffffu, lane < WARPS ? s_cnt[parity][lane][0] : 0);
      c2 = __reduce_add_sync(0xffffffffu, lane < WARPS ? s_cnt[parity][lane][1] : 0);
      c3 = __reduce_add_sync(0xffffffffu, lane < WARPS ? s_cnt[parity][lane][2] : 0);
    }
    if (c3 >= want) T = t3;
    else if (c2 >= want) T = t2, above = c3;
    else if (c1 >= want) T = t1, above = c2;
    else above = c1;
  }
}

// Numbers of the pages of a sequence of n > top_k pages, by a CTA: `keys` are the
// ordered scores of the pages between the first and the last ones.  A thread
// keeps 16 keys in registers (keys i = r * THREADS + tid).  Returns whether this
// thread saw a page outside the bounds.
template <int THREADS>
__device__ __forceinline__ bool select_top(const SelectParams &p, int n, const uint32_t *keys,
                                           int32_t *out, int (*s_cnt)[32][3], int (*s_scan)[32]) {
  constexpr int kHeld = 16, WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = p.first_pages, m = n - p.first_pages - p.last_pages;
  const int want = p.top_k - p.first_pages - p.last_pages;  // 0 <= want < m
  uint32_t held[kHeld];
  bool lost = false;
#pragma unroll
  for (int r = 0; r < kHeld; ++r) {
    const int i = r * THREADS + tid;
    held[r] = i < m ? keys[i] : 0u;
    lost |= i < m && held[r] == 0u;
  }
  for (int i = kHeld * THREADS + tid; i < m; i += THREADS) lost |= keys[i] == 0u;
  for (int i = tid; i < p.first_pages; i += THREADS) out[i] = i;
  for (int i = tid; i < p.last_pages; i += THREADS)
    out[p.top_k - p.last_pages + i] = n - p.last_pages + i;
  if (want == 0) return lost;

  uint32_t T;
  int above;
  if (m <= THREADS) threshold<THREADS, 1>(keys, m, want, held, s_cnt, T, above);
  else if (m <= 2 * THREADS) threshold<THREADS, 2>(keys, m, want, held, s_cnt, T, above);
  else if (m <= 4 * THREADS) threshold<THREADS, 4>(keys, m, want, held, s_cnt, T, above);
  else if (m <= 8 * THREADS) threshold<THREADS, 8>(keys, m, want, held, s_cnt, T, above);
  else threshold<THREADS, 16>(keys, m, want, held, s_cnt, T, above);
  const int ties = want - above;  // keys equal to T that are taken, lowest first

  // the pages in order: a running count of keys above T and equal to it
  int gt = 0, eq = 0;
  auto place = [&](int r, uint32_t k) {
    const int i = r * THREADS + tid;
    const unsigned g = __ballot_sync(0xffffffffu, i < m && k > T);
    const unsigned q = __ballot_sync(0xffffffffu, i < m && k == T);
    int all = __popc(g) | (__popc(q) << 16), before = 0;
    if constexpr (WARPS > 1) {
      if (lane == 0) s_scan[r & 1][warp] = all;
      __syncthreads();
      const int x = lane < WARPS ? s_scan[r & 1][lane] : 0;
      all = __reduce_add_sync(0xffffffffu, x);
      before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
    }
    const unsigned below = (1u << lane) - 1u;
    const int my_gt = gt + (before & 0xFFFF) + __popc(g & below);
    const int my_eq = eq + (before >> 16) + __popc(q & below);
    // (pos < want always, but where two calls use one workspace at once)
    const int pos = my_gt + min(my_eq, ties);
    if (i < m && (k > T || (k == T && my_eq < ties)) && pos < want) out[lo + pos] = lo + i;
    gt += all & 0xFFFF;
    eq += all >> 16;
  };
#pragma unroll
  for (int r = 0; r < kHeld; ++r)
    if (r * THREADS < m) place(r, held[r]);
  for (int r = kHeld; r * THREADS < m; ++r) {
    const int i = r * THREADS + tid;
    place(r, i < m ? keys[i] : 0u);
  }
  return lost;
}

// Whether kv_indptr decreases anywhere (a CTA asks together).  Sequences may then
// overlap, and of the keys in the workspace, one an entry of kv_indices and KV head,
// some be another sequence's.
template <int THREADS>
__device__ __forceinline__ bool decreases(const int32_t *indptr, int batch) {
  bool any = false;
  for (int i = threadIdx.x; i < batch; i += THREADS) any |= __ldg(indptr + i + 1) < __ldg(indptr + i);
  return __syncthreads_or(any);
}

// One CTA for each (sequence, KV head): its pages' numbers from the keys in the
// workspace.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) page_select_kernel(const SelectParams p) {
  __shared__ int s_cnt[2][32][3];
  __shared__ int s_scan[2][32];
  grid_dep_wait();
  grid_dep_launch();
  const int b = blockIdx.x / p.hkv, h = blockIdx.x - b * p.hkv;
  const int64_t at = __ldg(p.kv_indptr + b);
  const int64_t n64 = (int64_t)__ldg(p.kv_indptr + b + 1) - at;
  int32_t *out = p.selected + (int64_t)blockIdx.x * p.top_k;
  const bool bad = at < 0 || n64 < 0 || at + n64 > p.n_indices ||
                   (n64 > p.top_k && decreases<THREADS>(p.kv_indptr, p.batch));
  bool lost = bad;
  const int n = bad ? 0 : (int)n64;
  if (n <= p.top_k) {  // every page
    for (int i = threadIdx.x; i < p.top_k; i += THREADS) out[i] = i < n ? i : -1;
  } else {
    lost = select_top<THREADS>(p, n, p.keys + (int64_t)h * p.n_indices + at + p.first_pages, out,
                               s_cnt, s_scan);
  }
  if (lost) atomicCAS(&p.hdr->status, 0, PKX_EDEVICE);
}

// Scores and selection in one: a CTA for each (sequence, KV head), whose warps
// take eight copies of bounds at a time and leave the keys in shared memory (in
// the workspace past kFusedKeys pages).  The queries are summed once a CTA and the
// keys make no round trip; it needs CTAs enough to fill the GPU.  A warp keeps the
// next eight copies on their way (cp.async, each lane its own 16 bytes).  64
// sequences of 512 pages, 8 KV heads of 128 (134 MB): 31 us back to back in a
// captured graph and 41 from a cold cache, by two kernels 48 and 58.
constexpr int kFusedKeys = 2048;
constexpr int kFusedRing = 2 * 8 * 512;  // bytes of a warp
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 640 / THREADS) page_score_select_kernel(
    const ScoreParams p, const SelectParams sp) {
  constexpr int LP = D / 4, PPW = 32 / LP, CH = D / 8, WARPS = THREADS / 32;
  constexpr int STEP = 8 * PPW;  // pages of a warp's step
  __shared__ uint32_t s_keys[kFusedKeys];
  extern __shared__ __align__(16) uint8_t smem[];  // [WARPS][2][8 copies]
  __shared__ int s_cnt[2][32][3];
  __shared__ int s_scan[2][32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / p.hkv, h = blockIdx.x - b * p.hkv;
  const int64_t at = __ldg(p.kv_indptr + b);
  const int64_t n64 = (int64_t)__ldg(p.kv_indptr + b + 1) - at;
  int32_t *out = sp.selected + (int64_t)blockIdx.x * p.top_k;
  const bool bad = at < 0 || n64 < 0 || at + n64 > p.n_indices ||
                   (n64 - sp.first_pages - sp.last_pages > kFusedKeys &&
                    decreases<THREADS>(p.kv_indptr, p.batch));
  bool lost = bad;
  const int n = bad ? 0 : (int)n64;
  if (n <= p.top_k) {  // every page
    for (int i = threadIdx.x; i < p.top_k; i += THREADS) out[i] = i < n ? i : -1;
  } else {
    const int sub = lane / LP, l = lane - sub * LP;
    const bool is_hi = l >= CH;
    const int32_t *ids = p.kv_indices + at + sp.first_pages;
    const int m = n - sp.first_pages - sp.last_pages;
    uint32_t *keys = m <= kFusedKeys ? s_keys : p.keys + (int64_t)h * p.n_indices + at;
    auto fetch = [&](int i0) {  // page ids of a step, a lane each
      const int i = i0 + lane;
      const int page = lane < STEP && i < m ? __ldg(ids + i) : -1;
      return page < p.num_pages ? page : -1;
    };
    const uint4 *box = p.bounds + (int64_t)h * LP + l;
    const uint32_t mine = smem_u32(smem) + warp * kFusedRing + lane * 16;
    auto issue = [&](int stage, int pages) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int page = __shfl_sync(0xffffffffu, pages, u * PPW + sub);
        if (page >= 0)
          cp_async_16(mine + stage * 4096 + u * 512, box + (int64_t)page * p.hkv * LP, 16u);
      }
      cp_async_commit();
    };
    int here = fetch(warp * STEP), next = fetch((warp + WARPS) * STEP);
    issue(0, here);
    float f[8];
    query_sums<D>(p.q, (int64_t)b * p.hq + (int64_t)h * p.group, p.group, is_hi ? l - CH : l, is_hi,
                  f);
    int stage = 0;
    for (int i0 = warp * STEP; i0 < m; i0 += WARPS * STEP, stage ^= 1) {
      issue(stage ^ 1, next);
      const int after = fetch(i0 + 2 * WARPS * STEP);
      cp_async_wait_group<1>();
      const float score = eight_scores<D>(
          f, [&](int u) { return ld_shared_u4(mine + stage * 4096 + u * 512); });
      const int j = (lane & 7) * PPW + sub;
      const int page = __shfl_sync(0xffffffffu, here, j);
      if (l < 8 && i0 + j < m) keys[i0 + j] = page < 0 ? 0u : score_key(score);
      here = next;
      next = after;
    }
    cp_async_wait_all();
    __syncthreads();
    lost = select_top<THREADS>(sp, n, keys, out, s_cnt, s_scan);
  }
  lost = __syncthreads_or(lost);
  if (threadIdx.x == 0) {
    sp.err[blockIdx.x] = lost;
    if (blockIdx.x == 0) set_status_in_units(p.hdr, sp.err, gridDim.x);
  }
}

static size_t select_keys_offset(int batch, int hkv) {
  return 256 + ((sizeof(int32_t) * (size_t)batch * (size_t)hkv + 255) & ~(size_t)255);
}
size_t select_pages_workspace(int batch, int hkv, int64_t n_indices) {
  return select_keys_offset(batch, hkv) +
         ((sizeof(uint32_t) * (size_t)hkv * (size_t)n_indices + 255) & ~(size_t)255);
}

template <int D, int THREADS>
static int launch_score_select(const ScoreParams &p, const SelectParams &s, dim3 pairs,
                               cudaStream_t st) {
  constexpr int smem = THREADS / 32 * kFusedRing;
  static PerDevice configured;
  std::atomic<int> *done = configured.here();
  cudaError_t e = cudaSuccess;
  if (!done || done->load(std::memory_order_acquire) == 0) {
    e = cudaFuncSetAttribute(page_score_select_kernel<D, THREADS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && done) done->store(1, std::memory_order_release);
  }
  if (e == cudaSuccess)
    e = launch_pdl(page_score_select_kernel<D, THREADS>, pairs, dim3(THREADS), smem, st, p, s);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "page_score_select launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

int launch_select_pages(const SelectArgs &a) {
  if (a.batch == 0) return PKX_OK;
  const int nsm = num_sms_current_device();
  if (nsm <= 0) return set_error(PKX_ECUDA, "cannot query the current device");
  WsHeader *hdr = static_cast<WsHeader *>(a.workspace);
  uint32_t *keys = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.workspace) +
                                                select_keys_offset(a.batch, a.hkv));
  ScoreParams p;
  p.q = static_cast<const uint16_t *>(a.q);
  p.bounds = static_cast<const uint4 *>(a.bounds);
  p.num_pages = a.num_pages;
  p.kv_indptr = a.kv_indptr;
  p.kv_indices = a.kv_indices;
  p.n_indices = a.n_indices;
  p.batch = a.batch;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = a.hq / a.hkv;
  p.top_k = a.top_k;
  p.keys = keys;
  p.hdr = hdr;
  SelectParams s;
  s.kv_indptr = a.kv_indptr;
  s.n_indices = a.n_indices;
  s.batch = a.batch;
  s.hkv = a.hkv;
  s.top_k = a.top_k;
  s.first_pages = a.first_pages;
  s.last_pages = a.last_pages;
  s.keys = keys;
  s.selected = a.selected;
  s.hdr = hdr;
  s.err = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(a.workspace) + 256);
  if ((int64_t)a.batch * a.hkv >= (1ll << 31))
    return set_error(PKX_EUNSUPPORTED, "select_pages: batch too large");
  const dim3 pairs((unsigned)(a.batch * a.hkv));
  // One kernel where the (sequence, KV head) pairs fill the GPU or where there is
  // too little to spread, else scores by runs of pages, then the selection.  Back
  // to back in a captured graph, 8 KV heads of 128, one kernel / two: 64 sequences of
  // 512 pages 31 / 48 us, 24 of them 16.5 / 23; 5 sequences of up to 49 pages, 3 KV
  // heads 8.3 / 10.3.  The rules below go by the number of pairs and the batch's
  // average, which the host knows, not by each sequence: one sequence of 8192 pages
  // and 23 of 20 take 90 us (two kernels: 109), one of 6000 and 15 of 20, whose long
  // rows a warp selects from, 82.
  const int64_t mean = a.n_indices / a.batch;
  if ((int64_t)a.batch * a.hkv >= nsm || mean <= 256) {
    // eight warps a pair for up to three pairs an SM, else four (512 pages each, 8 KV
    // heads, from a cold cache, eight / four: 24 sequences 25 / 28 us, 57: 37 / 37, 64:
    // 48 / 41, 96: 58 / 64)
    if (pairs.x <= 3u * nsm)
      return a.d == 128 ? launch_score_select<128, 256>(p, s, pairs, a.stream)
                        : launch_score_select<64, 256>(p, s, pairs, a.stream);
    return a.d == 128 ? launch_score_select<128, 128>(p, s, pairs, a.stream)
                      : launch_score_select<64, 128>(p, s, pairs, a.stream);
  }
  // a warp's run: 32 entries, or fewer where that leaves less than 16 warps an
  // SM (a run reads the group's query rows once)
  int64_t run = a.n_indices * a.hkv / ((int64_t)nsm * 16);
  run = run < 8 ? 8 : run > kScoreRun ? kScoreRun : run / 8 * 8;
  p.run = (int)run;
  p.runs = (a.n_indices + run - 1) / run;
  int64_t grid = (p.runs * a.hkv + kScoreThreads / 32 - 1) / (kScoreThreads / 32);
  if (grid < 1) grid = 1;  // (the status word)
  if (grid >= (1ll << 31))
    return set_error(PKX_EUNSUPPORTED, "select_pages: too many pages in one call");
  auto score = a.d == 128 ? page_score_kernel<128> : page_score_kernel<64>;
  const size_t smem = (size_t)(kScoreThreads / 32) * kScoreRun * a.d * 4;  // 64 KB at most
  static PerDevice configured[2];
  std::atomic<int> *done = configured[a.d == 128].here();
  cudaError_t e = cudaSuccess;
  if (!done || done->load(std::memory_order_acquire) == 0) {
    e = cudaFuncSetAttribute(score, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && done) done->store(1, std::memory_order_release);
  }
  if (e == cudaSuccess)
    e = launch_pdl(score, dim3((unsigned)grid), dim3(kScoreThreads), smem, a.stream, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "page_score launch: %s", cudaGetErrorString(e));
  // By the batch's average: a warp holds 512 keys and needs no barrier, 256
  // threads hold 4096, 1024 hold 16384.
  if (mean <= 512)
    e = launch_pdl(page_select_kernel<32>, pairs, dim3(32), 0, a.stream, s);
  else if (mean <= 4096)
    e = launch_pdl(page_select_kernel<256>, pairs, dim3(256), 0, a.stream, s);
  else
    e = launch_pdl(page_select_kernel<1024>, pairs, dim3(1024), 0, a.stream, s);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "page_select launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
