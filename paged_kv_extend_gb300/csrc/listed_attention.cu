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
//  * selected pages: each (sequence, KV head) attends to pages of its own; a
//    first kernel writes its list of pool slots, and the units follow from the
//    batch alone (equal shares of the longest list), so no scan is needed.
//
// Partials are fp32 (o normalised, lse in natural logs) and merged as
//   lse = log sum_i exp(lse_i),  o = sum_i exp(lse_i - lse) o_i.
// A unit's partial rows lie in granules of Hq / Hkv rows (one token's heads of
// one KV head): n_tok granules a key stream, so that a one-token unit takes two
// and not two whole tiles.
#include <algorithm>
#include <climits>
#include <cstring>
#include <cuda_runtime.h>

#include "attn_kernel.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

// Position of every listed unit's queries: past every key, so that no causal
// mask applies.
constexpr int kPastAll = 1 << 30;

// Where a token's partials lie: granule a + kvh * a_head + i * a_step + s *
// a_stream for its prefix (i < a_n splits, s < a_streams), likewise b for its own
// keys (two streams, one granule apart).
struct __align__(16) ListedRow {
  int32_t a, a_n, a_head, a_step, a_streams, a_stream, b, b_n;
};

struct ListedLayout {
  size_t seq_off, grp_off, units_off, order_off, rows_off, idx_off, ptr_off, err_off, plse_off,
      po_off, total;
  int unit_max;
  int64_t gran_max;
  int unit_target;
};

static size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// ------------------------------------------------------------------ combine
// One warp a (token, head) row: the lanes hold up to 32 partials' weights, the
// row's dims are split over the lanes (float4 each).
template <int D>
__global__ void __launch_bounds__(256) listed_combine_kernel(
    const ListedRow *__restrict__ rows, const float *__restrict__ plse,
    const float *__restrict__ po, bf16 *__restrict__ o, float *__restrict__ lse, int batch, int hq,
    int group, int b_head, int b_step, const int32_t *__restrict__ err, int n_err,
    int32_t *status) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr float kLog2e = 1.4426950408889634f;
  if (err && blockIdx.x == 0)  // errors that the listing kernel's CTAs found
    for (int i = threadIdx.x; i < n_err; i += blockDim.x)
      if (err[i]) record_status(status, PKX_EDEVICE);
  const int lane = threadIdx.x & 31;
  const int nw = (gridDim.x * blockDim.x) >> 5;
  for (int64_t r = (blockIdx.x * blockDim.x + threadIdx.x) >> 5; r < (int64_t)batch * hq; r += nw) {
    const int t = (int)(r / hq), head = (int)(r - (int64_t)t * hq);
    const int kvh = head / group, g = head - kvh * group;
    const ListedRow R = rows[t];
    const int na = R.a_n * R.a_streams, n = na + 2 * R.b_n;
    auto row_of = [&](int i) -> int64_t {
      int64_t gr;
      if (i < na) {
        const int sp = R.a_streams == 2 ? i >> 1 : i, s = i - sp * R.a_streams;
        gr = (int64_t)R.a + (int64_t)kvh * R.a_head + (int64_t)sp * R.a_step + s * R.a_stream;
      } else {
        const int j = i - na;
        gr = (int64_t)R.b + (int64_t)kvh * b_head + (int64_t)(j >> 1) * b_step + (j & 1);
      }
      return gr * group + g;
    };
    // maximum of the partials' log sums (fmaxf drops a NaN one, which comes
    // back as a NaN weight below)
    float mx = -INFINITY;
    bool any = false;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const float x = i0 + lane < n ? plse[row_of(i0 + lane)] : -INFINITY;
      any |= !(x == -INFINITY);
      mx = fmaxf(mx, x);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    any = __any_sync(0xffffffffu, any);
    bf16 *orow = o + r * D;
    if (!any) {  // no visible key
      if (lane * 4 < D) *reinterpret_cast<uint2 *>(orow + lane * 4) = make_uint2(0, 0);
      if (lane == 0 && lse) lse[r] = -INFINITY;
      continue;
    }
    float wsum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < n; i0 += 32) {
      const bool have = i0 + lane < n;
      const int64_t row = have ? row_of(i0 + lane) : 0;
      const float w = have ? exp2f((plse[row] - mx) * kLog2e) : 0.f;
      wsum += w;
      const int m = min(32, n - i0);
      for (int i = 0; i < m; i += 8) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t at = __shfl_sync(0xffffffffu, row, (i + u) & 31);
          if (i + u < m && lane * 4 < D)
            v[u] = *reinterpret_cast<const float4 *>(po + at * D + lane * 4);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float wi = __shfl_sync(0xffffffffu, w, (i + u) & 31);
          // (a stream without keys has weight 0 and a row of zeros)
          if (i + u < m && lane * 4 < D) {
            acc[0] += wi * v[u].x;
            acc[1] += wi * v[u].y;
            acc[2] += wi * v[u].z;
            acc[3] += wi * v[u].w;
          }
        }
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, s);
    const float inv = 1.0f / wsum;
    if (lane * 4 < D)
      *reinterpret_cast<uint2 *>(orow + lane * 4) =
          make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    if (lane == 0 && lse) lse[r] = mx + logf(wsum);
  }
}

// --------------------------------------------------------- shared prefixes
struct SharedParams {
  const int32_t *kv_indptr, *group_indptr, *shared_lens;
  int batch, num_groups, hkv;
  int tok;          // tokens of a query tile
  int target;       // units wanted
  int unit_max;
  int64_t gran_max;
  int32_t *seq;     // [3][batch + 1]: keys, shared keys, first unit of own keys
  int32_t *grp;     // [3][num_groups + 1]: shared keys, first unit, first granule
  WorkUnit *units;
  int32_t *order;
  ListedRow *rows;
  WsHeader *hdr;
};

// Exclusive sum over a block of 1024 threads of one value each, and the total.
__device__ int64_t block_sum_before(int64_t v, int64_t *sh, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    const int64_t y = sh[w];
    if (w < warp) before += y;
    all += y;
  }
  __syncthreads();
  total = all;
  return before + x - v;
}

// One CTA of 1024 threads: the units of every group's prefix and of every
// sequence's own keys.  A group shares min(shared_lens, the shortest of its
// sequences) keys, nothing if that is less than a tile of keys or if it has one
// sequence.  Key ranges are cut into equal pieces of at most C tiles, C chosen
// for about `target` units.
__global__ void __launch_bounds__(1024, 1) shared_sched_kernel(const SharedParams p) {
  __shared__ int64_t sh[32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.batch, NG = p.num_groups;
  int32_t *sT = p.seq, *sS = p.seq + (B + 1), *sU = p.seq + 2 * (B + 1);
  int32_t *gS = p.grp, *gU = p.grp + (NG + 1), *gG = p.grp + 2 * (NG + 1);
  const int blk = 2 * p.tok;  // tokens of a prefix unit
  if (tid == 0) s_bad = 0;
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  bool bad = false;
  // sequences
  for (int b = tid; b < B; b += 1024) {
    const int k0 = p.kv_indptr[b], T = p.kv_indptr[b + 1] - k0;
    const bool ok = k0 >= 0 && T >= 0;
    bad |= !ok;
    sT[b] = ok ? T : 0;
    sS[b] = 0;
  }
  // groups: consecutive runs of sequences, else nothing is shared
  bool bad_groups = false;
  for (int g = tid; g < NG; g += 1024) {
    const int lo = p.group_indptr[g], hi = p.group_indptr[g + 1];
    bad_groups |= lo < 0 || hi < lo || hi > B || p.shared_lens[g] < 0;
  }
  if (bad_groups) s_bad = 1;
  bad |= bad_groups;
  if (tid == 0) {
    p.hdr->status = 0;
    p.hdr->next_unit = 0;
  }
  __syncthreads();
  if (bad) record_status(&p.hdr->status, PKX_EDEVICE);
  const bool share = s_bad == 0;
  // shared keys of each group (a warp each)
  for (int g = warp; g < NG; g += 32) {
    int S = 0;
    if (share) {
      const int lo = p.group_indptr[g], hi = p.group_indptr[g + 1];
      int least = p.shared_lens[g];
      for (int b = lo + lane; b < hi; b += 32) least = min(least, sT[b]);
      least = __reduce_min_sync(0xffffffffu, least);
      if (hi - lo >= 2 && least >= kBlockN) S = least;
      for (int b = lo + lane; b < hi; b += 32) sS[b] = S;
    }
    if (lane == 0) gS[g] = S;
  }
  __syncthreads();
  // size of a piece
  auto tiles = [](int keys) { return keys / kBlockN + (keys % kBlockN != 0); };
  auto group_blocks = [&](int g) {
    return gS[g] > 0 ? (p.group_indptr[g + 1] - p.group_indptr[g] + blk - 1) / blk : 0;
  };
  int64_t cost = 0;
  for (int b = tid; b < B; b += 1024) cost += tiles(sT[b] - sS[b]);
  for (int g = tid; g < NG; g += 1024) cost += (int64_t)group_blocks(g) * tiles(gS[g]);
  int64_t all_cost;
  block_sum_before(cost, sh, all_cost);
  const int64_t c64 = (all_cost * p.hkv + p.target - 1) / p.target;
  const int C = (int)max(c64, (int64_t)kMinSplitTiles);
  auto pieces = [&](int nt) { return (nt + C - 1) / C; };
  // granules of a group's piece (all its blocks, one KV head): two streams of
  // partials where the block is one tile of rows
  auto group_granules = [&](int g) {
    const int nb = group_blocks(g);
    const int last = p.group_indptr[g + 1] - p.group_indptr[g] - (nb - 1) * blk;
    return (nb - 1) * blk + (last <= p.tok ? 2 * last : last);
  };
  // first unit and granule of each group, first unit of each sequence
  const int gc = (NG + 1023) / 1024, g0 = min(NG, tid * gc), g1 = min(NG, g0 + gc);
  int64_t nu = 0, ng = 0;
  for (int g = g0; g < g1; ++g) {
    if (gS[g] <= 0) continue;
    const int s = pieces(tiles(gS[g]));
    nu += (int64_t)s * group_blocks(g) * p.hkv;
    ng += (int64_t)s * p.hkv * group_granules(g);
  }
  int64_t pre_units, pre_gran, own_units;
  nu = block_sum_before(nu, sh, pre_units);
  ng = block_sum_before(ng, sh, pre_gran);
  const int bc = (B + 1023) / 1024, b0 = min(B, tid * bc), b1 = min(B, b0 + bc);
  int64_t bu = 0;
  for (int b = b0; b < b1; ++b) bu += pieces(tiles(sT[b] - sS[b]));
  bu = block_sum_before(bu, sh, own_units);
  own_units *= p.hkv;
  // (cannot be false: the workspace is sized for the largest counts)
  const bool fits = pre_units + own_units <= p.unit_max &&
                    pre_gran + 2 * own_units <= p.gran_max;
  if (!fits) {
    if (tid == 0) {
      record_status(&p.hdr->status, PKX_EDEVICE);
      p.hdr->n_units = 0;
    }
    for (int b = tid; b < B; b += 1024) p.rows[b] = ListedRow{};
    return;
  }
  for (int g = g0; g < g1; ++g) {
    gU[g] = (int)nu;
    gG[g] = (int)ng;
    if (gS[g] <= 0) continue;
    const int s = pieces(tiles(gS[g]));
    nu += (int64_t)s * group_blocks(g) * p.hkv;
    ng += (int64_t)s * p.hkv * group_granules(g);
  }
  for (int b = b0; b < b1; ++b) {
    sU[b] = (int)bu;
    bu += pieces(tiles(sT[b] - sS[b]));
  }
  __syncthreads();
  // units of the prefixes: group, piece, KV head, block (blocks of one piece
  // and head next to each other: they read the same keys)
  for (int u = tid; u < (int)pre_units; u += 1024) {
    int lo = 0, hi = NG - 1;  // last g with gU[g] <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (gU[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    const int g = lo, nb = group_blocks(g), nt = tiles(gS[g]), S = pieces(nt);
    int r = u - gU[g];
    const int k = r % nb;
    r /= nb;
    const int kvh = r % p.hkv, sp = r / p.hkv;
    const int first = p.group_indptr[g], n = p.group_indptr[g + 1] - first;
    WorkUnit w;
    w.q_tok0 = first + k * blk;
    w.n_tok = min(blk, n - k * blk);
    w.qpos0 = kPastAll;
    w.kvh = kvh;
    w.k_begin = (int)min((int64_t)gS[g], (int64_t)sp * nt / S * kBlockN);
    w.k_end = (int)min((int64_t)gS[g], (int64_t)(sp + 1) * nt / S * kBlockN);
    w.k_split = INT_MAX;
    w.n_tiles = tiles(w.k_end - w.k_begin);
    w.b = first;
    w.slot = gG[g] + (sp * p.hkv + kvh) * group_granules(g) + k * blk;
    w.dq = w.claim = 0;
    p.units[u] = w;
    p.order[u] = u;
  }
  // units of the sequences' own keys: sequence, piece, KV head
  for (int i = tid; i < (int)own_units; i += 1024) {
    const int x = i / p.hkv, kvh = i - x * p.hkv;
    int lo = 0, hi = B - 1;  // last b with sU[b] <= x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sU[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo, nt = tiles(sT[b] - sS[b]), S = pieces(nt), sp = x - sU[b];
    WorkUnit w;
    w.q_tok0 = b;
    w.n_tok = 1;
    w.qpos0 = kPastAll;
    w.kvh = kvh;
    w.k_begin = (int)min((int64_t)sT[b], sS[b] + (int64_t)sp * nt / S * kBlockN);
    w.k_end = (int)min((int64_t)sT[b], sS[b] + (int64_t)(sp + 1) * nt / S * kBlockN);
    w.k_split = INT_MAX;
    w.n_tiles = tiles(w.k_end - w.k_begin);
    w.b = b;
    w.slot = (int)pre_gran + 2 * i;
    w.dq = w.claim = 0;
    p.units[(int)pre_units + i] = w;
    p.order[(int)pre_units + i] = (int)pre_units + i;
  }
  // where each token's partials lie
  for (int b = tid; b < B; b += 1024) {
    ListedRow R{};
    if (sS[b] > 0) {
      int lo = 0, hi = NG - 1;  // last g with group_indptr[g] <= b
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.group_indptr[mid] <= b) lo = mid;
        else hi = mid - 1;
      }
      const int g = lo, i = b - p.group_indptr[g], k = i / blk;
      const int n_tok = min(blk, p.group_indptr[g + 1] - p.group_indptr[g] - k * blk);
      R.a = gG[g] + i;
      R.a_n = pieces(tiles(gS[g]));
      R.a_head = group_granules(g);
      R.a_step = p.hkv * R.a_head;
      R.a_streams = n_tok <= p.tok ? 2 : 1;
      R.a_stream = n_tok;
    }
    R.b = (int)pre_gran + 2 * sU[b] * p.hkv;
    R.b_n = pieces(tiles(sT[b] - sS[b]));
    p.rows[b] = R;
  }
  if (tid == 0) p.hdr->n_units = (int)(pre_units + own_units);
}

static ListedLayout shared_layout(int batch, int num_groups, int hkv, int group, int d,
                                  int num_sms) {
  ListedLayout L{};
  const int tok = tokens_per_block(group), blk = 2 * tok;
  L.unit_target = 3 * (num_sms > 0 ? num_sms : 160);
  // blocks: at most one partly filled a group (of two sequences or more)
  const int64_t blocks = batch / blk + std::min(num_groups, batch / 2);
  const int64_t units = L.unit_target + (int64_t)hkv * (blocks + batch);
  L.unit_max = (int)std::min<int64_t>(units, INT_MAX / 4);
  // a prefix unit has at most blk granules, and a block's first piece twice
  // its tokens; a unit of own keys has two
  L.gran_max = (int64_t)L.unit_target * (blk + 2) + 4 * (int64_t)hkv * batch;
  size_t off = up256(sizeof(WsHeader));
  L.seq_off = off;
  off = up256(off + sizeof(int32_t) * 3 * (size_t)(batch + 1));
  L.grp_off = off;
  off = up256(off + sizeof(int32_t) * 3 * (size_t)(num_groups + 1));
  L.units_off = off;
  off = up256(off + sizeof(WorkUnit) * (size_t)L.unit_max);
  L.order_off = off;
  off = up256(off + sizeof(int32_t) * (size_t)L.unit_max);
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
  int cap;         // keys of its list: top_k * page_size
  int32_t *slots;  // [batch * hkv][cap]
  int32_t *ptr;    // [batch * hkv] first key of each list
  int32_t *err;    // [batch * hkv]
  WorkUnit *units;
  int32_t *order;
  ListedRow *rows;
  WsHeader *hdr;
};

// One CTA for each (sequence, KV head): the pool slots of its selected pages
// one after another, and its units (equal shares of the list).
__global__ void __launch_bounds__(256) list_pages_kernel(const PagesParams p) {
  extern __shared__ int s_first[];  // [top_k + 1] first key of each entry
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
  // first key of each entry: a running sum of the entries' lengths
  for (int e0 = 0; e0 < p.top_k; e0 += 256) {
    const int e = e0 + tid;
    int len = 0;
    if (e < p.top_k) {
      const int s = sel[e];
      bad |= s >= n;
      if (s >= 0 && s < n) len = s == n - 1 ? min(max(last, 0), p.page_size) : p.page_size;
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
      R.b = pair * p.pieces * 2;
      R.b_n = p.pieces;
      p.rows[b] = R;
    }
  }
  const int nt = (keys + kBlockN - 1) / kBlockN;
  for (int s = tid; s < p.pieces; s += 256) {
    const int u = pair * p.pieces + s;
    WorkUnit w;
    w.q_tok0 = b;
    w.n_tok = 1;
    w.qpos0 = kPastAll;
    w.kvh = kvh;
    w.k_begin = (int)min((int64_t)keys, (int64_t)s * nt / p.pieces * kBlockN);
    w.k_end = (int)min((int64_t)keys, (int64_t)(s + 1) * nt / p.pieces * kBlockN);
    w.k_split = INT_MAX;
    w.n_tiles = (w.k_end - w.k_begin + kBlockN - 1) / kBlockN;
    w.b = pair;
    w.slot = 2 * u;
    w.dq = w.claim = 0;
    p.units[u] = w;
    p.order[u] = u;
  }
  // the slots; a page outside the pool is listed as -1, which the attention
  // kernel reads as a zero row and reports
  int32_t *out = p.slots + (int64_t)pair * p.cap;
  const int64_t pages = p.num_slots / p.page_size;
  for (int i = tid; i < p.top_k * p.page_size; i += 256) {
    const int e = i / p.page_size, j = i - e * p.page_size;
    if (j >= s_first[e + 1] - s_first[e]) continue;
    const int page = __ldg(p.kv_indices + at + sel[e]);
    out[s_first[e] + j] = page >= 0 && page < pages ? page * p.page_size + j : -1;
  }
}

// Units of a (sequence, KV head): at least kMinSplitTiles tiles each, and no
// more than make four units an SM.
static int pages_pieces(int batch, int hkv, int page_size, int top_k, int num_sms) {
  const int64_t nt = ((int64_t)top_k * page_size + kBlockN - 1) / kBlockN;
  const int64_t pairs = (int64_t)batch * hkv;
  const int64_t want = (4ll * (num_sms > 0 ? num_sms : 160) + pairs - 1) / std::max<int64_t>(pairs, 1);
  return (int)std::max<int64_t>(1, std::min(want, nt / kMinSplitTiles));
}

static ListedLayout pages_layout(int batch, int hkv, int group, int d, int page_size, int top_k,
                                 int num_sms) {
  ListedLayout L{};
  const int64_t pairs = (int64_t)batch * hkv;
  const int64_t units = pairs * pages_pieces(batch, hkv, page_size, top_k, num_sms);
  L.unit_max = (int)std::min<int64_t>(units, INT_MAX / 4);
  L.gran_max = 2 * units;
  size_t off = up256(sizeof(WsHeader));
  L.units_off = off;
  off = up256(off + sizeof(WorkUnit) * (size_t)units);
  L.order_off = off;
  off = up256(off + sizeof(int32_t) * (size_t)units);
  L.rows_off = off;
  off = up256(off + sizeof(ListedRow) * (size_t)batch);
  L.ptr_off = off;
  off = up256(off + sizeof(int32_t) * (size_t)pairs);
  L.err_off = off;
  off = up256(off + sizeof(int32_t) * (size_t)pairs);
  L.idx_off = off;
  off = up256(off + sizeof(int32_t) * (size_t)pairs * top_k * page_size);
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

// The attention kernel and the combine over the units in the workspace.
static int run_listed(const ListedArgs &a, const ListedMaps &tm, const ListedLayout &L, int nsm,
                      const int32_t *kv_indptr, const int32_t *kv_indices, int b_head, int b_step,
                      const int32_t *err, int n_err) {
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
  kp.uorder = reinterpret_cast<int32_t *>(ws + L.order_off);
  kp.next_unit = &hdr->next_unit;
  kp.hdr = hdr;
  kp.status = &hdr->status;
  kp.plse = reinterpret_cast<float *>(ws + L.plse_off);
  kp.po = reinterpret_cast<float *>(ws + L.po_off);
  wait_settings(&kp.wait_ns, &kp.stall);
  cudaEvent_t ev_before = nullptr, ev_after = nullptr;
  attention_events(&ev_before, &ev_after);
  if (ev_before) cudaEventRecord(ev_before, a.stream);
  const int rc = a.d == 128 ? launch_listed<128>(a.kv_fmt, tm, kp, nsm, a.stream)
                            : launch_listed<64>(a.kv_fmt, tm, kp, nsm, a.stream);
  if (rc != PKX_OK) return rc;
  if (ev_after) cudaEventRecord(ev_after, a.stream);
  const int64_t ctas = ((int64_t)a.batch * a.hq + 7) / 8;
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, (int64_t)nsm * 8);
  cudaError_t e = launch_pdl(
      a.d == 128 ? listed_combine_kernel<128> : listed_combine_kernel<64>, dim3(grid), dim3(256), 0,
      a.stream, reinterpret_cast<const ListedRow *>(ws + L.rows_off), (const float *)kp.plse,
      (const float *)kp.po, kp.o, a.lse, a.batch, a.hq, group, b_head, b_step, err, n_err,
      &hdr->status);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "listed_combine launch: %s", cudaGetErrorString(e));
  return PKX_OK;
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
  ListedMaps tm;
  if ((rc = make_maps(tm, a)) != PKX_OK) return rc;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  SharedParams p;
  p.kv_indptr = a.kv_indptr;
  p.group_indptr = a.group_indptr;
  p.shared_lens = a.shared_lens;
  p.batch = a.batch;
  p.num_groups = a.num_groups;
  p.hkv = a.hkv;
  p.tok = tokens_per_block(group);
  p.target = L.unit_target;
  p.unit_max = L.unit_max;
  p.gran_max = L.gran_max;
  p.seq = reinterpret_cast<int32_t *>(ws + L.seq_off);
  p.grp = reinterpret_cast<int32_t *>(ws + L.grp_off);
  p.units = reinterpret_cast<WorkUnit *>(ws + L.units_off);
  p.order = reinterpret_cast<int32_t *>(ws + L.order_off);
  p.rows = reinterpret_cast<ListedRow *>(ws + L.rows_off);
  p.hdr = reinterpret_cast<WsHeader *>(ws);
  cudaError_t e = launch_pdl(shared_sched_kernel, dim3(1), dim3(1024), 0, a.stream, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "shared_sched launch: %s", cudaGetErrorString(e));
  return run_listed(a, tm, L, nsm, a.kv_indptr, a.kv_indices, 2, 2 * a.hkv, nullptr, 0);
}

int launch_decode_pages(const ListedArgs &a) {
  const int nsm = num_sms_current_device();
  if (nsm <= 0) return set_error(PKX_ECUDA, "cannot query the current device");
  const int group = a.hq / a.hkv;
  const int64_t pairs = (int64_t)a.batch * a.hkv;
  if (pairs * a.top_k * a.page_size >= INT_MAX)
    return set_error(PKX_EUNSUPPORTED,
                     "decode_pages: batch * hkv * top_k * page_size must be below 2^31");
  const ListedLayout L = pages_layout(a.batch, a.hkv, group, a.d, a.page_size, a.top_k, nsm);
  int rc = check_workspace(a, L);
  if (rc != PKX_OK) return rc;
  ListedMaps tm;
  if ((rc = make_maps(tm, a)) != PKX_OK) return rc;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
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
  p.pieces = pages_pieces(a.batch, a.hkv, a.page_size, a.top_k, nsm);
  p.cap = a.top_k * a.page_size;
  p.slots = reinterpret_cast<int32_t *>(ws + L.idx_off);
  p.ptr = reinterpret_cast<int32_t *>(ws + L.ptr_off);
  p.err = reinterpret_cast<int32_t *>(ws + L.err_off);
  p.units = reinterpret_cast<WorkUnit *>(ws + L.units_off);
  p.order = reinterpret_cast<int32_t *>(ws + L.order_off);
  p.rows = reinterpret_cast<ListedRow *>(ws + L.rows_off);
  p.hdr = reinterpret_cast<WsHeader *>(ws);
  const size_t smem = sizeof(int) * ((size_t)a.top_k + 1);
  cudaError_t e = launch_pdl(list_pages_kernel, dim3((unsigned)pairs), dim3(256), smem, a.stream, p);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "list_pages launch: %s", cudaGetErrorString(e));
  return run_listed(a, tm, L, nsm, p.ptr, p.slots, 2 * p.pieces, 2, p.err, (int)pairs);
}

}  // namespace pkx
