// attention.cu -- extend and decode attention over a page-size-1 KV pool for
// sm_103a: a device-side work scheduler, a warp-specialised tcgen05/TMEM
// attention kernel whose K/V rows are gathered by cp.async copy warps, and
// the split-KV combine.
//
// Method (sglang extend_attention.py, _fwd_kernel_unified and
// extend_attention_fwd; flashinfer_backend.py, forward_decode):
//   for each query row and each visible key j:  s_j = sm_scale * <q, k_j>,
//   optionally s_j = cap * tanh(s_j / cap); visible iff j <= qpos (or, with a
//   custom mask, iff its mask byte is set) and, with a window W > 0,
//   qpos - j <= W; o = sum_j softmax(s)_j v_j (a sink logit per head joins
//   the denominator); lse = log sum exp s.  The online softmax keeps a
//   running max and sum per row and rescales the accumulator when the max
//   moves.
//
// GB300 design (differs from the pages' Triton kernel, which launches one
// program per (sequence, q head, 128-row block) and re-reads K/V per q head):
//  * a Q tile = 128 rows = (tokens x the Hq/Hkv query heads of one KV head),
//    and a CTA runs two Q tiles of consecutive tokens against each K/V tile:
//    K/V of a KV head are gathered once for 2 x 128 query rows;
//  * K and V rows are gathered from the pool by four warps with 16-byte
//    cp.async copies placed straight into the 128-byte-swizzled layout the
//    MMA descriptors read (random 256-byte rows need many copying threads
//    to reach HBM bandwidth; a TMA gather4 moves only four 128-byte rows
//    per instruction and stalls on its issue rate); each copying thread
//    arrives on the stage barrier when its own copies land.  An index warp
//    claims work units, resolves every tile's slot indices into a small smem
//    ring ahead of the copy warps and loads the Q tiles (3-D TMA boxes).
//    setmaxnreg moves registers from these warps to the softmax warpgroups;
//  * QK^T and PV are tcgen05.mma (M=128, bf16 in, fp32 accumulate in TMEM).
//    TMEM holds S and O of both Q tiles (4 x 128 columns).  The softmax
//    warpgroup of a tile writes P (bf16) back over its S columns and PV
//    reads A = P straight from TMEM.  While one warpgroup runs its softmax,
//    the tensor core runs the other tile's PV and QK^T;
//  * a unit with one Q tile (every decode unit; split extend units of at
//    most 128/G tokens) runs two key streams instead: the two warpgroups
//    take alternate K/V tiles with their own S/P and O, and the combine
//    merges the two partials;
//  * an fp8 pool (e4m3 / e5m2 codes with k_scale, v_scale) is staged as
//    codes and converted in place to exact bf16 (f16 for decode) by the
//    copy warps; the scales go into the logit scale and P (or the output);
//  * a 4-bit pool (extend only) is staged as codes with their block scales
//    and converted in place the same way;
//  * the KV loop stops at the causal diagonal and starts at the window edge
//    (the Triton kernel walks every tile and masks).  First tokens that stay
//    visible before a window come in front: a block's visible keys are then
//    numbered without the gap between them and the window, so that no tile is
//    spent on it (FIRST instantiations);
//  * a device-built work list (no host sync, graph-safe) splits long key
//    ranges across CTAs (split-KV); a combine kernel merges the partial
//    (o, lse) pairs with the merge_state formula;
//  * a persistent grid of one CTA per SM claims the work units in cost
//    order.
#include <algorithm>
#include <climits>
#include <cstdio>
#include <cstring>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "attn_kernel.cuh"
#include "fp4.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

// ============================================================ scheduler ====
struct SchedParams {
  int mode;
  const int32_t *qo_indptr, *kv_indptr, *prefix_lens;
  int batch, hkv, tok, window, num_q_tokens;
  int first;       // with a window: first tokens that stay visible (0: none)
  int head_minor;  // number a block's units of all KV heads one after another
  int bn;        // keys per K/V tile
  int q_tile_tok;  // query tokens of one Q tile
  int no_causal;   // a custom mask replaces the causal mask: blocks see every key
  int key_set;     // two-stage form only: kAllKeys, kPrefixKeys or kExtendKeys
  int keep_status; // leave the status word as an earlier pass left it
  int two_streams; // GQA kernel: decode units run two key streams, each with its own
                   // partial slot; split extend units of one query tile run two
                   // streams into the two halves of their slot
  int n_dsplit;  // units per (block, split): value-dim slices (1, or 4 for MLA)
  int unit_target, qb_max, unit_max, comb_max, slot_max;
  // Stream partition (parts > 0, a multiple of hkv): per KV head, the
  // blocks' key tiles laid end to end, each weighted by its block's Q tiles,
  // are cut into parts / hkv equal shares of that cost (the same cuts for
  // every head), a block is split at the first tile boundary of each share,
  // each piece is claimed by its share's CTA (or CTA pair), and
  // part_first[k] is the first claim position of share k (k <= parts).
  int parts;
  int32_t *part_first;
  int32_t *seq;  // 8 arrays of batch+1 ints
  int32_t *qbt;  // [6][qb_max]: tiles, sequence, unit / slot / combine offsets, tile offset per block
  int seq_in_smem, blk_in_smem;  // those arrays in dynamic shared memory instead
  WorkUnit *units;
  int32_t *uorder;  // units by cost, largest first
  CombineEntry *comb;
  WsHeader *hdr;
};

struct SeqDims {
  int P, E, T, qbase, nqb;
};

// Prefix length, extend length, key count and first query row of sequence b.
// Inconsistent values are recorded and the sequence is treated as empty.
__device__ SeqDims seq_dims(const SchedParams &p, int b) {
  SeqDims d;
  if (p.mode == kDecode) {
    d.T = p.kv_indptr[b + 1] - p.kv_indptr[b];
    d.E = 1;
    d.P = d.T - 1;
    d.qbase = b;
    if (d.T < 0 || p.kv_indptr[b] < 0) {
      record_status(&p.hdr->status, PKX_EDEVICE);
      d.T = 0;
      d.P = -1;
    }
    d.nqb = 1;
    return d;
  }
  d.qbase = p.qo_indptr[b];
  d.E = p.qo_indptr[b + 1] - d.qbase;
  if (p.mode == kTwoStage) {
    d.P = p.kv_indptr[b + 1] - p.kv_indptr[b];
    d.T = d.P + d.E;
    // One half of the ragged + paged split: the prefix keys alone (every
    // one visible to every extend query), or the extend keys alone with
    // causal positions counted from the first extend token.
    if (p.key_set == kPrefixKeys) d.T = d.P;
    else if (p.key_set == kExtendKeys) { d.P = 0; d.T = d.E; }
  } else {
    d.T = p.kv_indptr[b + 1] - p.kv_indptr[b];
    d.P = p.prefix_lens[b];
    if (d.P + d.E != d.T) record_status(&p.hdr->status, PKX_EDEVICE);
  }
  bool bad = d.E < 0 || d.P < 0 || d.T < 0 || d.qbase < 0 || p.kv_indptr[b] < 0 ||
             (long long)d.qbase + d.E > p.num_q_tokens;
  if (bad) {
    record_status(&p.hdr->status, PKX_EDEVICE);
    d.E = 0;
  }
  d.nqb = d.E > 0 ? (d.E + p.tok - 1) / p.tok : 0;
  return d;
}

// Key range [lo, hi) of query block qb of a sequence (key numbers where first
// tokens stay visible).
__device__ __forceinline__ void qblock_range(const SchedParams &p, const SeqDims &d, int qb,
                                             int &lo, int &hi, int &i0, int &i1) {
  i0 = qb * p.tok;
  i1 = min(d.E, i0 + p.tok);
  const int qmin = d.P + i0, qmax = d.P + i1 - 1;
  hi = p.no_causal ? d.T : min(qmax + 1, d.T);
  lo = p.window > 0 ? max(0, qmin - p.window) : 0;
  if (hi < lo) hi = lo;
  if (p.first > 0 && p.window > 0) {
    hi = key_number(hi, p.first, block_gap(qmin, p.window, p.first));
    lo = 0;
  }
}

// Number of K/V tiles of the key range [kb, ke) when tiles may not straddle
// `split` (the prefix / extend boundary of the two-stage form).
__device__ __forceinline__ int range_tiles(int kb, int ke, int split, int bn) {
  const int pe = min(ke, split), eb = max(kb, split);
  const int n_pre = pe > kb ? (pe - kb + bn - 1) / bn : 0;
  const int n_ext = ke > eb ? (ke - eb + bn - 1) / bn : 0;
  return n_pre + n_ext;
}

// Exclusive scan of one value per thread over the 1024-thread block (warp
// shuffles, then one warp over the 32 warp totals: three block barriers);
// the total goes to *total.  sh must hold 32 ints.
__device__ int block_scan_value(int v, int *sh, int &total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[wid] = x;
  __syncthreads();
  if (wid == 0) {
    int t = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    sh[lane] = t;
  }
  __syncthreads();
  const int excl = (wid ? sh[wid - 1] : 0) + x - v;
  total = sh[31];
  __syncthreads();  // sh may be reused by the caller
  return excl;
}

// Maximum of one value per thread over the 1024-thread block.
__device__ int block_max(int v, int *sh) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (lane == 0) sh[wid] = v;
  __syncthreads();
  int m = sh[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  __syncthreads();  // sh may be reused by the caller
  return m;
}

// Exclusive scan of in[0..n) into out[0..n) by the whole 1024-thread block
// (each thread a contiguous chunk); returns the total.  in and out may
// alias.
__device__ int block_exclusive_scan(const int32_t *in, int32_t *out, int n, int *sh) {
  const int tid = threadIdx.x;
  const int ch = (n + 1023) / 1024;
  const int beg = min(n, tid * ch), end = min(n, beg + ch);
  int local = 0;
  for (int i = beg; i < end; ++i) local += in[i];
  int total;
  int run = block_scan_value(local, sh, total);
  for (int i = beg; i < end; ++i) {
    int v = in[i];
    out[i] = run;
    run += v;
  }
  __syncthreads();
  return total;
}

// Buckets of the counting sorts (claim order, sequence ranks).
constexpr int kCostBuckets = 2048;
// Dynamic shared memory the scheduler may take: the histogram always, and
// the per-sequence and per-block arrays when they fit (else they live in
// the workspace, which is slower but has no size limit).
constexpr int kSchedSmemMax = 200 * 1024;
// Per-sequence and per-block arrays of the scheduler.
constexpr int kSchedSeqArrays = 5, kSchedBlockArrays = 6;

// Relative cost of a unit: its K/V tiles times its Q tiles, plus one for the
// per-unit prologue and epilogue (clamped to the sort's bucket range).
__device__ __forceinline__ int unit_cost(const WorkUnit &w, int q_tile_tok) {
  const int nq = (w.n_tok + q_tile_tok - 1) / q_tile_tok;
  return min(w.n_tiles * max(nq, 1) + 1, kCostBuckets - 1);
}

// Device-side work list.  Only the first phase reads global memory (the
// indptrs); the per-sequence and per-block values then live in shared memory
// (or, for very large batches, in the workspace), so the later phases are
// throughput-bound rather than chains of dependent global loads.
//   1. per sequence: P, E, T, first query row and query blocks; a scan gives
//      each sequence's first block;
//   2. per query block (of one KV head): its K/V tiles; their total sets the
//      split-KV chunk C;
//   3. per block: units (splits x value slices), partial slots and combine
//      entries, and their offsets (scans);
//   4-6. combine entries; every unit written and counted by its claim key
//      (its cost, largest first), then placed in the claim order.
// Largest first balances the CTAs, which claim units at run time.  (Orders
// that keep a sequence's units together cut DRAM re-reads of K/V but cost
// more in balance than they save: the kernel is not bound by DRAM.)
__global__ void __launch_bounds__(1024, 1) sched_kernel(SchedParams p) {
  extern __shared__ int sdyn[];
  __shared__ int sh[32];
  __shared__ int s_c, s_share;
  const int tid = threadIdx.x;
  const int B = p.batch;
  const int S1 = B + 1;
  int *hist = sdyn;
  int *seqa = p.seq_in_smem ? sdyn + kCostBuckets : p.seq;
  int *sP = seqa, *sE = seqa + S1, *sT = seqa + 2 * S1, *sQ0 = seqa + 3 * S1;
  int *sOff = seqa + 4 * S1;   // first query block of each sequence; [B] = total
  int *blk = p.blk_in_smem ? sdyn + kCostBuckets + (p.seq_in_smem ? kSchedSeqArrays * S1 : 0)
                           : p.qbt;
  int *bNt = blk, *bSeq = blk + p.qb_max, *bUo = blk + 2 * p.qb_max;
  int *bSo = blk + 3 * p.qb_max, *bCo = blk + 4 * p.qb_max;
  int *bTo = blk + 5 * p.qb_max;  // stream partition: first tile of the block in the stream

  grid_dep_wait();    // inputs written by the previous kernel on the stream
  grid_dep_launch();  // the attention grid may start its prologue now
  if (tid == 0) {
    if (!p.keep_status) p.hdr->status = 0;
    p.hdr->next_unit = 0;
  }

  // 1. per sequence
  for (int b = tid; b < B; b += 1024) {
    const SeqDims d = seq_dims(p, b);
    sP[b] = d.P;
    sE[b] = d.E;
    sT[b] = d.T;
    sQ0[b] = d.qbase;
    sOff[b] = d.nqb;
  }
  __syncthreads();
  const int total_qb = block_exclusive_scan(sOff, sOff, B, sh);
  if (tid == 0) sOff[B] = total_qb;
  if (total_qb >= p.qb_max) {  // cannot happen for consistent indptrs (one entry spare)
    if (tid == 0) {
      record_status(&p.hdr->status, PKX_EDEVICE);
      p.hdr->n_units = 0;
      p.hdr->n_combine = 0;
    }
    return;
  }
  __syncthreads();
  auto dims = [&](int b) {
    SeqDims d;
    d.P = sP[b];
    d.E = sE[b];
    d.T = sT[b];
    d.qbase = sQ0[b];
    d.nqb = sOff[b + 1] - sOff[b];
    return d;
  };
  // the sequence of query block qb: the last b with sOff[b] <= qb
  auto seq_of = [&](int qb) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sOff[mid] <= qb) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };

  // 2. K/V tiles per query block; total tiles -> chunk size C
  int my_tiles = 0;
  for (int qb = tid; qb < total_qb; qb += 1024) {
    const int b = seq_of(qb);
    const SeqDims d = dims(b);
    int lo, hi, i0, i1;
    qblock_range(p, d, qb - sOff[b], lo, hi, i0, i1);
    const int nt = (hi - lo + p.bn - 1) / p.bn;
    bNt[qb] = nt;
    bSeq[qb] = b;
    my_tiles = min(my_tiles + nt, 0x1fffff);
    // stream partition: the block's cost, its tiles times its Q tiles
    if (p.parts > 0) bTo[qb] = nt * max(1, (i1 - i0 + p.q_tile_tok - 1) / p.q_tile_tok);
  }
  int tiles_all;
  block_scan_value(my_tiles, sh, tiles_all);
  const bool stream = p.parts > 0;
  int cost_all = 0;
  if (stream) {
    __syncthreads();
    cost_all = block_exclusive_scan(bTo, bTo, total_qb, sh);  // first cost of each block
    if (tid == 0) bTo[total_qb] = cost_all;
  }
  if (tid == 0) {
    const long long total_tiles = (long long)tiles_all * p.hkv * p.n_dsplit;
    const long long c = (total_tiles + p.unit_target - 1) / p.unit_target;
    s_c = (int)max((long long)kMinSplitTiles, c);
    const int ppk = stream ? p.parts / p.hkv : 1;  // shares per KV head
    // at least two, the largest tile cost, so that every share holds a tile
    // boundary and no piece is empty
    s_share = stream ? max(2, (cost_all + ppk - 1) / ppk) : 0;
    p.hdr->split_tiles = stream ? s_share : s_c;
  }
  __syncthreads();
  const int C = s_c, share = s_share;

  // 3. per query block: units, slots, combine entries; their offsets
  const int nd = p.n_dsplit;
  // splits of block qb: chunks of C tiles, or (stream partition) one piece
  // per share its tiles touch
  auto splits = [&](int qb) {
    const int nt = bNt[qb];
    if (nt <= 0) return 1;
    if (!stream) return (nt + C - 1) / C;
    // a tile belongs to the share its first cost falls in
    const int g0 = bTo[qb], wq = (bTo[qb + 1] - g0) / nt;
    return (g0 + (nt - 1) * wq) / share - g0 / share + 1;
  };
  // two key streams: every decode unit has two partial slots and every
  // block a combine entry
  const bool dec2 = p.two_streams && p.mode == kDecode;
  const int spu = dec2 ? 2 : 1;
  auto combined = [&](int S) { return S > 1 || dec2; };
  const int chunk = (total_qb + 1023) / 1024;
  const int qb_beg = min(total_qb, tid * chunk), qb_end = min(total_qb, qb_beg + chunk);
  int lu = 0, ls = 0, lc = 0;
  for (int qb = qb_beg; qb < qb_end; ++qb) {
    const int S = splits(qb);
    lu += S * nd;
    if (combined(S)) {
      ls += S * spu;
      lc += 1;
    }
  }
  int tu, ts, tcm;
  int u0 = block_scan_value(lu, sh, tu);
  int s0 = block_scan_value(ls, sh, ts);
  int c0 = block_scan_value(lc, sh, tcm);
  for (int qb = qb_beg; qb < qb_end; ++qb) {
    bUo[qb] = u0;
    bSo[qb] = s0;
    bCo[qb] = c0;
    const int S = splits(qb);
    u0 += S * nd;
    if (combined(S)) {
      s0 += S * spu;
      c0 += 1;
    }
  }
  const long long n_units_l = (long long)tu * p.hkv, n_slots_l = (long long)ts * p.hkv,
                  n_comb_l = (long long)tcm * p.hkv;
  if (n_units_l > p.unit_max || n_slots_l > p.slot_max || n_comb_l > p.comb_max) {
    if (tid == 0) {
      record_status(&p.hdr->status, PKX_EDEVICE);
      p.hdr->n_units = 0;
      p.hdr->n_combine = 0;
    }
    return;
  }
  const int n_units = (int)n_units_l, n_comb = (int)n_comb_l;

  // 4. claim keys: the unit's cost, largest first
  for (int i = tid; i < kCostBuckets; i += 1024) hist[i] = 0;
  __syncthreads();
  auto claim_key = [&](const WorkUnit &w) { return kCostBuckets - 1 - unit_cost(w, p.q_tile_tok); };

  // 5. combine entries, one (KV head, query block) pair per thread
  const int n_pairs = p.hkv * total_qb;
  for (int idx = tid; idx < n_pairs; idx += 1024) {
    const int kvh = idx / total_qb, qb = idx - kvh * total_qb;
    const int S = splits(qb);
    if (!combined(S)) continue;
    const int b = bSeq[qb];
    const SeqDims d = dims(b);
    int lo, hi, i0, i1;
    qblock_range(p, d, qb - sOff[b], lo, hi, i0, i1);
    CombineEntry e;
    e.q_tok0 = d.qbase + i0;
    e.n_tok = i1 - i0;
    e.kvh = kvh;
    e.slot0 = kvh * ts + bSo[qb];
    e.n_split = S * spu;
    // a split extend block of one query tile: its units' second stream
    // fills the second half of each slot
    e.pad[0] = p.two_streams && p.mode != kDecode && S > 1 && i1 - i0 <= p.q_tile_tok ? 2 : 1;
    e.pad[1] = e.pad[2] = 0;
    p.comb[kvh * tcm + bCo[qb]] = e;
  }
  // Unit u: KV head u / tu; within the head, query block qb is the last
  // block with bUo[qb] <= rest, and the unit is its (split, value slice)
  // number rest - bUo[qb].
  auto unit_at = [&](int u) {
    // (head_minor: unit u is of KV head u % hkv, so that the heads' units of a
    // block are claimed close together)
    const int kvh = p.head_minor ? u % p.hkv : u / tu;
    const int rest = p.head_minor ? u / p.hkv : u - kvh * tu;
    int lo_b = 0, hi_b = total_qb - 1;
    while (lo_b < hi_b) {
      const int mid = (lo_b + hi_b + 1) >> 1;
      if (bUo[mid] <= rest) lo_b = mid;
      else hi_b = mid - 1;
    }
    const int qb = lo_b, k = rest - bUo[qb];
    const int sp = k / nd, dq = k - sp * nd;
    const int b = bSeq[qb];
    const SeqDims d = dims(b);
    int lo, hi, i0, i1;
    qblock_range(p, d, qb - sOff[b], lo, hi, i0, i1);
    const int split_at = p.mode != kTwoStage ? INT_MAX
                         : p.first > 0 ? key_number(d.P, p.first, block_gap(d.P + i0, p.window, p.first))
                                       : d.P;
    const int nt = bNt[qb], S = splits(qb);
    // split sp covers tiles [sp nt / S, (sp + 1) nt / S) (sizes differ by
    // one at most), or (stream partition) the block's tiles inside share
    // g0 / share + sp
    int t0 = (int)((long long)sp * nt / S), t1 = (int)((long long)(sp + 1) * nt / S);
    int part = 0;
    if (stream) {
      // share k of the head takes the block's tiles whose first cost lies
      // in [k share, (k + 1) share); a tile costs wq (the block's Q tiles),
      // at most share, so every share between the first and the last tile's
      // holds a tile
      const int g0 = bTo[qb], ppk = p.parts / p.hkv;
      const int wq = nt > 0 ? (bTo[qb + 1] - g0) / nt : 1;
      const int k = min(g0 / share + sp, ppk - 1);  // the share within the head
      t0 = sp == 0 ? 0 : min(nt, (k * share - g0 + wq - 1) / wq);
      t1 = sp == S - 1 ? nt : min(nt, ((k + 1) * share - g0 + wq - 1) / wq);
      part = kvh * ppk + k;
    }
    WorkUnit w;
    w.q_tok0 = d.qbase + i0;
    w.n_tok = i1 - i0;
    w.qpos0 = d.P + i0;
    w.kvh = kvh;
    w.k_begin = min(hi, lo + t0 * p.bn);
    w.k_end = min(hi, lo + t1 * p.bn);
    w.k_split = split_at;
    w.n_tiles = range_tiles(w.k_begin, w.k_end, split_at, p.bn);
    w.b = b;
    w.slot = combined(S) ? kvh * ts + bSo[qb] + sp * spu : -1;
    w.dq = dq;
    w.claim = stream ? part : 0;
    return w;
  };

  // 6. units, consecutive threads on consecutive units (their records go
  //    out as 16-byte stores); pass 0 builds and writes them with their
  //    claim keys and counts the keys, pass 1 reads the keys back and places
  //    the units in the claim order.  Lanes of a warp whose units share a
  //    key make one atomic for the group (units of one sequence and cost
  //    class share a key, so per-unit atomics serialise).
  const int lane = tid & 31;
  for (int pass = 0; pass < 2; ++pass) {
    for (int base = tid - lane; base < n_units; base += 1024) {
      const int u = base + lane;
      const bool act = u < n_units;
      WorkUnit w;
      int key = -1;
      if (act) {
        if (pass == 0) {
          w = unit_at(u);
          key = stream ? w.claim : claim_key(w);  // stream partition: the share, in order
          w.claim = key;
        } else {
          key = p.units[u].claim;  // written in pass 0 (the block barrier between passes orders it)
        }
      }
      const unsigned grp = __match_any_sync(0xffffffffu, key);
      const int leader = __ffs(grp) - 1;
      int first = 0;
      if (act && lane == leader) first = atomicAdd(&hist[key], __popc(grp));
      first = __shfl_sync(0xffffffffu, first, leader);
      if (act) {
        if (pass == 0) p.units[u] = w;
        else p.uorder[first + __popc(grp & ((1u << lane) - 1u))] = u;
      }
    }
    __syncthreads();
    if (pass == 0) {
      block_exclusive_scan(hist, hist, kCostBuckets, sh);
      // each share's first claim position (keys are shares, all below parts)
      if (stream)
        for (int k = tid; k <= p.parts; k += 1024) p.part_first[k] = hist[k];
    }
  }
  if (tid == 0) {
    p.hdr->n_units = n_units;
    p.hdr->n_combine = n_comb;
  }
}

// ================================================================== MLA ====
#include "mla_pair_kernel.cuh"

// ============================================================== combine ====
// Merge the split-KV partials of every split query block: with lse_i the
// partial log-sum-exps and o_i the partial (normalised) outputs,
//   lse = log sum_i exp(lse_i),  o = sum_i exp(lse_i - lse) o_i
// (the merge_state formula applied n ways).
__global__ void __launch_bounds__(256) combine_kernel(const WsHeader *hdr, const CombineEntry *ce,
                                                      const float *__restrict__ plse,
                                                      const float *__restrict__ po,
                                                      bf16 *__restrict__ o, float *__restrict__ lse,
                                                      const float *sinks, int hq, int group,
                                                      int hdv, int rows_per_slot) {
  grid_dep_wait();  // the attention kernel's partials
  const int n_comb = hdr->n_combine;
  const int lane = threadIdx.x & 31;
  const int gw = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int nw = (gridDim.x * blockDim.x) >> 5;
  for (int64_t idx = gw; idx < (int64_t)n_comb * rows_per_slot; idx += nw) {
    const int e = (int)(idx / rows_per_slot), r = (int)(idx % rows_per_slot);
    const CombineEntry E = ce[e];
    if (r >= E.n_tok * group) continue;
    // partial i: slot slot0 + i / halves, half i % halves (halves = 2 when
    // the block's two key streams share each slot)
    const int halves = E.pad[0] == 2 ? 2 : 1, n_part = E.n_split * halves;
    auto prow = [&](int i) {
      return (int64_t)(E.slot0 + i / halves) * rows_per_slot + (i % halves) * (rows_per_slot / 2) +
             r;
    };
    float mx = -INFINITY;
    bool empty = true;  // every partial is -inf (fmaxf drops a NaN one)
    for (int i = 0; i < n_part; ++i) {
      const float x = plse[prow(i)];
      mx = fmaxf(mx, x);
      empty &= x == -INFINITY;
    }
    const int t = r / group, g = r - t * group;
    const int64_t orow = (int64_t)(E.q_tok0 + t) * hq + E.kvh * group + g;
    // a sink (natural-log logit of the head) joins the denominator once
    const float sink = sinks ? __ldg(sinks + E.kvh * group + g) : -INFINITY;
    mx = fmaxf(mx, sink);
    if (empty) {
      for (int c = lane * 4; c < hdv; c += 128)
        *reinterpret_cast<uint2 *>(o + orow * hdv + c) = make_uint2(0, 0);
      if (lane == 0 && lse) lse[orow] = sink;  // -inf without a sink
      continue;
    }
    float wsum = sinks ? exp2f((sink - mx) * 1.4426950408889634f) : 0.f;
    for (int i = 0; i < n_part; ++i) wsum += exp2f((plse[prow(i)] - mx) * 1.4426950408889634f);
    const float inv = 1.0f / wsum;
    // every lane takes 4 consecutive value dims of each 128-dim pass (at
    // most four passes: Lv <= 512); a partial's loads for all passes go out
    // together, and the row is stored once every partial is added
    constexpr int kPasses = 4;
    float acc[kPasses][4] = {};
    for (int i = 0; i < n_part; ++i) {
      const int64_t sr = prow(i);
      const float wi = exp2f((plse[sr] - mx) * 1.4426950408889634f) * inv;
      const float *src = po + sr * hdv + lane * 4;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        if (k * 128 + lane * 4 < hdv) {
          const float4 a = *reinterpret_cast<const float4 *>(src + k * 128);
          acc[k][0] += wi * a.x; acc[k][1] += wi * a.y; acc[k][2] += wi * a.z; acc[k][3] += wi * a.w;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int c = k * 128 + lane * 4;
      if (c < hdv)
        *reinterpret_cast<uint2 *>(o + orow * hdv + c) =
            make_uint2(pack_bf16(acc[k][0], acc[k][1]), pack_bf16(acc[k][2], acc[k][3]));
    }
    if (lane == 0 && lse) lse[orow] = mx + logf(wsum);
  }
}

// ================================================================= host ====
int num_sms_current_device() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

int tokens_per_block(int group) { return group >= 1 && group <= kBlockM ? kBlockM / group : 0; }

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Rows of one split-KV partial slot: both Q tiles of an extend block, or the
// group's rows of a decode query.
bool split_head_dims(int lq, int lv) { return (lq == 192 && lv == 128) || (lq == 288 && lv == 256); }

int q_tiles_per_unit(int lq, int lv) {
  return (lq == 576 && lv == 512) || split_head_dims(lq, lv) ? 1 : 2;
}

int rows_per_slot(bool decode, int group, int nqt) {
  return decode ? group : nqt * tokens_per_block(group) * group;
}

WsLayout ws_layout(int batch, int num_q_tokens, int hkv, int group, int lq, int lv, int num_sms,
                   bool decode, bool two_streams) {
  WsLayout L{};
  const bool mla = lq == 576 && lv == 512;
  // tokens of a query block: two Q tiles (GQA kernel, Lq = Lv <= 128) or one
  // (MLA kernel, split head dims)
  const int nqt = q_tiles_per_unit(lq, lv);
  const int tok = nqt * tokens_per_block(group);
  L.unit_target = 4 * (num_sms > 0 ? num_sms : 160);
  L.qb_max = (tok > 0 ? (num_q_tokens + tok - 1) / tok : 0) + batch + 1;
  L.unit_max = (L.unit_target + hkv * L.qb_max) * (mla ? 4 : 1);
  L.slot_max = 2 * L.unit_target;
  L.comb_max = L.unit_target;
  if (decode && !mla && !split_head_dims(lq, lv) && two_streams) {
    // two key streams per unit: two partial slots per unit, a combine entry
    // per (query block, KV head)
    L.slot_max = 2 * L.unit_max;
    L.comb_max = L.unit_target + hkv * L.qb_max;
  }
  L.rows_per_slot = rows_per_slot(decode, group, nqt);
  size_t off = align256(sizeof(WsHeader));
  L.seq_off = off;
  off = align256(off + sizeof(int32_t) * 8 * (size_t)(batch + 1));
  L.qb_off = off;
  off = align256(off + sizeof(int32_t) * kSchedBlockArrays * (size_t)L.qb_max);
  L.part_off = off;
  off = align256(off + sizeof(int32_t) * (size_t)(kMaxStreamParts + 1));
  L.units_off = off;
  off = align256(off + sizeof(WorkUnit) * (size_t)L.unit_max);
  L.uorder_off = off;
  off = align256(off + sizeof(int32_t) * (size_t)L.unit_max);
  L.comb_off = off;
  off = align256(off + sizeof(CombineEntry) * (size_t)L.comb_max);
  L.plse_off = off;
  off = align256(off + sizeof(float) * (size_t)L.slot_max * L.rows_per_slot);
  L.po_off = off;
  off = align256(off + sizeof(float) * (size_t)L.slot_max * L.rows_per_slot * lv);
  L.total = off;
  return L;
}

// cuTensorMapEncodeTiled from the driver, kept once it is found.
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_acquire);
  if (!fn) {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
      known.store(fn, std::memory_order_release);
    }
  }
  return fn;
}

// 3-D map over q [n, hq, lq]: box = 64 dims x G heads x tok tokens.
int make_q_map(CUtensorMap *m, const void *q, int64_t n, int hq, int lq, int G, int tok) {
  auto fn = encode_fn();
  if (!fn) return set_error(PKX_ECUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[3] = {(cuuint64_t)lq, (cuuint64_t)hq, (cuuint64_t)n};
  cuuint64_t strides[2] = {(cuuint64_t)lq * 2, (cuuint64_t)hq * lq * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tok};
  cuuint32_t es[3] = {1, 1, 1};
  auto encode = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // a thread's first CUDA call: the runtime binds the device's context to a
    // thread when a call needs it, the driver's own call does not
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  }
  if (r != CUDA_SUCCESS) return set_error(PKX_EINVAL, "q tensor map rejected: %d", (int)r);
  return PKX_OK;
}

// The three key modes of one head size over an fp8 pool (the two extend
// forms with or without a custom mask).
template <int HD, int FMT>
static int launch_attn_fp8(int mode, bool masked, const TMaps &tmaps, const KParams &kp,
                           int grid, cudaStream_t s) {
  if (mode == kTwoStage)
    return masked ? launch_attn_kernel<HD, kTwoStage, true, FMT>(tmaps, kp, grid, s)
                  : launch_attn_kernel<HD, kTwoStage, false, FMT>(tmaps, kp, grid, s);
  if (mode == kUnified)
    return masked ? launch_attn_kernel<HD, kUnified, true, FMT>(tmaps, kp, grid, s)
                  : launch_attn_kernel<HD, kUnified, false, FMT>(tmaps, kp, grid, s);
  return launch_attn_kernel<HD, kDecode, false, FMT>(tmaps, kp, grid, s);
}

// Two-stage extend over a 4-bit pool, and the two forms with first tokens that
// stay visible over a bf16 pool (Lq = Lv, one head size).
template <int HD>
static int launch_attn_fp4(bool masked, bool first, const TMaps &tmaps, const KParams &kp, int grid,
                           cudaStream_t s) {
  if (masked) return launch_attn_kernel<HD, kTwoStage, true, kKvFp4>(tmaps, kp, grid, s);
  return first ? launch_attn_kernel<HD, kTwoStage, false, kKvFp4, true>(tmaps, kp, grid, s)
               : launch_attn_kernel<HD, kTwoStage, false, kKvFp4>(tmaps, kp, grid, s);
}
template <int HD>
static int launch_attn_first(int mode, const TMaps &tmaps, const KParams &kp, int grid,
                             cudaStream_t s) {
  return mode == kDecode ? launch_attn_kernel<HD, kDecode, false, 0, true>(tmaps, kp, grid, s)
                         : launch_attn_kernel<HD, kTwoStage, false, 0, true>(tmaps, kp, grid, s);
}

// Pair kernel launch: clusters of two CTAs, programmatic dependent launch.
template <int MODE, bool MASK, int FMT = 0, bool SG = false>
static cudaError_t launch_pair(int pairs, cudaStream_t s, const KParams &kp, bool query_only,
                               int *max_pairs) {
  using C = std::conditional_t<SG, std::conditional_t<FMT != 0, MlaPairDec8Cfg, MlaPairDecCfg>,
                               MlaPairCfg>;
  static PerDevice configured;
  if (needs_config(configured)) {
    cudaError_t e = cudaFuncSetAttribute(mla_pair_kernel<MODE, MASK, FMT, SG>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    mark_configured(configured);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = query_only ? 1 : 2;
  if (query_only)
    return cudaOccupancyMaxActiveClusters(max_pairs, mla_pair_kernel<MODE, MASK, FMT, SG>, &cfg);
  return cudaLaunchKernelEx(&cfg, mla_pair_kernel<MODE, MASK, FMT, SG>, kp);
}

// CTA pairs of the MLA kernel that run at once on the current device (an SM
// group with an odd count of free SMs leaves one idle), queried once per
// device; 0 on error.
static int mla_pairs(int nsm) {
  static PerDevice known;
  std::atomic<int> *here = known.here();
  int n = here ? here->load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (launch_pair<kUnified, false>(nsm / 2, nullptr, KParams{}, true, &n) != cudaSuccess) {
    set_error(PKX_ECUDA, "cudaOccupancyMaxActiveClusters(mla_pair_kernel) failed");
    return 0;
  }
  n = std::min(n, nsm / 2);
  if (here && n > 0) here->store(n, std::memory_order_relaxed);
  return n;
}

template <int MODE, bool MASK = false, int FMT = 0>
static int launch_mla_pair(const KParams &kp, int pairs, cudaStream_t s) {
  cudaError_t e;
  if constexpr (MODE == kDecode && !MASK) {
    // decode of at most 32 rows per unit: the five-stage layout
    e = kp.group <= MlaPairDecCfg::XR ? launch_pair<MODE, false, FMT, true>(pairs, s, kp, false, nullptr)
                                      : launch_pair<MODE, false, FMT>(pairs, s, kp, false, nullptr);
  } else {
    e = launch_pair<MODE, MASK, FMT>(pairs, s, kp, false, nullptr);
  }
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "mla_pair_kernel launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

int launch_attention(const AttnArgs &a) {
  const int group = a.hq / a.hkv;
  const int nsm = num_sms_current_device();
  if (nsm <= 0) return set_error(PKX_ECUDA, "cannot query the current device");
  const bool decode = a.mode == kDecode;
  const bool mla = a.lq == 576 && a.lv == 512;
  const int nq = decode ? a.batch : a.num_q_tokens;
  const bool split = split_head_dims(a.lq, a.lv);
  WsLayout L = ws_layout(a.batch, nq, a.hkv, group, a.lq, a.lv, nsm, decode);
  // Decode runs two key streams when the workspace holds their partial
  // slots (pkx_decode_workspace_size asks for that), else one stream.  The
  // MLA kernel and the split head dims run one stream.
  bool dec_two = decode && !mla && !split;
  if (dec_two && a.workspace_bytes < L.total) {
    const WsLayout L1 = ws_layout(a.batch, nq, a.hkv, group, a.lq, a.lv, nsm, decode, false);
    if (a.workspace_bytes >= L1.total) {
      L = L1;
      dec_two = false;
    }
  }
  if (mla) {
    // V must be the first 512 dims of each K row (the MLA layout).
    const bool pool_alias = a.v_buf == a.k_buf && a.vb_ss == a.kb_ss && a.vb_sh == a.kb_sh;
    const bool ext_alias = a.mode != kTwoStage ||
                           (a.v_ext == a.k_ext && a.ve_st == a.ke_st && a.ve_sh == a.ke_sh);
    if (!pool_alias || !ext_alias)
      return set_error(PKX_EUNSUPPORTED,
                       "Lq=576/Lv=512 needs V to be the first 512 dims of each K row");
  }
  // the MLA kernel runs on CTA pairs: units for four rounds of the pairs
  int pairs = 0;
  if (mla) {
    pairs = mla_pairs(nsm);
    if (pairs <= 0) return set_error(PKX_ECUDA, "no CTA pair of the MLA kernel fits the device");
  }
  if (a.workspace == nullptr || a.workspace_bytes < L.total)
    return set_error(PKX_EWORKSPACE, "workspace of %zu bytes given, %zu needed",
                     a.workspace_bytes, L.total);
  if (reinterpret_cast<uintptr_t>(a.workspace) & 255)
    return set_error(PKX_EINVAL, "workspace must be 256-byte aligned");
  if (a.num_slots >= (int64_t)INT_MAX)
    return set_error(PKX_EUNSUPPORTED, "more than 2^31 pool slots");
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  WsHeader *hdr = reinterpret_cast<WsHeader *>(ws);
  const int tok = tokens_per_block(group);

  // tensor maps
  TMaps tm;
  memset(&tm, 0, sizeof tm);
  int rc = PKX_OK;
  if (!mla && (rc = make_q_map(&tm.q, a.q, nq, a.hq, a.lq, group, decode ? 1 : tok)) != PKX_OK)
    return rc;

  SchedParams sp;
  sp.mode = a.mode;
  sp.qo_indptr = a.qo_indptr;
  sp.kv_indptr = a.kv_indptr;
  sp.prefix_lens = a.prefix_lens;
  sp.batch = a.batch;
  sp.hkv = a.hkv;
  sp.tok = q_tiles_per_unit(a.lq, a.lv) * tok;
  sp.bn = mla ? MlaPairCfg::BN : kBlockN;
  sp.q_tile_tok = tok > 0 ? tok : 1;
  sp.no_causal = a.custom_mask != nullptr;
  sp.key_set = a.mode == kTwoStage ? a.key_set : kAllKeys;
  sp.keep_status = a.keep_status;
  sp.two_streams = !mla && !split && (!decode || dec_two);
  sp.n_dsplit = 1;
  sp.window = a.window;
  sp.first = a.window > 0 ? a.first_tokens : 0;
  // a 4-bit row is 64 bytes, and four heads' block scales share a DRAM sector
  sp.head_minor = a.kv_fmt == kKvFp4;
  sp.num_q_tokens = nq;
  sp.unit_target = mla ? 4 * pairs : L.unit_target;
  // MLA decode with one KV head: a stream partition, one share of the key
  // tiles per CTA pair (equal shares, where run-time claims of equal units
  // leave some pairs one unit more than others)
  // GQA decode over a bf16 pool: one share per CTA, nsm / hkv per KV head
  // (over an fp8 pool the conversion-bound pipeline does better with the
  // run-time claims of smaller units: 0.48 against 0.54 ms on decode_gqa)
  const bool stream =
      decode && (mla ? a.hkv == 1 && pairs <= kMaxStreamParts
                     : !split && a.kv_fmt == kKvBf16 && nsm <= kMaxStreamParts &&
                           nsm % a.hkv == 0);
  sp.parts = stream ? (mla ? pairs : nsm) : 0;
  sp.part_first = reinterpret_cast<int32_t *>(ws + L.part_off);
  sp.qb_max = L.qb_max;
  sp.unit_max = L.unit_max;
  sp.comb_max = L.comb_max;
  sp.slot_max = L.slot_max;
  sp.seq = reinterpret_cast<int32_t *>(ws + L.seq_off);
  sp.qbt = reinterpret_cast<int32_t *>(ws + L.qb_off);
  sp.units = reinterpret_cast<WorkUnit *>(ws + L.units_off);
  sp.uorder = reinterpret_cast<int32_t *>(ws + L.uorder_off);
  sp.comb = reinterpret_cast<CombineEntry *>(ws + L.comb_off);
  sp.hdr = hdr;
  size_t sched_smem = kCostBuckets * sizeof(int);
  {
    const size_t seq_b = (size_t)kSchedSeqArrays * (a.batch + 1) * sizeof(int);
    const size_t blk_b = (size_t)kSchedBlockArrays * L.qb_max * sizeof(int);
    sp.seq_in_smem = sched_smem + seq_b <= (size_t)kSchedSmemMax;
    if (sp.seq_in_smem) sched_smem += seq_b;
    sp.blk_in_smem = sched_smem + blk_b <= (size_t)kSchedSmemMax;
    if (sp.blk_in_smem) sched_smem += blk_b;
    static PerDevice configured;
    if (needs_config(configured)) {
      cudaError_t e = cudaFuncSetAttribute(sched_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kSchedSmemMax);
      if (e != cudaSuccess)
        return set_error(PKX_ECUDA, "cudaFuncSetAttribute(sched_kernel): %s", cudaGetErrorString(e));
      mark_configured(configured);
    }
  }
  {
    cudaError_t e = launch_pdl(sched_kernel, dim3(1), dim3(1024), sched_smem, a.stream, sp);
    if (e != cudaSuccess)
      return set_error(PKX_ECUDA, "sched_kernel launch: %s", cudaGetErrorString(e));
  }

  KParams kp;
  kp.q = static_cast<const bf16 *>(a.q);
  kp.o = static_cast<bf16 *>(a.o);
  kp.lse = a.lse;
  kp.k_pool = static_cast<const bf16 *>(a.k_buf);
  kp.v_pool = static_cast<const bf16 *>(a.v_buf);
  kp.k_ext = static_cast<const bf16 *>(a.mode == kTwoStage ? a.k_ext : a.k_buf);
  kp.v_ext = static_cast<const bf16 *>(a.mode == kTwoStage ? a.v_ext : a.v_buf);
  kp.kb_ss = a.kb_ss;
  kp.vb_ss = a.vb_ss;
  kp.ke_st = a.ke_st;
  kp.ve_st = a.ve_st;
  kp.kb_sh = a.kb_sh;
  kp.vb_sh = a.vb_sh;
  kp.ke_sh = a.ke_sh;
  kp.ve_sh = a.ve_sh;
  kp.num_slots = a.num_slots;
  kp.qo_indptr = a.qo_indptr;
  kp.kv_indptr = a.kv_indptr;
  kp.kv_indices = a.kv_indices;
  kp.hq = a.hq;
  kp.group = group;
  kp.tok = tok;
  kp.q_box_tok = decode ? 1 : tok;
  kp.window = a.window;
  kp.first = sp.first;
  kp.k_bs = static_cast<const uint8_t *>(a.k_bscale);
  kp.v_bs = static_cast<const uint8_t *>(a.v_bscale);
  kp.kbs_ss = a.kbs_ss; kp.kbs_sh = a.kbs_sh; kp.vbs_ss = a.vbs_ss; kp.vbs_sh = a.vbs_sh;
  kp.rows_per_slot = L.rows_per_slot;
  const float log2e = 1.4426950408889634f;
  const float sm_scale = a.sm_scale > 0.f ? a.sm_scale : 1.0f / sqrtf((float)a.lq);
  kp.use_cap = a.logit_cap > 0.f;
  kp.scale_log2 = sm_scale * log2e;
  kp.cap_pre = kp.use_cap ? sm_scale / a.logit_cap : 0.f;
  kp.cap_log2 = kp.use_cap ? a.logit_cap * log2e : 0.f;
  kp.scale_log2_k = kp.scale_log2 * a.k_scale;
  if (sp.first > 0 || a.kv_fmt == kKvFp4) {  // never 0: a hidden logit is -inf before its scale
    kp.scale_log2 = std::max(kp.scale_log2, 1e-37f);
    kp.scale_log2_k = std::max(kp.scale_log2_k, 1e-37f);
  }
  kp.cap_pre_k = kp.cap_pre * a.k_scale;
  kp.custom_mask = a.custom_mask;
  kp.mask_indptr = a.mask_indptr;
  kp.sinks = a.sinks;
  kp.dec_two = dec_two ? 1 : 0;
  kp.log2_v_scale = log2f(a.v_scale);
  kp.v_scale = a.v_scale;
  kp.inv_v_scale = 1.0f / a.v_scale;
  kp.prefix_lens = a.prefix_lens;
  kp.units = sp.units;
  kp.uorder = sp.uorder;
  kp.next_unit = &hdr->next_unit;
  kp.part_first = stream ? sp.part_first : nullptr;
  kp.hdr = hdr;
  kp.status = &hdr->status;
  kp.plse = reinterpret_cast<float *>(ws + L.plse_off);
  kp.po = reinterpret_cast<float *>(ws + L.po_off);
  wait_settings(&kp.wait_ns, &kp.stall);
  kp.cache_loc = a.cache_loc;
  kp.k_pool_w = static_cast<bf16 *>(const_cast<void *>(a.k_buf));
  kp.v_pool_w = static_cast<bf16 *>(const_cast<void *>(a.v_buf));

  const int grid = nsm;
  cudaEvent_t ev_before = nullptr, ev_after = nullptr;
  attention_events(&ev_before, &ev_after);
  if (ev_before) cudaEventRecord(ev_before, a.stream);
  const bool masked = a.custom_mask != nullptr;
  if (a.kv_fmt == kKvFp4) {  // Lq = Lv = 64 or 128, two-stage (the entry point checks)
    rc = a.lq == 128 ? launch_attn_fp4<128>(masked, sp.first > 0, tm, kp, grid, a.stream)
                     : launch_attn_fp4<64>(masked, sp.first > 0, tm, kp, grid, a.stream);
  } else if (sp.first > 0) {  // bf16 pool, Lq = Lv = 64 or 128, two-stage or decode, no mask
    rc = a.lq == 128 ? launch_attn_first<128>(a.mode, tm, kp, grid, a.stream)
                     : launch_attn_first<64>(a.mode, tm, kp, grid, a.stream);
  } else if (a.kv_fmt != kKvBf16 && mla) {
    // the MLA pair kernel over an fp8 pool
    const bool e4 = a.kv_fmt == kKvFp8E4M3;
    if (a.mode == kTwoStage)
      rc = masked ? (e4 ? launch_mla_pair<kTwoStage, true, 1>(kp, pairs, a.stream)
                        : launch_mla_pair<kTwoStage, true, 2>(kp, pairs, a.stream))
                  : (e4 ? launch_mla_pair<kTwoStage, false, 1>(kp, pairs, a.stream)
                        : launch_mla_pair<kTwoStage, false, 2>(kp, pairs, a.stream));
    else if (a.mode == kUnified)
      rc = masked ? (e4 ? launch_mla_pair<kUnified, true, 1>(kp, pairs, a.stream)
                        : launch_mla_pair<kUnified, true, 2>(kp, pairs, a.stream))
                  : (e4 ? launch_mla_pair<kUnified, false, 1>(kp, pairs, a.stream)
                        : launch_mla_pair<kUnified, false, 2>(kp, pairs, a.stream));
    else
      rc = e4 ? launch_mla_pair<kDecode, false, 1>(kp, pairs, a.stream)
              : launch_mla_pair<kDecode, false, 2>(kp, pairs, a.stream);
  } else if (a.kv_fmt != kKvBf16 && split) {
    // the split head dims over an fp8 pool: the two extend forms, no mask
    if (a.mode == kDecode || masked)
      return set_error(PKX_EUNSUPPORTED,
                       "an fp8 pool with split head dims is built for extend without a mask");
    const bool e4 = a.kv_fmt == kKvFp8E4M3, two = a.mode == kTwoStage;
    if (a.lq == 192)
      rc = two ? (e4 ? launch_attn_kernel<192, kTwoStage, false, 1>(tm, kp, grid, a.stream)
                     : launch_attn_kernel<192, kTwoStage, false, 2>(tm, kp, grid, a.stream))
               : (e4 ? launch_attn_kernel<192, kUnified, false, 1>(tm, kp, grid, a.stream)
                     : launch_attn_kernel<192, kUnified, false, 2>(tm, kp, grid, a.stream));
    else
      rc = two ? (e4 ? launch_attn_kernel<288, kTwoStage, false, 1>(tm, kp, grid, a.stream)
                     : launch_attn_kernel<288, kTwoStage, false, 2>(tm, kp, grid, a.stream))
               : (e4 ? launch_attn_kernel<288, kUnified, false, 1>(tm, kp, grid, a.stream)
                     : launch_attn_kernel<288, kUnified, false, 2>(tm, kp, grid, a.stream));
  } else if (a.kv_fmt != kKvBf16) {
    if (!((a.lq == 128 && a.lv == 128) || (a.lq == 64 && a.lv == 64)))
      return set_error(PKX_EUNSUPPORTED,
                       "an fp8 pool is built for Lq = Lv = 64 or 128, for Lq / Lv = 576 / 512 and "
                       "for the split head dims in extend");
    const bool e4 = a.kv_fmt == kKvFp8E4M3;
    if (a.lq == 128)
      rc = e4 ? launch_attn_fp8<128, 1>(a.mode, masked, tm, kp, grid, a.stream)
              : launch_attn_fp8<128, 2>(a.mode, masked, tm, kp, grid, a.stream);
    else
      rc = e4 ? launch_attn_fp8<64, 1>(a.mode, masked, tm, kp, grid, a.stream)
              : launch_attn_fp8<64, 2>(a.mode, masked, tm, kp, grid, a.stream);
  } else if (a.lq == 128 && a.lv == 128) {
    if (a.mode == kTwoStage)
      rc = masked ? launch_attn_kernel<128, kTwoStage, true>(tm, kp, grid, a.stream)
                  : launch_attn_kernel<128, kTwoStage>(tm, kp, grid, a.stream);
    else if (a.mode == kUnified)
      rc = masked ? launch_attn_kernel<128, kUnified, true>(tm, kp, grid, a.stream)
                  : launch_attn_kernel<128, kUnified>(tm, kp, grid, a.stream);
    else rc = launch_attn_kernel<128, kDecode>(tm, kp, grid, a.stream);
  } else if (a.lq == 64 && a.lv == 64) {
    if (a.mode == kTwoStage)
      rc = masked ? launch_attn_kernel<64, kTwoStage, true>(tm, kp, grid, a.stream)
                  : launch_attn_kernel<64, kTwoStage>(tm, kp, grid, a.stream);
    else if (a.mode == kUnified)
      rc = masked ? launch_attn_kernel<64, kUnified, true>(tm, kp, grid, a.stream)
                  : launch_attn_kernel<64, kUnified>(tm, kp, grid, a.stream);
    else rc = launch_attn_kernel<64, kDecode>(tm, kp, grid, a.stream);
  } else if (split) {
    if (masked)
      return set_error(PKX_EUNSUPPORTED, "a custom mask is not built for head dims (%d, %d)",
                       a.lq, a.lv);
    if (a.lq == 192) {
      if (a.mode == kTwoStage) rc = launch_attn_kernel<192, kTwoStage>(tm, kp, grid, a.stream);
      else if (a.mode == kUnified) rc = launch_attn_kernel<192, kUnified>(tm, kp, grid, a.stream);
      else rc = launch_attn_kernel<192, kDecode>(tm, kp, grid, a.stream);
    } else {
      if (a.mode == kTwoStage) rc = launch_attn_kernel<288, kTwoStage>(tm, kp, grid, a.stream);
      else if (a.mode == kUnified) rc = launch_attn_kernel<288, kUnified>(tm, kp, grid, a.stream);
      else rc = launch_attn_kernel<288, kDecode>(tm, kp, grid, a.stream);
    }
  } else if (mla) {
    if (a.mode == kTwoStage)
      rc = masked ? launch_mla_pair<kTwoStage, true>(kp, pairs, a.stream)
                  : launch_mla_pair<kTwoStage>(kp, pairs, a.stream);
    else if (a.mode == kUnified)
      rc = masked ? launch_mla_pair<kUnified, true>(kp, pairs, a.stream)
                  : launch_mla_pair<kUnified>(kp, pairs, a.stream);
    else rc = launch_mla_pair<kDecode>(kp, pairs, a.stream);
  } else {
    return set_error(PKX_EUNSUPPORTED, "head dims (%d, %d) not built", a.lq, a.lv);
  }
  if (rc != PKX_OK) return rc;
  if (ev_after) cudaEventRecord(ev_after, a.stream);
  // one warp per combined row: enough CTAs for a full wave of warps (the
  // rows' partial reads are latency-bound), eight per SM at most
  const size_t comb_rows = (size_t)L.comb_max * L.rows_per_slot;
  const int comb_grid = (int)std::min<size_t>((comb_rows + 7) / 8, (size_t)nsm * 8);
  cudaError_t e = launch_pdl(combine_kernel, dim3(comb_grid > 0 ? comb_grid : 1), dim3(256), 0,
                             a.stream,
                             (const WsHeader *)hdr, (const CombineEntry *)sp.comb,
                             (const float *)kp.plse, (const float *)kp.po, kp.o, a.lse, a.sinks,
                             a.hq, group, a.lv, L.rows_per_slot);
  if (e != cudaSuccess) return set_error(PKX_ECUDA, "attention launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
