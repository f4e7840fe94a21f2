// fp4_decode.cu -- decode attention over a 4-bit KV pool (fp4.cuh).
//
// Per sequence, one query row of every head attends to the sequence's keys
// j < T (position T - 1; with a window W the keys j >= T - 1 - W and the
// first S tokens):
//   s_j = sm_scale <q, k_j> (capped: cap tanh(s_j / cap)),
//   o = sum_j softmax(s)_j v_j,  lse = log sum_j exp s_j.
//
// What bounds it.  A key of one KV head is 2 * (D / 2 + D / 16) bytes (144 at
// D = 128), and every one of its 2 D codes has to become a 16-bit number
// before a product: at the copy bandwidth an SM receives 41 elements a clock,
// and two elements take a conversion (two clocks of a quarter SM) and a product
// with their scale.  So a code is converted once, in registers, straight into the
// operand fragment of the product that uses it, and never goes back to shared
// memory (a tcgen05 product would need the converted tile there or in tensor
// memory: 82 bytes a clock written and 82 read back beside the copies).  The
// products are mma.sync m16n8k16 with the keys (then the value dims) as the
// 16 rows and eight query heads as the columns, so a group of up to eight
// heads wastes nothing on padding to 128 rows.
//
// Shape.
//  * S^T = K Q^T.  Lane (g, t) of a warp (g = lane / 4, t = lane % 4) holds D
//    / 4 consecutive dims of two key rows: one 16-byte shared load a row.  The
//    contraction may run over the dims in any order, so a word's eight codes
//    are used in the order the conversion yields them and Q's fragment is
//    permuted once to match.  Each element is multiplied by its block scale
//    (exact in f16).
//  * The online softmax keeps one running maximum per head in all lanes and
//    moves it only when a logit exceeds it by kPLag (in log2), which a vote
//    finds; sums and outputs are fp32, P is rounded to f16 (error 2^-11).
//    f16's normal range ends at 2^-14, and a first token with a large logit
//    and a small value leaves the output to keys far below the maximum: P is
//    taken 2^kPShift times too large (the sum too, so the factor cancels), so
//    that it stays below 2^15 and keeps its 11 bits down to 2^-26 of the
//    maximum (18 nats).
//  * O^T = V^T P^T.  P^T is S^T's accumulator layout transposed 8 x 8
//    (movmatrix).  Lane g holds D / 8 dims of the keys whose P its t holds;
//    two keys' words are interleaved by codes, so the conversion yields (key,
//    next key) pairs of one dim.
//  * A warp is one (KV head, eight query heads) and a contiguous share of the
//    batch's key tiles (32 keys), with its own softmax state; the warps of a
//    CTA that share keys (a stream, one warp a KV head) copy each slot's rows
//    together, by cp.async into a ring of tiles with full / empty barriers.
//  * Measured, 64 x 8192 keys, 32 query and 8 KV heads of 128: 122 us, 5.0 TB/s
//    (0.73 of the copy bandwidth), bound by issue: 667 instructions a tile and
//    head, 65 % of the slots, ALU pipe 55 %, tensor pipe 25 %.
//  * The shares are equal (sizes differ by one tile), computed on the device
//    from kv_indptr by every CTA.  A sequence that lies in one share is
//    finished by its warp; the parts of one that several shares hold go to
//    the workspace as (o, lse) and are merged by a second kernel.
#include <algorithm>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fp4.cuh"
#include "pkx_internal.h"
#include "ptx.cuh"

namespace pkx {

constexpr int kTile = 32;          // keys of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kPShift = 12.0f, kPLag = 3.0f;  // P <= 2^(kPShift + kPLag)

template <int D, int NT>  // head dim; column tiles of eight query heads
struct DecCfg {
  static constexpr int WARPS = NT == 1 ? 16 : 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROW = D / 2, SROW = D / 16;  // code and scale bytes of a row
  static constexpr int OFF_V = kTile * ROW, OFF_KS = 2 * kTile * ROW;
  static constexpr int OFF_VS = OFF_KS + kTile * SROW;
  static constexpr int STAGE = OFF_VS + kTile * SROW;
  static constexpr int STAGES = (NT == 1 ? 3 : 6) * (D == 64 ? 2 : 1);
  // a warp's ring; the odd 64 bytes put neighbouring heads' rows, which one
  // copy instruction writes, in different halves of the banks
  static constexpr int RING = STAGES * STAGE + 64;
  static constexpr int SMEM = WARPS * RING;
  static_assert(SMEM <= 226 * 1024, "shared memory budget");
};

struct Fp4DecParams {
  const __nv_bfloat16 *q;
  __nv_bfloat16 *o;
  float *lse;
  const uint8_t *k, *ks, *v, *vs;
  uint32_t k_ss, ks_ss, v_ss, vs_ss;  // slot strides, bytes
  int64_t k_sh, ks_sh, v_sh, vs_sh;   // head strides, bytes
  uint32_t num_slots;
  const int32_t *kv_indptr, *kv_indices;
  int batch, hq, hkv, group;
  int window, first;
  int head_tiles;   // column tiles per KV head: ceil(group / (8 NT))
  int cta_heads;    // (KV head, column tile) pairs of a CTA
  int head_groups;  // CTAs that share one set of shares
  int streams;      // shares a CTA works on
  int max_shares;
  float scale_log2;  // sm_scale * log2 e * k_scale
  float cap_pre, cap_log2;  // sm_scale * k_scale / cap; cap * log2 e
  int use_cap;
  float v_scale;
  uint64_t wait_ns;  // time limit of every bounded wait
  int stall;
  int32_t *cta_err;  // [grid] status of each CTA
  int2 *entries;     // [max_shares] (sequence, parts) of the sequence split from this share on
  float *plse, *po;  // [2 max_shares][hq], [2 max_shares][hq][D]
};

// Visible keys of sequence b: n keys, of which key v >= first sits gap further on.
__device__ __forceinline__ int visible_keys(const Fp4DecParams &p, int b, int &gap, bool &bad) {
  const int k0 = __ldg(p.kv_indptr + b), T = __ldg(p.kv_indptr + b + 1) - k0;
  gap = 0;
  if (T < 0 || k0 < 0) {
    bad = true;
    return 0;
  }
  if (p.window > 0) gap = (int)max((long long)T - 1 - p.window - p.first, 0ll);
  return T - gap;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},"
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src),
               "r"(src_bytes), "n"(BYTES)
               : "memory");
}

// A word of eight dims' codes of two keys as (key a, key b) f16 pairs of each
// dim: each byte that goes to the converter holds one code of each key.
__device__ __forceinline__ void value_pairs(uint32_t a, uint32_t b, uint32_t (&even)[4],
                                            uint32_t (&odd)[4]) {
  e2m1x8_to_f16((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), even);
  e2m1x8_to_f16(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), odd);
}

// The share that holds tile t when `shares` equal ones hold `tiles`: share w
// begins at tile floor(w tiles / shares).
__device__ __forceinline__ int share_of(int64_t t, int64_t tiles, int64_t shares) {
  return (int)(((t + 1) * shares - 1) / tiles);
}

template <int D, int NT>
__global__ void __launch_bounds__(DecCfg<D, NT>::THREADS, 1)
    decode_fp4_kernel(const Fp4DecParams p) {
  using C = DecCfg<D, NT>;
  constexpr int KW = D / 32;   // words of a key row that a lane holds for K
  constexpr int VW = D / 64;   // words of a key row that a lane holds for V
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_warp[32];
  __shared__ int s_seq[C::WARPS], s_tile0[C::WARPS];  // per stream: first sequence, its first tile
  __shared__ int s_err, s_abort;
  __shared__ uint64_t s_full[C::WARPS][C::STAGES], s_empty[C::WARPS][C::STAGES];  // [stream]
  __shared__ uint64_t s_never;  // no thread arrives (the stall hook waits on it)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int cta_set = blockIdx.x / p.head_groups, hg = blockIdx.x - cta_set * p.head_groups;
  // (KV head, column tile) pairs of this CTA: the warps of a stream
  const int heads = min(p.cta_heads, p.hkv * p.head_tiles - hg * p.cta_heads);
  if (tid == 0) {
    s_err = s_abort = 0;
    mbar_init(&s_never, 1);
  }
  for (int i = tid; i < p.streams * C::STAGES; i += C::THREADS) {
    mbar_init(&s_full[i / C::STAGES][i % C::STAGES], heads * 32);
    mbar_init(&s_empty[i / C::STAGES][i % C::STAGES], heads);
  }
  fence_barrier_init();
  grid_dep_wait();
  grid_dep_launch();

  // ---- the batch's tiles and this CTA's shares of them
  const int ch = (p.batch + C::THREADS - 1) / C::THREADS;
  const int sb0 = min(p.batch, tid * ch), sb1 = min(p.batch, sb0 + ch);
  int mine = 0;
  bool bad = false;
  for (int b = sb0; b < sb1; ++b) {
    int gap;
    mine += (visible_keys(p, b, gap, bad) + kTile - 1) / kTile;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0, tiles = 0;
#pragma unroll
  for (int w = 0; w < C::WARPS; ++w) {
    const int x = s_warp[w];
    if (w < warp) before += x;
    tiles += x;
  }
  const int excl = before + incl - mine;
  const int shares = min(p.max_shares, tiles);
  for (int st = 0; st < p.streams; ++st) {
    const int w = cta_set * p.streams + st;
    if (w >= shares) break;
    const int first_tile = (int)((int64_t)w * tiles / shares);
    if (mine > 0 && first_tile >= excl && first_tile < excl + mine) {
      int at = excl;
      for (int b = sb0; b < sb1; ++b) {
        int gap;
        const int n = (visible_keys(p, b, gap, bad) + kTile - 1) / kTile;
        if (first_tile < at + n) {
          s_seq[st] = b;
          s_tile0[st] = at;
          break;
        }
        at += n;
      }
    }
  }
  // sequences without keys: zero output, spread over the CTAs
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    int gap;
    if (visible_keys(p, b, gap, bad) > 0) continue;
    uint4 *row = reinterpret_cast<uint4 *>(p.o + (int64_t)b * p.hq * D);
    for (int i = tid; i < p.hq * D / 8; i += C::THREADS) row[i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = tid; i < p.hq; i += C::THREADS) p.lse[(int64_t)b * p.hq + i] = -INFINITY;
  }
  __syncthreads();

  // ---- this warp: a share and a (KV head, column tile)
  const int stream = warp / p.cta_heads, head_slot = warp - stream * p.cta_heads;
  const int vh = hg * p.cta_heads + head_slot;
  const int share = cta_set * p.streams + stream;
  if (stream < p.streams && head_slot < heads && share < p.max_shares) {
    const int kvh = vh / p.head_tiles;
    const int head0 = (vh - kvh * p.head_tiles) * (8 * NT);  // first head within the group
    int2 entry = make_int2(0, 0);
    if (share < shares) {
      const int tile_end = (int)((int64_t)(share + 1) * tiles / shares);
      const int tile_beg = (int)((int64_t)share * tiles / shares);
      const uint32_t ring = smem_u32(smem) + warp * C::RING;
      volatile int *abort_flag = &s_abort;

      // -- copy side: the tile `ctile` of sequence cb, whose tiles begin at
      // cbase.  The stream's warps copy a tile together, consecutive lanes on
      // consecutive heads of one slot, so that a slot's row is fetched as one
      // run: with each warp copying its own head's rows, the warps drifted
      // apart and 64 x 8192 keys at random slots took 229 us against 139 at
      // sequential ones.
      int cb = s_seq[stream], cbase = s_tile0[stream], ctile = tile_beg;
      int cgap, cn = visible_keys(p, cb, cgap, bad);
      const int32_t *cidx = p.kv_indices + __ldg(p.kv_indptr + cb);
      const int flat = head_slot * 32 + lane;  // lane of the stream
      constexpr int CPR = C::ROW / 16;         // 16-byte chunks of a row
      constexpr int NCOPY = CPR;               // rows of K (and of V) a lane copies a chunk of
      const int chunk = flat % CPR, chead = flat / CPR % heads, ckey = flat / (CPR * heads);
      const int shead = flat % heads, skey = flat / heads;  // its block scales
      auto kv_head = [&](int slot) { return (hg * p.cta_heads + slot) / p.head_tiles; };
      const uint8_t *kp = p.k + kv_head(chead) * p.k_sh + chunk * 16;
      const uint8_t *vp = p.v + kv_head(chead) * p.v_sh + chunk * 16;
      const uint8_t *ksp = p.ks + kv_head(shead) * p.ks_sh, *vsp = p.vs + kv_head(shead) * p.vs_sh;
      // V's chunks swap halves every two rows, so that the four rows of a V
      // load lie in different banks; a lane's rows are a multiple of 4 apart
      const int vchunk = D == 128 ? chunk ^ (((ckey >> 1) & 1) << 1) : chunk;
      const uint32_t ring0 = smem_u32(smem) + stream * p.cta_heads * C::RING;
      const uint32_t kdst = ring0 + chead * C::RING + ckey * C::ROW + chunk * 16;
      const uint32_t vdst = ring0 + chead * C::RING + C::OFF_V + ckey * C::ROW + vchunk * 16;
      const uint32_t sdst = ring0 + shead * C::RING + C::OFF_KS + skey * C::SROW;
      // this lane's key of the next tile: its slot as it stands in the list
      // (looked at a tile later, so that no lane waits for the load here),
      // and whether there is one
      int next_slot = 0;
      bool next_have = false;
      auto fetch_index = [&]() {
        next_have = false;
        if (ctile >= tile_end) return;
        while ((ctile - cbase) * kTile >= cn) {  // on to the next sequence with keys
          cbase += (cn + kTile - 1) / kTile;
          cn = visible_keys(p, ++cb, cgap, bad);
          cidx = p.kv_indices + __ldg(p.kv_indptr + cb);
        }
        const int v = (ctile - cbase) * kTile + lane;
        ++ctile;
        next_have = v < cn;
        if (next_have) next_slot = __ldg(cidx + (v < p.first ? v : v + cgap));
      };
      auto copy_tile = [&](int stage) {
        const bool in_pool = (uint32_t)next_slot < p.num_slots;
        bad |= next_have && !in_pool;
        const int slot = next_have && in_pool ? next_slot : -1;
#pragma unroll
        for (int i = 0; i < NCOPY; ++i) {
          const int s = __shfl_sync(0xffffffffu, slot, ckey + i * (kTile / NCOPY));
          const uint32_t n = s >= 0 ? 16u : 0u, su = (uint32_t)max(s, 0);
          const uint32_t at = stage * C::STAGE + i * (kTile / NCOPY) * C::ROW;
          cp_async_16(kdst + at, kp + (uint64_t)su * p.k_ss, n);
          cp_async_16(vdst + at, vp + (uint64_t)su * p.v_ss, n);
        }
        const int s = __shfl_sync(0xffffffffu, slot, skey);
        const uint32_t su = (uint32_t)max(s, 0), n = s >= 0 ? (uint32_t)C::SROW : 0u;
        const uint32_t at = sdst + stage * C::STAGE;
        cp_async_small<C::SROW>(at, ksp + (uint64_t)su * p.ks_ss, n);
        cp_async_small<C::SROW>(at + (C::OFF_VS - C::OFF_KS), vsp + (uint64_t)su * p.vs_ss, n);
        cp_async_arrive_noinc(&s_full[stream][stage]);
      };
      const int n_tiles = tile_end - tile_beg;
      fetch_index();
      for (int s = 0; s < C::STAGES - 1 && s < n_tiles; ++s) {
        copy_tile(s);
        fetch_index();
      }

      // -- compute side
      // key rows of this lane: row r of an 8-row half tile is key r / 2 (even
      // r) or 4 + (r / 2 ^ 3) (odd r), which keeps the loads below free of
      // bank conflicts
      const int krow = (g & 1) ? 4 + ((g >> 1) ^ 3) : g >> 1;
      const int va = t, vb = 4 + (t ^ 3);  // V rows of this lane in a half tile
      auto v_off = [&](int row) -> uint32_t {
        if constexpr (D == 128)
          return row * C::ROW + (((g >> 1) ^ (((row >> 1) & 1) << 1)) << 4) + (g & 1) * 8;
        else
          return row * C::ROW + g * 4;
      };
      const uint32_t voff_a = v_off(va), voff_b = v_off(vb);
      const int sblk = D == 128 ? g : g >> 1;  // the scale block of this lane's value dims

      int b = s_seq[stream], base = s_tile0[stream], tile = tile_beg, stage = 0;
      uint32_t round = 0;  // times the ring has gone round
      bool ok = true;          // warp-uniform: no wait ran out
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.wait_ns));
        if (!ok) *abort_flag = 1;
        return ok;
      };
      if (p.stall) wait(&s_never, 0);  // test hook: the limit runs out
      while (ok && tile < tile_end) {
        int gap;
        int n = visible_keys(p, b, gap, bad);
        while ((tile - base) * kTile >= n) {
          base += (n + kTile - 1) / kTile;
          n = visible_keys(p, ++b, gap, bad);
        }
        const int nt = (n + kTile - 1) / kTile;
        const int piece_end = min(tile_end, base + nt);
        const bool starts = tile == base, ends = piece_end == base + nt;

        // Q^T fragments: f16, each head scaled by a power of two (its logit
        // factor takes it back) to a largest element in [2^14, 2^15), so that
        // a bf16 query keeps its bits (elements below 2^-31 of the head's
        // largest lose some)
        uint32_t qf[NT][KW][4];
        float mult[NT][2];  // accumulator -> log2 domain, or -> tanh's argument
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          const int head = head0 + c * 8 + g;
          const uint4 *qr = reinterpret_cast<const uint4 *>(
              p.q + ((int64_t)b * p.hq + kvh * p.group + min(head, p.group - 1)) * D + t * (D / 4));
          uint32_t qw[KW][4];
          uint32_t top = 0;
#pragma unroll
          for (int w = 0; w < KW; ++w) {
            const uint4 x = __ldg(qr + w);
            qw[w][0] = x.x; qw[w][1] = x.y; qw[w][2] = x.z; qw[w][3] = x.w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top = max(top, max((qw[w][i] >> 7) & 0xFFu, (qw[w][i] >> 23) & 0xFFu));
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = min(max(top, 15u), 254u);  // biased exponent of the head's largest element
          const float down = __uint_as_float((268u - top) << 23);
          const float up = __uint_as_float((top - 14u) << 23);
#pragma unroll
          for (int w = 0; w < KW; ++w) {
#pragma unroll
            for (int i = 0; i < 4; ++i)  // elements 2 i and 2 i + 1 of the word's eight
              qf[c][w][i] = f16_pair(__uint_as_float(qw[w][i] << 16) * down,
                                     __uint_as_float(qw[w][i] & 0xFFFF0000u) * down);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // heads 2 t and 2 t + 1 of the accumulators
            const float u = __shfl_sync(0xffffffffu, up, (2 * t + j) * 4);
            // (never 0, so that a masked logit stays -inf)
            mult[c][j] = fmaxf((p.use_cap ? p.cap_pre : p.scale_log2) * u, 1e-37f);
          }
        }

        float m[NT][2], l[NT][2], acc[NT][MT][4];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          m[c][0] = m[c][1] = -INFINITY;
          l[c][0] = l[c][1] = 0.f;
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[c][i][j] = 0.f;
        }

        for (; tile < piece_end; ++tile) {
          if (!wait(&s_full[stream][stage], round & 1u)) break;
          const uint32_t st = ring + stage * C::STAGE;
          // S^T of the tile's two key halves of 16
          float s[2][NT][4];
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
            for (int c = 0; c < NT; ++c) s[kt][c][0] = s[kt][c][1] = s[kt][c][2] = s[kt][c][3] = 0.f;
            uint32_t kw[2][KW];  // rows g and g + 8
            uint32_t sc[2][KW / 2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int row = kt * 16 + r * 8 + krow;
              if constexpr (D == 128) {
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3},[%4];"
                             : "=r"(kw[r][0]), "=r"(kw[r][1]), "=r"(kw[r][2]), "=r"(kw[r][3])
                             : "r"(st + row * C::ROW + t * 16));
                uint16_t two;
                asm volatile("ld.shared.u16 %0,[%1];"
                             : "=h"(two)
                             : "r"(st + C::OFF_KS + row * C::SROW + t * 2));
                const __half2 f = e4m3x2_to_f16x2(two);
                const uint32_t u = *reinterpret_cast<const uint32_t *>(&f);
                sc[r][0] = __byte_perm(u, u, 0x1010);
                sc[r][1] = __byte_perm(u, u, 0x3232);
              } else {
                asm volatile("ld.shared.v2.u32 {%0,%1},[%2];"
                             : "=r"(kw[r][0]), "=r"(kw[r][1])
                             : "r"(st + row * C::ROW + t * 8));
                uint32_t one;
                asm volatile("ld.shared.u8 %0,[%1];"
                             : "=r"(one)
                             : "r"(st + C::OFF_KS + row * C::SROW + t));
                const __half2 f = e4m3x2_to_f16x2(one | (one << 8));
                sc[r][0] = *reinterpret_cast<const uint32_t *>(&f);
              }
            }
#pragma unroll
            for (int w = 0; w < KW; ++w) {
              uint32_t a[2][4];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                e2m1x8_to_f16(kw[r][w], a[r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[r][i] = hmul2_u32(a[r][i], sc[r][w / 2]);
              }
#pragma unroll
              for (int c = 0; c < NT; ++c) {
                mma_f16(s[kt][c], a[0][0], a[1][0], a[0][1], a[1][1], qf[c][w][0], qf[c][w][1]);
                mma_f16(s[kt][c], a[0][2], a[1][2], a[0][3], a[1][3], qf[c][w][2], qf[c][w][3]);
              }
            }
          }

          // softmax.  s[kt][c][2 r + j]: key row 8 r + g of half kt, head 2 t + j
          const int left = n - (tile - base) * kTile;  // keys of the tile (32 or fewer)
          if (p.use_cap) {
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float &x = s[i >> 2][c][i & 3];
                x = p.cap_log2 * tanhf(x * mult[c][i & 1]);
              }
          }
          if (left < kTile) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                if (kt * 16 + r * 8 + krow >= left) {
#pragma unroll
                  for (int c = 0; c < NT; ++c) s[kt][c][2 * r] = s[kt][c][2 * r + 1] = -INFINITY;
                }
          }
          bool grow = false;
          float mx[NT][2], mul[NT][2];
#pragma unroll
          for (int c = 0; c < NT; ++c) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              mul[c][j] = p.use_cap ? 1.0f : mult[c][j];
              mx[c][j] = mul[c][j] * fmaxf(fmaxf(s[0][c][j], s[0][c][2 + j]),
                                           fmaxf(s[1][c][j], s[1][c][2 + j]));
              grow |= mx[c][j] > m[c][j] + kPLag;
            }
          }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int c = 0; c < NT; ++c) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float x = mx[c][j];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                const float mn = fmaxf(m[c][j], x);
                const float a = mn == -INFINITY ? 1.0f : ex2_approx(m[c][j] - mn);
                m[c][j] = mn;
                l[c][j] *= a;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  acc[c][i][j] *= a;
                  acc[c][i][2 + j] *= a;
                }
              }
            }
          }
          uint32_t pb[2][NT][2];
#pragma unroll
          for (int c = 0; c < NT; ++c) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float nm = m[c][j] == -INFINITY ? 0.f : kPShift - m[c][j];
#pragma unroll
              for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  float &x = s[kt][c][2 * r + j];
                  x = ex2_approx(fmaf(x, mul[c][j], nm));
                  l[c][j] += x;
                }
            }
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
              for (int r = 0; r < 2; ++r)
                pb[kt][c][r] = transpose8x8(f16_pair(s[kt][c][2 * r], s[kt][c][2 * r + 1]));
          }

          // O^T += V^T P^T
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            const uint32_t vt = st + C::OFF_V + kt * 16 * C::ROW;
            const uint32_t vst = st + C::OFF_VS + kt * 16 * C::SROW + sblk;
            uint32_t wa[2][VW], wb[2][VW], sc[2];  // keys va, vb of the two 8-key halves
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (D == 128) {
                const uint2 x = ld_shared_u2(vt + r * 8 * C::ROW + voff_a);
                const uint2 y = ld_shared_u2(vt + r * 8 * C::ROW + voff_b);
                wa[r][0] = x.x; wa[r][1] = x.y;
                wb[r][0] = y.x; wb[r][1] = y.y;
              } else {
                asm volatile("ld.shared.u32 %0,[%1];" : "=r"(wa[r][0]) : "r"(vt + r * 8 * C::ROW + voff_a));
                asm volatile("ld.shared.u32 %0,[%1];" : "=r"(wb[r][0]) : "r"(vt + r * 8 * C::ROW + voff_b));
              }
              uint32_t x, y;
              asm volatile("ld.shared.u8 %0,[%1];" : "=r"(x) : "r"(vst + (r * 8 + va) * C::SROW));
              asm volatile("ld.shared.u8 %0,[%1];" : "=r"(y) : "r"(vst + (r * 8 + vb) * C::SROW));
              const __half2 f = e4m3x2_to_f16x2(x | (y << 8));
              sc[r] = *reinterpret_cast<const uint32_t *>(&f);
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              // row g of tile 4 w + i is dim 2 i of the word, row g + 8 dim 2 i + 1
              uint32_t even[2][4], odd[2][4];
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                value_pairs(wa[r][w], wb[r][w], even[r], odd[r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  even[r][i] = hmul2_u32(even[r][i], sc[r]);
                  odd[r][i] = hmul2_u32(odd[r][i], sc[r]);
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NT; ++c)
                  mma_f16(acc[c][4 * w + i], even[0][i], odd[0][i], even[1][i], odd[1][i],
                          pb[kt][c][0], pb[kt][c][1]);
            }
          }
          // this warp is done with the stage; refill the one before it with the
          // tile STAGES - 1 ahead once the stream's other warps are done too
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[stream][stage]);
          if (tile + C::STAGES - 1 < tile_end) {
            const int fill = stage == 0 ? C::STAGES - 1 : stage - 1;
            if (tile > tile_beg &&
                !wait(&s_empty[stream][fill], (stage == 0 ? round - 1 : round) & 1u))
              break;
            copy_tile(fill);
            fetch_index();
          }
          if (++stage == C::STAGES) {
            stage = 0;
            ++round;
          }
        }
        if (!ok) break;

        // ---- the piece's result.  Lane (g, t) holds dims (D / 8) g + ... of
        // heads 2 t and 2 t + 1
        const bool whole = starts && ends;
        const int64_t slot = 2 * (int64_t)share + (starts ? 1 : 0);
        if (starts && !ends)
          entry = make_int2(b, share_of(base + nt - 1, tiles, shares) - share + 1);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float ls = l[c][j];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
            const int head = head0 + c * 8 + 2 * t + j;
            if (head >= p.group) continue;
            const int hqi = kvh * p.group + head;
            const float inv = ls == 0.f ? 0.f : p.v_scale / ls;  // a NaN sum stays NaN
            const float lse = ls == 0.f ? -INFINITY : (m[c][j] - kPShift + __log2f(ls)) * kLn2;
            float x[D / 8];
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x[8 * w + 2 * i] = acc[c][4 * w + i][j] * inv;
                x[8 * w + 2 * i + 1] = acc[c][4 * w + i][2 + j] * inv;
              }
            if (whole) {
              uint4 *row = reinterpret_cast<uint4 *>(p.o + ((int64_t)b * p.hq + hqi) * D + g * (D / 8));
#pragma unroll
              for (int w = 0; w < VW; ++w)
                row[w] = make_uint4(pack_bf16(x[8 * w], x[8 * w + 1]), pack_bf16(x[8 * w + 2], x[8 * w + 3]),
                                    pack_bf16(x[8 * w + 4], x[8 * w + 5]),
                                    pack_bf16(x[8 * w + 6], x[8 * w + 7]));
              if (p.lse && g == 0) p.lse[(int64_t)b * p.hq + hqi] = lse;
            } else {
              float4 *row = reinterpret_cast<float4 *>(p.po + (slot * p.hq + hqi) * D + g * (D / 8));
#pragma unroll
              for (int w = 0; w < 2 * VW; ++w)
                row[w] = make_float4(x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]);
              if (g == 0) p.plse[slot * p.hq + hqi] = lse;
            }
          }
        }
      }
      cp_async_wait_all();
    }
    if (vh == 0 && lane == 0) p.entries[share] = entry;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) s_err = PKX_EDEVICE;
  __syncthreads();
  if (tid == 0) p.cta_err[blockIdx.x] = s_abort ? PKX_ETIMEOUT : s_err;
}

// Merge of the sequences that several shares hold: part i of entry `share`
// lies in slot 2 share + 1 (i = 0) or 2 (share + i).  lse = log sum exp lse_i,
// o = sum exp(lse_i - lse) o_i.  Few parts: a warp a row; many (a long
// sequence over the whole device): a CTA a row, its warps taking every eighth
// part.
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeWarpParts = 32;
// Sequences of more than kMergeWarpParts parts: n parts take n - 1 share
// borders, so there are at most max_shares / kMergeWarpParts of them.
constexpr int kMergeLong = 128;
constexpr int kMaxShares = kMergeLong * kMergeWarpParts;

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    decode_fp4_merge_kernel(WsHeader *hdr, const int32_t *cta_err, int n_err, const int2 *entries,
                            int max_shares, const float *__restrict__ plse,
                            const float *__restrict__ po, __nv_bfloat16 *o, float *lse_out, int hq) {
  constexpr int E = D / 32;  // elements a lane holds
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps], s_o[kMergeWarps][D];
  __shared__ int s_few[kMaxShares], s_long[kMergeLong];
  __shared__ int2 s_count[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x == 0) {
    bool late = false, bad = false;
    for (int i = threadIdx.x; i < n_err; i += kMergeThreads) {
      late |= cta_err[i] == PKX_ETIMEOUT;
      bad |= cta_err[i] == PKX_EDEVICE;
    }
    late = __syncthreads_or(late);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) hdr->status = late ? PKX_ETIMEOUT : bad ? PKX_EDEVICE : PKX_OK;
  }
  // parts [i0, n) by step: running maximum, sum and weighted sum of one row
  auto gather = [&](int share, int h, int i0, int n, int step, float &m, float &l, float (&a)[E]) {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
    // sixteen parts' loads go out together: one at a time, a row of 300 parts
    // was a chain of 38 loads a warp (16 us)
    constexpr int U = 16;
    for (int i = i0; i < n; i += step * U) {
      float pl[U], x[U][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u * step;
        pl[u] = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) x[u][e] = 0.f;
        if (k < n) {
          const int64_t row = (k == 0 ? 2 * (int64_t)share + 1 : 2 * ((int64_t)share + k)) * hq + h;
          pl[u] = __ldcg(plse + row);
          if constexpr (E == 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(po + row * D) + lane);
            x[u][0] = f.x; x[u][1] = f.y; x[u][2] = f.z; x[u][3] = f.w;
          } else {
            const float2 f = __ldcg(reinterpret_cast<const float2 *>(po + row * D) + lane);
            x[u][0] = f.x; x[u][1] = f.y;
          }
        }
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < U; ++u) mn = fmaxf(mn, pl[u]);
      const float mr = mn == -INFINITY ? 0.f : mn;
      const float wo = ex2_approx((m - mr) * kLog2e);
      m = mn;
      l *= wo;
#pragma unroll
      for (int e = 0; e < E; ++e) a[e] *= wo;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = ex2_approx((pl[u] - mr) * kLog2e);
        l += w;
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] += w * x[u][e];
      }
    }
  };
  auto store = [&](int b, int h, float m, float l, const float (&a)[E]) {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const int64_t row = (int64_t)b * hq + h;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t *>(o + row * D + lane * E + e) = pack_bf16(a[e] * inv, a[e + 1] * inv);
    if (lse_out && lane == 0) lse_out[row] = l == 0.f ? -INFINITY : m + __logf(l);
  };
  // the split sequences' shares, in order (every CTA takes its rows by their
  // place in this list, so it has to be the same list in all of them): of few
  // parts in s_few, of many in s_long
  int n_few = 0, n_long = 0;
  for (int base = 0; base < max_shares; base += kMergeThreads) {
    const int i = base + (int)threadIdx.x;
    const int n = i < max_shares ? entries[i].y : 0;
    const unsigned few = __ballot_sync(0xffffffffu, n > 0 && n <= kMergeWarpParts);
    const unsigned many = __ballot_sync(0xffffffffu, n > kMergeWarpParts);
    if (lane == 0) s_count[warp] = make_int2(__popc(few), __popc(many));
    __syncthreads();
    int at_few = n_few, at_long = n_long;
    for (int w = 0; w < kMergeWarps; ++w) {
      const int2 c = s_count[w];
      if (w < warp) {
        at_few += c.x;
        at_long += c.y;
      }
      n_few += c.x;
      n_long += c.y;
    }
    const unsigned below = (1u << lane) - 1u;
    if (n > kMergeWarpParts) {
      const int at = at_long + __popc(many & below);
      if (at < kMergeLong) s_long[at] = i;
    } else if (n > 0) {
      s_few[at_few + __popc(few & below)] = i;
    }
    __syncthreads();
  }
  n_long = min(n_long, kMergeLong);
  for (int i = blockIdx.x * kMergeWarps + warp; i < n_few * hq; i += gridDim.x * kMergeWarps) {
    const int k = i / hq, h = i - k * hq, share = s_few[k];
    const int2 e = entries[share];
    float m, l, a[E];
    gather(share, h, 0, e.y, 1, m, l, a);
    store(e.x, h, m, l, a);
  }
  for (int i = blockIdx.x; i < n_long * hq; i += gridDim.x) {
    const int k = i / hq, h = i - k * hq, share = s_long[k];
    const int2 e = entries[share];
    float m, l, a[E];
    gather(share, h, warp, e.y, kMergeWarps, m, l, a);
    __syncthreads();  // the previous row's partials are read
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
#pragma unroll
    for (int x = 0; x < E; ++x) s_o[warp][lane * E + x] = a[x];
    __syncthreads();
    if (warp == 0) {
      m = -INFINITY;
      for (int w = 0; w < kMergeWarps; ++w) m = fmaxf(m, s_m[w]);
      const float mr = m == -INFINITY ? 0.f : m;
      l = 0.f;
#pragma unroll
      for (int x = 0; x < E; ++x) a[x] = 0.f;
      for (int w = 0; w < kMergeWarps; ++w) {
        const float f = ex2_approx((s_m[w] - mr) * kLog2e);
        l += s_l[w] * f;
#pragma unroll
        for (int x = 0; x < E; ++x) a[x] += s_o[w][lane * E + x] * f;
      }
      store(e.x, h, m, l, a);
    }
  }
}

// ===================================================================== host
// How the (KV head, column tile) pairs lie over CTAs and warps.  Groups of more
// than eight heads give a warp two column tiles: a code is converted once for
// both, but the registers leave room for eight warps an SM instead of sixteen.
// 64 x 8192 keys, 64 query and 4 KV heads: 102 us against 124 us with one
// column tile (D = 64: 78 against 89; 128 query heads and one KV head: 186
// against 247).
struct Fp4DecPlan {
  int nt, warps, head_tiles, cta_heads, head_groups, streams, sets, max_shares, grid;
};

static Fp4DecPlan decode_plan(int hq, int hkv) {
  Fp4DecPlan P;
  const int group = hq / hkv;
  P.nt = group <= 8 ? 1 : 2;
  P.warps = P.nt == 1 ? 16 : 8;
  P.head_tiles = (group + 8 * P.nt - 1) / (8 * P.nt);
  const int heads = hkv * P.head_tiles;
  P.head_groups = (heads + P.warps - 1) / P.warps;
  P.cta_heads = (heads + P.head_groups - 1) / P.head_groups;
  P.streams = P.warps / P.cta_heads;
  const int nsm = num_sms_current_device();
  P.sets = nsm > P.head_groups ? nsm / P.head_groups : 1;
  P.sets = std::min(P.sets, kMaxShares / P.streams);
  P.max_shares = P.sets * P.streams;
  P.grid = P.sets * P.head_groups;
  return P;
}

struct Fp4DecLayout {
  size_t err, entries, plse, po, total;
};

static Fp4DecLayout decode_layout(const Fp4DecPlan &P, int hq, int d) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  Fp4DecLayout L;
  L.err = up(sizeof(WsHeader));
  L.entries = up(L.err + sizeof(int32_t) * (size_t)P.grid);
  L.plse = up(L.entries + sizeof(int2) * (size_t)P.max_shares);
  L.po = up(L.plse + sizeof(float) * 2 * (size_t)P.max_shares * hq);
  L.total = up(L.po + sizeof(float) * 2 * (size_t)P.max_shares * hq * d);
  return L;
}

size_t fp4_decode_workspace(int hq, int hkv, int d) {
  return decode_layout(decode_plan(hq, hkv), hq, d).total;
}

template <int D, int NT>
static cudaError_t launch_decode(const Fp4DecParams &p, int grid, cudaStream_t st) {
  using C = DecCfg<D, NT>;
  // the shared-memory limit is a property of the device's copy of the kernel
  static PerDevice configured;
  std::atomic<int> *done = configured.here();
  if (!done || done->load(std::memory_order_acquire) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(
        decode_fp4_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (done) done->store(1, std::memory_order_release);
  }
  return launch_pdl(decode_fp4_kernel<D, NT>, dim3(grid), dim3(C::THREADS), C::SMEM, st, p);
}

int launch_decode_fp4(const Fp4DecodeArgs &a) {
  const Fp4DecPlan P = decode_plan(a.hq, a.hkv);
  const Fp4DecLayout L = decode_layout(P, a.hq, a.d);
  if (a.workspace == nullptr || a.workspace_bytes < L.total)
    return set_error(PKX_EWORKSPACE, "workspace of %zu bytes given, %zu needed", a.workspace_bytes,
                     L.total);
  if (reinterpret_cast<uintptr_t>(a.workspace) & 255)
    return set_error(PKX_EINVAL, "workspace must be 256-byte aligned");
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  Fp4DecParams p{};
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.o = static_cast<__nv_bfloat16 *>(a.o);
  p.lse = a.lse;
  p.k = a.pool.k; p.ks = a.pool.ks; p.v = a.pool.v; p.vs = a.pool.vs;
  p.k_ss = (uint32_t)a.pool.k_ss; p.ks_ss = (uint32_t)a.pool.ks_ss;
  p.v_ss = (uint32_t)a.pool.v_ss; p.vs_ss = (uint32_t)a.pool.vs_ss;
  p.k_sh = a.pool.k_sh; p.ks_sh = a.pool.ks_sh; p.v_sh = a.pool.v_sh; p.vs_sh = a.pool.vs_sh;
  p.num_slots = (uint32_t)a.pool.num_slots;
  p.kv_indptr = a.kv_indptr;
  p.kv_indices = a.kv_indices;
  p.batch = a.batch; p.hq = a.hq; p.hkv = a.hkv; p.group = a.hq / a.hkv;
  p.window = a.window;
  p.first = a.first_tokens;
  p.head_tiles = P.head_tiles;
  p.cta_heads = P.cta_heads;
  p.head_groups = P.head_groups;
  p.streams = P.streams;
  p.max_shares = P.max_shares;
  const float sm_scale = (a.sm_scale > 0.f ? a.sm_scale : 1.0f / sqrtf((float)a.d)) * a.k_scale;
  p.scale_log2 = sm_scale * kLog2e;
  p.use_cap = a.logit_cap > 0.f;
  p.cap_pre = p.use_cap ? sm_scale / a.logit_cap : 0.f;
  p.cap_log2 = p.use_cap ? a.logit_cap * kLog2e : 0.f;
  p.v_scale = a.v_scale;
  wait_settings(&p.wait_ns, &p.stall);
  p.cta_err = reinterpret_cast<int32_t *>(ws + L.err);
  p.entries = reinterpret_cast<int2 *>(ws + L.entries);
  p.plse = reinterpret_cast<float *>(ws + L.plse);
  p.po = reinterpret_cast<float *>(ws + L.po);
  cudaEvent_t ev_before = nullptr, ev_after = nullptr;
  attention_events(&ev_before, &ev_after);
  if (ev_before) cudaEventRecord(ev_before, a.stream);
  cudaError_t e = a.d == 128 ? (P.nt == 1 ? launch_decode<128, 1>(p, P.grid, a.stream)
                                          : launch_decode<128, 2>(p, P.grid, a.stream))
                             : (P.nt == 1 ? launch_decode<64, 1>(p, P.grid, a.stream)
                                          : launch_decode<64, 2>(p, P.grid, a.stream));
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "decode_fp4_kernel launch: %s", cudaGetErrorString(e));
  if (ev_after) cudaEventRecord(ev_after, a.stream);
  WsHeader *hdr = reinterpret_cast<WsHeader *>(ws);
  const int64_t rows = (int64_t)P.max_shares * a.hq;
  const int grid = (int)std::min<int64_t>((rows + kMergeWarps - 1) / kMergeWarps,
                                          (int64_t)num_sms_current_device() * 4);
  const int32_t *err = p.cta_err;
  const int2 *ent = p.entries;
  const float *plse = p.plse, *po = p.po;
  e = a.d == 128 ? launch_pdl(decode_fp4_merge_kernel<128>, dim3(grid), dim3(kMergeThreads), 0,
                              a.stream, hdr, err, P.grid, ent, P.max_shares, plse, po, p.o, p.lse,
                              a.hq)
                 : launch_pdl(decode_fp4_merge_kernel<64>, dim3(grid), dim3(kMergeThreads), 0,
                              a.stream, hdr, err, P.grid, ent, P.max_shares, plse, po, p.o, p.lse,
                              a.hq);
  if (e != cudaSuccess)
    return set_error(PKX_ECUDA, "decode_fp4_merge_kernel launch: %s", cudaGetErrorString(e));
  return PKX_OK;
}

}  // namespace pkx
