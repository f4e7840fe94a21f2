// api.cu -- the extern "C" entry points of libpkx (declared in include/pkx.h):
// host-side argument validation, then the launchers.  No entry point
// allocates device memory or synchronises the stream (except
// pkx_workspace_status, whose job is to read the device status word).
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstddef>
#include <cstdio>
#include <cuda_runtime.h>

#include "pkx_internal.h"

namespace pkx {

static thread_local char g_err[512] = "";
static thread_local cudaEvent_t g_ev_before = nullptr, g_ev_after = nullptr;
static thread_local uint64_t g_wait_ns = 0;
static thread_local int g_stall = 0;

void attention_events(cudaEvent_t *before, cudaEvent_t *after) {
  *before = g_ev_before;
  *after = g_ev_after;
}

void wait_settings(uint64_t *wait_ns, int *stall) {
  *wait_ns = g_wait_ns ? g_wait_ns : 2000000000ull;
  *stall = g_stall;
}

int set_error(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}

static bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static int check_heads(int hq, int hkv, int lq, int lv) {
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0)
    return set_error(PKX_EINVAL, "hq=%d must be a positive multiple of hkv=%d", hq, hkv);
  if (hq / hkv > kBlockM)
    return set_error(PKX_EUNSUPPORTED, "group size hq/hkv=%d > %d not built", hq / hkv, kBlockM);
  const bool ok = (lq == 64 && lv == 64) || (lq == 128 && lv == 128) || (lq == 576 && lv == 512) ||
                  split_head_dims(lq, lv);
  if (!ok) return set_error(PKX_EUNSUPPORTED, "head dims (lq=%d, lv=%d) not built", lq, lv);
  return PKX_OK;
}

static int check_rows(const char *name, const void *p, int64_t s0, int64_t s1) {
  if (!p) return set_error(PKX_EINVAL, "%s is null", name);
  if (!aligned(p, 16)) return set_error(PKX_EINVAL, "%s must be 16-byte aligned", name);
  if (s0 < 0 || s1 < 0 || s0 % 8 || s1 % 8)
    return set_error(PKX_EINVAL, "%s strides (%lld, %lld) must be non-negative multiples of 8",
                     name, (long long)s0, (long long)s1);
  return PKX_OK;
}

// A custom mask needs its offsets.
static int check_mask_sinks(const uint8_t *custom_mask, const int32_t *mask_indptr,
                            const float *sinks) {
  if (custom_mask && (!mask_indptr || !aligned(mask_indptr, 4)))
    return set_error(PKX_EINVAL, "custom_mask needs an aligned int32 mask_indptr");
  if (sinks && !aligned(sinks, 4)) return set_error(PKX_EINVAL, "sinks misaligned");
  return PKX_OK;
}

// The pool's element format and its scales (an fp8 pool: Lq = Lv = 64 or
// 128, or the MLA head 576 / 512; with or without a custom mask).
static int check_kv_format(int kv_dtype, float k_scale, float v_scale, int lq, int lv,
                           bool decode) {
  if (kv_dtype == kKvBf16) return PKX_OK;
  if (kv_dtype != kKvFp8E4M3 && kv_dtype != kKvFp8E5M2)
    return set_error(PKX_EINVAL, "kv_dtype %d is not a PKX_KV_* value", kv_dtype);
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return set_error(PKX_EINVAL, "k_scale and v_scale must be positive and finite");
  if (!((lq == 64 && lv == 64) || (lq == 128 && lv == 128) || (lq == 576 && lv == 512) ||
        (split_head_dims(lq, lv) && !decode)))
    return set_error(PKX_EUNSUPPORTED,
                     "an fp8 pool is built for Lq = Lv = 64 or 128, for Lq / Lv = 576 / 512 and, "
                     "in extend, for the split head dims 192 / 128 and 288 / 256");
  return PKX_OK;
}

static int check_scalars(float sm_scale, float logit_cap) {
  if (!std::isfinite(sm_scale) || !std::isfinite(logit_cap))
    return set_error(PKX_EINVAL, "sm_scale and logit_cap must be finite");
  return PKX_OK;
}

}  // namespace pkx

using namespace pkx;

extern "C" {

const char *pkx_last_error_string(void) { return g_err; }

const char *pkx_version(void) { return "pkx 0.1 (sm_103a)"; }

void pkx_set_attention_events(void *before, void *after) {
  g_ev_before = static_cast<cudaEvent_t>(before);
  g_ev_after = static_cast<cudaEvent_t>(after);
}

void pkx_set_wait_limit_ns(uint64_t ns) { g_wait_ns = ns; }

void pkx_set_stall_injection(int on) { g_stall = on ? 1 : 0; }

size_t pkx_extend_workspace_size(int batch, int num_q_tokens, int hq, int hkv, int lq, int lv) {
  if (batch < 0 || num_q_tokens < 0 || hkv <= 0 || hq <= 0 || hq % hkv || hq / hkv > kBlockM ||
      lv <= 0)
    return 0;
  return ws_layout(batch, num_q_tokens, hkv, hq / hkv, lq, lv, num_sms_current_device(), false)
      .total;
}

size_t pkx_decode_workspace_min_size(int batch, int hq, int hkv, int lq, int lv) {
  if (batch < 0 || hkv <= 0 || hq <= 0 || hq % hkv || hq / hkv > kBlockM || lv <= 0) return 0;
  return ws_layout(batch, batch, hkv, hq / hkv, lq, lv, num_sms_current_device(), true, false)
      .total;
}

size_t pkx_decode_workspace_size(int batch, int hq, int hkv, int lq, int lv) {
  if (batch < 0 || hkv <= 0 || hq <= 0 || hq % hkv || hq / hkv > kBlockM || lv <= 0) return 0;
  return ws_layout(batch, batch, hkv, hq / hkv, lq, lv, num_sms_current_device(), true)
      .total;
}

int pkx_workspace_status(const void *workspace, void *stream) {
  if (!workspace) return set_error(PKX_EINVAL, "workspace is null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  WsHeader hdr = {};
  const size_t used = offsetof(WsHeader, pad) + (kUnitsPlace + 1) * sizeof(int32_t);
  cudaError_t e = cudaMemcpyAsync(&hdr, workspace, used, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  int32_t st = hdr.status;
  if (e == cudaSuccess && st == kStatusInUnits) {  // the units' own words
    st = PKX_OK;
    const uint8_t *at =
        static_cast<const uint8_t *>(workspace) + 256 * (size_t)hdr.pad[kUnitsPlace];
    int32_t part[1024];
    for (int64_t i = 0; i < hdr.pad[kUnitsCount] && st == PKX_OK && e == cudaSuccess; i += 1024) {
      const int64_t n = std::min<int64_t>(1024, hdr.pad[kUnitsCount] - i);
      e = cudaMemcpyAsync(part, at + i * sizeof(int32_t), n * sizeof(int32_t),
                          cudaMemcpyDeviceToHost, s);
      if (e == cudaSuccess) e = cudaStreamSynchronize(s);
      for (int64_t k = 0; k < n && e == cudaSuccess; ++k)
        if (part[k]) st = PKX_EDEVICE;
    }
  }
  if (e != cudaSuccess) return set_error(PKX_ECUDA, "status read: %s", cudaGetErrorString(e));
  if (st == PKX_EDEVICE) return set_error(PKX_EDEVICE, "device-side index or indptr check failed");
  if (st == PKX_ETIMEOUT) return set_error(PKX_ETIMEOUT, "a device wait ran out of time");
  if (st != 0) return set_error(st, "device status %d", st);
  return PKX_OK;
}

}  // extern "C"

// Validation and argument packing shared by the two-stage entry points.
static int two_stage_args(AttnArgs &a, const void *q_extend, const void *k_extend,
                          const void *v_extend, void *o_extend, const void *k_buffer,
                          const void *v_buffer, const int32_t *qo_indptr,
                          const int32_t *kv_indptr, const int32_t *kv_indices, int batch,
                          int num_q_tokens, int hq, int hkv, int lq, int lv, int64_t ke_st,
                          int64_t ke_sh, int64_t ve_st, int64_t ve_sh, int64_t kb_ss,
                          int64_t kb_sh, int64_t vb_ss, int64_t vb_sh, int64_t num_slots,
                          float sm_scale, float logit_cap, int sliding_window,
                          const uint8_t *custom_mask, const int32_t *mask_indptr,
                          const float *sinks, int kv_dtype, float k_scale, float v_scale,
                          float *lse_out, bool *nothing_to_do) {
  int rc;
  *nothing_to_do = false;
  if (batch < 0 || num_q_tokens < 0) return set_error(PKX_EINVAL, "negative batch or token count");
  if ((rc = check_heads(hq, hkv, lq, lv))) return rc;
  if ((rc = check_scalars(sm_scale, logit_cap))) return rc;
  if ((rc = check_mask_sinks(custom_mask, mask_indptr, sinks))) return rc;
  if ((rc = check_kv_format(kv_dtype, k_scale, v_scale, lq, lv, false))) return rc;
  if (batch == 0 || num_q_tokens == 0) {
    *nothing_to_do = true;
    return PKX_OK;
  }
  if ((rc = check_rows("q_extend", q_extend, 8, 8))) return rc;
  if ((rc = check_rows("o_extend", o_extend, 8, 8))) return rc;
  if ((rc = check_rows("k_extend", k_extend, ke_st, ke_sh))) return rc;
  if ((rc = check_rows("v_extend", v_extend, ve_st, ve_sh))) return rc;
  if ((rc = check_rows("k_buffer", k_buffer, kb_ss, kb_sh))) return rc;
  if ((rc = check_rows("v_buffer", v_buffer, vb_ss, vb_sh))) return rc;
  if (!qo_indptr || !kv_indptr || !aligned(qo_indptr, 4) || !aligned(kv_indptr, 4))
    return set_error(PKX_EINVAL, "qo_indptr / kv_indptr null or misaligned");
  if (kv_indices && !aligned(kv_indices, 4)) return set_error(PKX_EINVAL, "kv_indices misaligned");
  if (lse_out && !aligned(lse_out, 4)) return set_error(PKX_EINVAL, "lse_out misaligned");
  if (num_slots <= 0) return set_error(PKX_EINVAL, "num_slots must be positive");
  a.mode = kTwoStage;
  a.q = q_extend;
  a.o = o_extend;
  a.lse = lse_out;
  a.k_ext = k_extend;
  a.v_ext = v_extend;
  a.ke_st = ke_st; a.ke_sh = ke_sh; a.ve_st = ve_st; a.ve_sh = ve_sh;
  a.k_buf = k_buffer;
  a.v_buf = v_buffer;
  a.kb_ss = kb_ss; a.kb_sh = kb_sh; a.vb_ss = vb_ss; a.vb_sh = vb_sh;
  a.num_slots = num_slots;
  a.qo_indptr = qo_indptr;
  a.kv_indptr = kv_indptr;
  a.prefix_lens = nullptr;
  a.kv_indices = kv_indices;
  a.batch = batch; a.num_q_tokens = num_q_tokens; a.hq = hq; a.hkv = hkv; a.lq = lq; a.lv = lv;
  a.sm_scale = sm_scale; a.logit_cap = logit_cap; a.window = sliding_window;
  a.custom_mask = custom_mask; a.mask_indptr = mask_indptr; a.sinks = sinks;
  a.kv_fmt = kv_dtype; a.k_scale = k_scale; a.v_scale = v_scale;
  return PKX_OK;
}

// Validation and argument packing shared by the decode entry points.
static int decode_args(AttnArgs &a, const void *q, void *o, const void *k_buffer,
                       const void *v_buffer, const int32_t *kv_indptr, const int32_t *kv_indices,
                       int batch, int hq, int hkv, int lq, int lv, int64_t kb_ss, int64_t kb_sh,
                       int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale,
                       float logit_cap, int sliding_window, int kv_dtype, float k_scale,
                       float v_scale, float *lse_out, bool *nothing_to_do) {
  int rc;
  *nothing_to_do = false;
  if (batch < 0) return set_error(PKX_EINVAL, "negative batch");
  if ((rc = check_heads(hq, hkv, lq, lv))) return rc;
  if ((rc = check_scalars(sm_scale, logit_cap))) return rc;
  if ((rc = check_kv_format(kv_dtype, k_scale, v_scale, lq, lv, true))) return rc;
  if (batch == 0) {
    *nothing_to_do = true;
    return PKX_OK;
  }
  if ((rc = check_rows("q", q, 8, 8))) return rc;
  if ((rc = check_rows("o", o, 8, 8))) return rc;
  if ((rc = check_rows("k_buffer", k_buffer, kb_ss, kb_sh))) return rc;
  if ((rc = check_rows("v_buffer", v_buffer, vb_ss, vb_sh))) return rc;
  if (!kv_indptr || !aligned(kv_indptr, 4))
    return set_error(PKX_EINVAL, "kv_indptr null or misaligned");
  if (kv_indices && !aligned(kv_indices, 4)) return set_error(PKX_EINVAL, "kv_indices misaligned");
  if (lse_out && !aligned(lse_out, 4)) return set_error(PKX_EINVAL, "lse_out misaligned");
  if (num_slots <= 0) return set_error(PKX_EINVAL, "num_slots must be positive");
  a.mode = kDecode;
  a.q = q;
  a.o = o;
  a.lse = lse_out;
  a.k_buf = k_buffer;
  a.v_buf = v_buffer;
  a.kb_ss = kb_ss; a.kb_sh = kb_sh; a.vb_ss = vb_ss; a.vb_sh = vb_sh;
  a.num_slots = num_slots;
  a.qo_indptr = nullptr;
  a.kv_indptr = kv_indptr;
  a.prefix_lens = nullptr;
  a.kv_indices = kv_indices;
  a.batch = batch; a.num_q_tokens = batch; a.hq = hq; a.hkv = hkv; a.lq = lq; a.lv = lv;
  a.sm_scale = sm_scale; a.logit_cap = logit_cap; a.window = sliding_window;
  a.kv_fmt = kv_dtype; a.k_scale = k_scale; a.v_scale = v_scale;
  return PKX_OK;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace of the ragged + paged split: one attention pass's scratch (the
// passes run one after the other on the stream and share it), the paged
// pass's bf16 output and both passes' lse.
struct SplitLayout {
  size_t attn, o_paged, lse_paged, lse_ragged, total;
};

static SplitLayout split_layout(int batch, int num_q_tokens, int hq, int hkv, int lq, int lv) {
  SplitLayout L;
  L.attn = 0;
  const size_t attn = align256(ws_layout(batch, num_q_tokens, hkv, hq / hkv, lq, lv,
                                         num_sms_current_device(), false).total);
  const size_t rows = (size_t)num_q_tokens * hq;
  L.o_paged = attn;
  L.lse_paged = L.o_paged + align256(rows * lv * 2);
  L.lse_ragged = L.lse_paged + align256(rows * 4);
  L.total = L.lse_ragged + align256(rows * 4);
  return L;
}

extern "C" {

int pkx_extend_attention_fwd(const void *q_extend, const void *k_extend, const void *v_extend,
                             void *o_extend, const void *k_buffer, const void *v_buffer,
                             const int32_t *qo_indptr, const int32_t *kv_indptr,
                             const int32_t *kv_indices, int batch, int num_q_tokens, int hq,
                             int hkv, int lq, int lv, int64_t ke_st, int64_t ke_sh,
                             int64_t ve_st, int64_t ve_sh, int64_t kb_ss, int64_t kb_sh,
                             int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale,
                             float logit_cap, int sliding_window, const uint8_t *custom_mask,
                             const int32_t *mask_indptr, const float *sinks, int kv_dtype,
                             float k_scale, float v_scale, float *lse_out, void *workspace,
                             size_t workspace_bytes, void *stream) {
  AttnArgs a{};
  bool done;
  int rc = two_stage_args(a, q_extend, k_extend, v_extend, o_extend, k_buffer, v_buffer,
                          qo_indptr, kv_indptr, kv_indices, batch, num_q_tokens, hq, hkv, lq, lv,
                          ke_st, ke_sh, ve_st, ve_sh, kb_ss, kb_sh, vb_ss, vb_sh, num_slots,
                          sm_scale, logit_cap, sliding_window, custom_mask, mask_indptr, sinks,
                          kv_dtype, k_scale, v_scale, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attention(a);
}

int pkx_extend_attention_fwd_kv_write(
    const void *q_extend, const void *k_extend, const void *v_extend, void *o_extend,
    void *k_buffer, void *v_buffer, const int32_t *qo_indptr, const int32_t *kv_indptr,
    const int32_t *kv_indices, int batch, int num_q_tokens, int hq, int hkv, int lq, int lv,
    int64_t ke_st, int64_t ke_sh, int64_t ve_st, int64_t ve_sh, int64_t kb_ss, int64_t kb_sh,
    int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale, float logit_cap,
    int sliding_window, const uint8_t *custom_mask, const int32_t *mask_indptr,
    const float *sinks, int kv_dtype, float k_scale, float v_scale, float *lse_out,
    const int64_t *cache_loc, void *workspace, size_t workspace_bytes, void *stream) {
  AttnArgs a{};
  bool done;
  int rc = two_stage_args(a, q_extend, k_extend, v_extend, o_extend, k_buffer, v_buffer,
                          qo_indptr, kv_indptr, kv_indices, batch, num_q_tokens, hq, hkv, lq, lv,
                          ke_st, ke_sh, ve_st, ve_sh, kb_ss, kb_sh, vb_ss, vb_sh, num_slots,
                          sm_scale, logit_cap, sliding_window, custom_mask, mask_indptr, sinks,
                          kv_dtype, k_scale, v_scale, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  if (!cache_loc || !aligned(cache_loc, 8))
    return set_error(PKX_EINVAL, "cache_loc null or misaligned");
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  const bool mla = lq == 576 && lv == 512;
  if (mla || kv_dtype != kKvBf16) {
    // not fused for these pools: the standalone write first, as the pages
    // order it (the MLA pool stores only the K row; V is its first 512 dims)
    rc = kv_dtype != kKvBf16
             ? pkx_set_kv_buffer_fp8(k_extend, ke_st, ke_sh, mla ? nullptr : v_extend, ve_st,
                                     ve_sh, cache_loc, num_q_tokens, hkv, lq, lv, k_scale,
                                     v_scale, kv_dtype, k_buffer, kb_ss, kb_sh, v_buffer, vb_ss,
                                     vb_sh, num_slots, stream)
             : pkx_set_kv_buffer(k_extend, ke_st, ke_sh, nullptr, ve_st, ve_sh, cache_loc,
                                 num_q_tokens, hkv, lq, lv, k_buffer, kb_ss, kb_sh, v_buffer,
                                 vb_ss, vb_sh, num_slots, stream);
    if (rc != PKX_OK) return rc;
    return launch_attention(a);
  }
  a.cache_loc = cache_loc;
  return launch_attention(a);
}

size_t pkx_ragged_paged_workspace_size(int batch, int num_q_tokens, int hq, int hkv, int lq,
                                       int lv) {
  if (batch < 0 || num_q_tokens < 0 || hkv <= 0 || hq <= 0 || hq % hkv || hq / hkv > kBlockM ||
      lv <= 0)
    return 0;
  return split_layout(batch, num_q_tokens, hq, hkv, lq, lv).total;
}

int pkx_extend_attention_fwd_ragged_paged(
    const void *q_extend, const void *k_extend, const void *v_extend, void *o_extend,
    const void *k_buffer, const void *v_buffer, const int32_t *qo_indptr,
    const int32_t *kv_indptr, const int32_t *kv_indices, int batch, int num_q_tokens, int hq,
    int hkv, int lq, int lv, int64_t ke_st, int64_t ke_sh, int64_t ve_st, int64_t ve_sh,
    int64_t kb_ss, int64_t kb_sh, int64_t vb_ss, int64_t vb_sh, int64_t num_slots,
    float sm_scale, float logit_cap, int sliding_window, int kv_dtype, float k_scale,
    float v_scale, float *lse_out, void *workspace, size_t workspace_bytes, void *stream) {
  AttnArgs a{};
  bool done;
  int rc = two_stage_args(a, q_extend, k_extend, v_extend, o_extend, k_buffer, v_buffer,
                          qo_indptr, kv_indptr, kv_indices, batch, num_q_tokens, hq, hkv, lq, lv,
                          ke_st, ke_sh, ve_st, ve_sh, kb_ss, kb_sh, vb_ss, vb_sh, num_slots,
                          sm_scale, logit_cap, sliding_window, nullptr, nullptr, nullptr,
                          kv_dtype, k_scale, v_scale, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  const SplitLayout L = split_layout(batch, num_q_tokens, hq, hkv, lq, lv);
  if (!workspace || workspace_bytes < L.total)
    return set_error(PKX_EWORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes,
                     L.total);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return set_error(PKX_EINVAL, "workspace must be 256-byte aligned");
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  void *o_paged = ws + L.o_paged;
  float *lse_paged = reinterpret_cast<float *>(ws + L.lse_paged);
  float *lse_ragged = reinterpret_cast<float *>(ws + L.lse_ragged);
  a.workspace = ws + L.attn;
  a.workspace_bytes = L.o_paged - L.attn;
  a.stream = static_cast<cudaStream_t>(stream);
  // ragged pass: extend keys only, causal, straight into o_extend
  a.key_set = kExtendKeys;
  a.lse = lse_ragged;
  if ((rc = launch_attention(a)) != PKX_OK) return rc;
  // paged pass: prefix keys only, all visible, into the workspace
  a.key_set = kPrefixKeys;
  a.keep_status = 1;
  a.o = o_paged;
  a.lse = lse_paged;
  if ((rc = launch_attention(a)) != PKX_OK) return rc;
  // merge the two states in place
  return launch_merge_state(o_extend, lse_ragged, o_paged, lse_paged, o_extend, lse_out,
                            num_q_tokens, hq, lv, a.stream);
}

int pkx_extend_attention_fwd_unified(const void *q, void *o, const void *k_buffer,
                                     const void *v_buffer, const int32_t *qo_indptr,
                                     const int32_t *kv_indptr, const int64_t *kv_indices,
                                     const int32_t *prefix_lens, int batch, int num_q_tokens,
                                     int hq, int hkv, int lq, int lv, int64_t kb_ss,
                                     int64_t kb_sh, int64_t vb_ss, int64_t vb_sh,
                                     int64_t num_slots, float sm_scale, float logit_cap,
                                     int sliding_window, const uint8_t *custom_mask,
                                     const int32_t *mask_indptr, const float *sinks,
                                     int kv_dtype, float k_scale, float v_scale, float *lse_out,
                                     void *workspace, size_t workspace_bytes, void *stream) {
  int rc;
  if (batch < 0 || num_q_tokens < 0) return set_error(PKX_EINVAL, "negative batch or token count");
  if ((rc = check_heads(hq, hkv, lq, lv))) return rc;
  if ((rc = check_scalars(sm_scale, logit_cap))) return rc;
  if ((rc = check_mask_sinks(custom_mask, mask_indptr, sinks))) return rc;
  if ((rc = check_kv_format(kv_dtype, k_scale, v_scale, lq, lv, false))) return rc;
  if (batch == 0 || num_q_tokens == 0) return PKX_OK;
  if ((rc = check_rows("q", q, 8, 8))) return rc;
  if ((rc = check_rows("o", o, 8, 8))) return rc;
  if ((rc = check_rows("k_buffer", k_buffer, kb_ss, kb_sh))) return rc;
  if ((rc = check_rows("v_buffer", v_buffer, vb_ss, vb_sh))) return rc;
  if (!qo_indptr || !kv_indptr || !prefix_lens || !aligned(qo_indptr, 4) ||
      !aligned(kv_indptr, 4) || !aligned(prefix_lens, 4))
    return set_error(PKX_EINVAL, "qo_indptr / kv_indptr / prefix_lens null or misaligned");
  if (kv_indices && !aligned(kv_indices, 8)) return set_error(PKX_EINVAL, "kv_indices misaligned");
  if (lse_out && !aligned(lse_out, 4)) return set_error(PKX_EINVAL, "lse_out misaligned");
  if (num_slots <= 0) return set_error(PKX_EINVAL, "num_slots must be positive");
  AttnArgs a{};
  a.mode = kUnified;
  a.q = q;
  a.o = o;
  a.lse = lse_out;
  a.k_buf = k_buffer;
  a.v_buf = v_buffer;
  a.kb_ss = kb_ss; a.kb_sh = kb_sh; a.vb_ss = vb_ss; a.vb_sh = vb_sh;
  a.num_slots = num_slots;
  a.qo_indptr = qo_indptr;
  a.kv_indptr = kv_indptr;
  a.prefix_lens = prefix_lens;
  a.kv_indices = kv_indices;
  a.batch = batch; a.num_q_tokens = num_q_tokens; a.hq = hq; a.hkv = hkv; a.lq = lq; a.lv = lv;
  a.sm_scale = sm_scale; a.logit_cap = logit_cap; a.window = sliding_window;
  a.custom_mask = custom_mask; a.mask_indptr = mask_indptr; a.sinks = sinks;
  a.kv_fmt = kv_dtype; a.k_scale = k_scale; a.v_scale = v_scale;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attention(a);
}

int pkx_decode_attention_fwd(const void *q, void *o, const void *k_buffer, const void *v_buffer,
                             const int32_t *kv_indptr, const int32_t *kv_indices, int batch,
                             int hq, int hkv, int lq, int lv, int64_t kb_ss, int64_t kb_sh,
                             int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale,
                             float logit_cap, int sliding_window, int kv_dtype, float k_scale,
                             float v_scale, float *lse_out, void *workspace,
                             size_t workspace_bytes, void *stream) {
  AttnArgs a{};
  bool done;
  int rc = decode_args(a, q, o, k_buffer, v_buffer, kv_indptr, kv_indices, batch, hq, hkv, lq, lv,
                       kb_ss, kb_sh, vb_ss, vb_sh, num_slots, sm_scale, logit_cap, sliding_window,
                       kv_dtype, k_scale, v_scale, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attention(a);
}

int pkx_merge_state(const void *v_a, const float *s_a, const void *v_b, const float *s_b,
                    void *v_out, float *s_out, int64_t n_tokens, int h, int dv, void *stream) {
  if (n_tokens < 0 || h <= 0 || dv <= 0 || dv % 8)
    return set_error(PKX_EINVAL, "merge_state: n_tokens >= 0, h > 0, dv a positive multiple of 8");
  if (n_tokens == 0) return PKX_OK;
  if (!v_a || !v_b || !v_out || !s_a || !s_b)
    return set_error(PKX_EINVAL, "merge_state: null input or output");
  if (!aligned(v_a, 16) || !aligned(v_b, 16) || !aligned(v_out, 16) || !aligned(s_a, 4) ||
      !aligned(s_b, 4) || (s_out && !aligned(s_out, 4)))
    return set_error(PKX_EINVAL, "merge_state: misaligned pointer");
  return launch_merge_state(v_a, s_a, v_b, s_b, v_out, s_out, n_tokens, h, dv,
                            static_cast<cudaStream_t>(stream));
}

int pkx_build_unified_kv_indices(const int32_t *prefix_kv_indptr,
                                 const int32_t *prefix_kv_indices,
                                 const int32_t *extend_start_loc, const int32_t *extend_seq_lens,
                                 const int32_t *extend_kv_indices, int batch,
                                 int32_t *unified_kv_indptr, int64_t *unified_kv_indices,
                                 int32_t *prefix_lens, void *stream) {
  if (batch < 0) return set_error(PKX_EINVAL, "negative batch");
  if (!prefix_kv_indptr || !unified_kv_indptr)
    return set_error(PKX_EINVAL, "prefix_kv_indptr / unified_kv_indptr null");
  if (batch > 0 && (!extend_start_loc || !extend_seq_lens || !prefix_lens || !unified_kv_indices))
    return set_error(PKX_EINVAL, "null argument");
  if (!aligned(unified_kv_indices, 8)) return set_error(PKX_EINVAL, "unified_kv_indices misaligned");
  return launch_build_unified(prefix_kv_indptr, prefix_kv_indices, extend_start_loc,
                              extend_seq_lens, extend_kv_indices, batch, unified_kv_indptr,
                              unified_kv_indices, prefix_lens, static_cast<cudaStream_t>(stream));
}

int pkx_set_kv_buffer(const void *k, int64_t k_ts, int64_t k_hs, const void *v, int64_t v_ts,
                      int64_t v_hs, const int64_t *cache_loc, int64_t n_tokens, int hkv, int lk,
                      int lv, void *k_buffer, int64_t kb_ss, int64_t kb_hs, void *v_buffer,
                      int64_t vb_ss, int64_t vb_hs, int64_t num_slots, void *stream) {
  if (n_tokens < 0 || hkv <= 0 || lk <= 0 || lk % 8 || (v && (lv <= 0 || lv % 8)))
    return set_error(PKX_EINVAL,
                     "set_kv_buffer: n_tokens >= 0, hkv > 0, lk (and lv) positive multiples of 8");
  if (num_slots < 0) return set_error(PKX_EINVAL, "set_kv_buffer: negative num_slots");
  if (n_tokens == 0) return PKX_OK;
  if (!cache_loc || !aligned(cache_loc, 8))
    return set_error(PKX_EINVAL, "set_kv_buffer: cache_loc null or misaligned");
  int rc;
  if ((rc = check_rows("k", k, k_ts, k_hs)) != PKX_OK) return rc;
  if ((rc = check_rows("k_buffer", k_buffer, kb_ss, kb_hs)) != PKX_OK) return rc;
  if (v) {
    if ((rc = check_rows("v", v, v_ts, v_hs)) != PKX_OK) return rc;
    if ((rc = check_rows("v_buffer", v_buffer, vb_ss, vb_hs)) != PKX_OK) return rc;
  }
  return launch_set_kv_buffer(k, k_ts, k_hs, v, v_ts, v_hs, cache_loc, n_tokens, hkv, lk, lv,
                              k_buffer, kb_ss, kb_hs, v_buffer, vb_ss, vb_hs, num_slots,
                              static_cast<cudaStream_t>(stream));
}

int pkx_set_kv_buffer_fp8(const void *k, int64_t k_ts, int64_t k_hs, const void *v,
                          int64_t v_ts, int64_t v_hs, const int64_t *cache_loc, int64_t n_tokens,
                          int hkv, int lk, int lv, float k_scale, float v_scale, int kv_dtype,
                          void *k_buffer, int64_t kb_ss, int64_t kb_hs, void *v_buffer,
                          int64_t vb_ss, int64_t vb_hs, int64_t num_slots, void *stream) {
  if (kv_dtype != kKvFp8E4M3 && kv_dtype != kKvFp8E5M2)
    return set_error(PKX_EINVAL, "set_kv_buffer_fp8: kv_dtype must be an fp8 PKX_KV_* value");
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return set_error(PKX_EINVAL, "set_kv_buffer_fp8: scales must be positive and finite");
  if (n_tokens < 0 || hkv <= 0 || lk <= 0 || lk % 8 || (v && (lv <= 0 || lv % 8)))
    return set_error(PKX_EINVAL,
                     "set_kv_buffer_fp8: n_tokens >= 0, hkv > 0, lk (and lv) multiples of 8");
  if (num_slots < 0) return set_error(PKX_EINVAL, "set_kv_buffer_fp8: negative num_slots");
  if (n_tokens == 0) return PKX_OK;
  if (!cache_loc || !aligned(cache_loc, 8))
    return set_error(PKX_EINVAL, "set_kv_buffer_fp8: cache_loc null or misaligned");
  int rc;
  if ((rc = check_rows("k", k, k_ts, k_hs)) != PKX_OK) return rc;
  if ((rc = check_rows("k_buffer", k_buffer, kb_ss, kb_hs)) != PKX_OK) return rc;
  if (v) {
    if ((rc = check_rows("v", v, v_ts, v_hs)) != PKX_OK) return rc;
    if ((rc = check_rows("v_buffer", v_buffer, vb_ss, vb_hs)) != PKX_OK) return rc;
  }
  return launch_set_kv_buffer_fp8(k, k_ts, k_hs, v, v_ts, v_hs, cache_loc, n_tokens, hkv, lk, lv,
                                  k_scale, v_scale, kv_dtype, k_buffer, kb_ss, kb_hs, v_buffer,
                                  vb_ss, vb_hs, num_slots, static_cast<cudaStream_t>(stream));
}

int pkx_expand_paged_kv_indices(const int32_t *kv_indptr, const int32_t *kv_indices,
                                const int32_t *kv_last_page_len, int page_size, int batch,
                                int32_t *token_indptr, int32_t *token_indices,
                                int64_t token_indices_capacity, void *stream) {
  if (batch < 0 || batch > kGatherMaxBatch)
    return set_error(PKX_EUNSUPPORTED, "expand_paged_kv_indices: batch %d outside [0, %d]",
                     batch, kGatherMaxBatch);
  if (page_size <= 0) return set_error(PKX_EINVAL, "expand_paged_kv_indices: page_size <= 0");
  if (token_indices_capacity < 0)
    return set_error(PKX_EINVAL, "expand_paged_kv_indices: negative capacity");
  if (!token_indptr || !aligned(token_indptr, 4))
    return set_error(PKX_EINVAL, "expand_paged_kv_indices: token_indptr null or misaligned");
  if (batch > 0) {
    if (!kv_indptr || !kv_last_page_len || !aligned(kv_indptr, 4) ||
        !aligned(kv_last_page_len, 4) || (kv_indices && !aligned(kv_indices, 4)))
      return set_error(PKX_EINVAL, "expand_paged_kv_indices: null or misaligned input");
    if (token_indices_capacity > 0 && (!token_indices || !aligned(token_indices, 4)))
      return set_error(PKX_EINVAL, "expand_paged_kv_indices: token_indices null or misaligned");
  }
  return launch_expand_paged(kv_indptr, kv_indices, kv_last_page_len, page_size, batch,
                             token_indptr, token_indices, token_indices_capacity,
                             static_cast<cudaStream_t>(stream));
}

int pkx_create_kv_indices(const int32_t *req_to_token, int64_t req_to_token_rows,
                          int64_t req_to_token_stride, const int64_t *req_pool_indices,
                          const int64_t *paged_kernel_lens, const int64_t *kv_start_idx,
                          int batch, int32_t *kv_indptr, int32_t *kv_indices,
                          int64_t kv_indices_capacity, void *stream) {
  if (batch < 0 || batch > kGatherMaxBatch)
    return set_error(PKX_EUNSUPPORTED, "create_kv_indices: batch %d outside [0, %d]", batch,
                     kGatherMaxBatch);
  if (req_to_token_rows < 0 || req_to_token_stride < 0 || kv_indices_capacity < 0)
    return set_error(PKX_EINVAL, "create_kv_indices: negative table size or capacity");
  if (!kv_indptr || !aligned(kv_indptr, 4))
    return set_error(PKX_EINVAL, "create_kv_indices: kv_indptr null or misaligned");
  if (batch > 0) {
    if (!req_pool_indices || !paged_kernel_lens || !aligned(req_pool_indices, 8) ||
        !aligned(paged_kernel_lens, 8) || (kv_start_idx && !aligned(kv_start_idx, 8)))
      return set_error(PKX_EINVAL, "create_kv_indices: null or misaligned per-sequence array");
    if (kv_indices_capacity > 0 && (!kv_indices || !aligned(kv_indices, 4)))
      return set_error(PKX_EINVAL, "create_kv_indices: kv_indices null or misaligned");
    if (req_to_token_rows > 0 && req_to_token_stride > 0 &&
        (!req_to_token || !aligned(req_to_token, 4)))
      return set_error(PKX_EINVAL, "create_kv_indices: req_to_token null or misaligned");
  }
  return launch_create_kv_indices(req_to_token, req_to_token_rows, req_to_token_stride,
                                  req_pool_indices, paged_kernel_lens, kv_start_idx, batch,
                                  kv_indptr, kv_indices, kv_indices_capacity,
                                  static_cast<cudaStream_t>(stream));
}

}  // extern "C"

// ------------------------------------------------------------- 4-bit pool
// The rows of one half (K or V) of a 4-bit pool: codes and block scales.
static int check_fp4_half(const char *name, const void *codes, int64_t ss, int64_t sh,
                          const void *scales, int64_t s_ss, int64_t s_sh, int code_align,
                          int scale_align) {
  if (!codes || !scales) return set_error(PKX_EINVAL, "%s codes or block scales null", name);
  if (!aligned(codes, code_align) || ss < 0 || sh < 0 || ss % code_align || sh % code_align)
    return set_error(PKX_EINVAL, "%s codes: base and strides (%lld, %lld) must be multiples of %d "
                     "bytes", name, (long long)ss, (long long)sh, code_align);
  if (!aligned(scales, scale_align) || s_ss < 0 || s_sh < 0 || s_ss % scale_align ||
      s_sh % scale_align)
    return set_error(PKX_EINVAL, "%s block scales: base and strides (%lld, %lld) must be "
                     "multiples of %d bytes", name, (long long)s_ss, (long long)s_sh, scale_align);
  return PKX_OK;
}

static int check_fp4_scales(float k_scale, float v_scale) {
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return set_error(PKX_EINVAL, "k_scale and v_scale must be positive and finite");
  return PKX_OK;
}

// Head dims, pool rows and scales of an attention call over a 4-bit pool.
static int check_fp4_attention(int hq, int hkv, int lq, int lv, float k_scale,
                               float v_scale) {
  int rc;
  if ((rc = check_heads(hq, hkv, lq, lv))) return rc;
  if (!((lq == 64 && lv == 64) || (lq == 128 && lv == 128)))
    return set_error(PKX_EUNSUPPORTED, "a 4-bit pool is built for Lq = Lv = 64 or 128");
  if ((rc = check_fp4_scales(k_scale, v_scale))) return rc;
  // the scales join fp32 factors of logits, sums and outputs, which they must
  // not drive out of range (extend divides P of its new rows by v_scale)
  if (k_scale < 0x1p-64f || k_scale > 0x1p64f || v_scale < 0x1p-64f || v_scale > 0x1p64f)
    return set_error(PKX_EUNSUPPORTED, "k_scale and v_scale of attention over a 4-bit pool must "
                     "lie in [2^-64, 2^64]");
  return PKX_OK;
}

static int check_fp4_attention_rows(const Fp4Pool &p, int d) {
  int rc;
  if ((rc = check_fp4_half("k_buffer", p.k, p.k_ss, p.k_sh, p.ks, p.ks_ss, p.ks_sh, 16, d / 16)))
    return rc;
  if ((rc = check_fp4_half("v_buffer", p.v, p.v_ss, p.v_sh, p.vs, p.vs_ss, p.vs_sh, 16, d / 16)))
    return rc;
  const int64_t lim = 1ll << 31;
  if (p.k_ss >= lim || p.v_ss >= lim || p.ks_ss >= lim || p.vs_ss >= lim)
    return set_error(PKX_EUNSUPPORTED, "a 4-bit pool's slot strides must be below 2^31 bytes");
  if (p.num_slots <= 0) return set_error(PKX_EINVAL, "num_slots must be positive");
  if (p.num_slots >= lim) return set_error(PKX_EUNSUPPORTED, "2^31 pool slots or more");
  return PKX_OK;
}

// First tokens that stay visible need no window to be valid, but no custom
// mask replaces their causal term.
static int check_first_tokens(int first_tokens, int window, bool masked) {
  if (first_tokens < 0) return set_error(PKX_EINVAL, "negative first_tokens");
  if (first_tokens > 0 && window > 0 && masked)
    return set_error(PKX_EUNSUPPORTED, "first_tokens with a custom mask is not built");
  return PKX_OK;
}

static int check_streaming(int hq, int hkv, int lq, int lv, int window, int first_tokens) {
  int rc;
  if ((rc = check_heads(hq, hkv, lq, lv))) return rc;
  if (!((lq == 64 && lv == 64) || (lq == 128 && lv == 128)))
    return set_error(PKX_EUNSUPPORTED, "the streaming window is built for Lq = Lv = 64 or 128");
  return check_first_tokens(first_tokens, window, false);
}

static Fp4Pool fp4_pool(const void *k, const void *ks, const void *v, const void *vs,
                        int64_t k_ss, int64_t k_sh, int64_t ks_ss, int64_t ks_sh, int64_t v_ss,
                        int64_t v_sh, int64_t vs_ss, int64_t vs_sh, int64_t num_slots) {
  auto w = [](const void *x) { return static_cast<uint8_t *>(const_cast<void *>(x)); };
  return Fp4Pool{w(k), w(ks), w(v), w(vs), k_ss, k_sh, ks_ss, ks_sh, v_ss, v_sh, vs_ss, vs_sh,
                 num_slots};
}

extern "C" {

int pkx_set_kv_buffer_fp4(const void *k, int64_t k_ts, int64_t k_hs, const void *v, int64_t v_ts,
                          int64_t v_hs, const int64_t *cache_loc, int64_t n_tokens, int hkv,
                          int lk, int lv, float k_scale, float v_scale, void *k_buffer,
                          int64_t kb_ss, int64_t kb_sh, void *k_block_scale, int64_t kbs_ss,
                          int64_t kbs_sh, void *v_buffer, int64_t vb_ss, int64_t vb_sh,
                          void *v_block_scale, int64_t vbs_ss, int64_t vbs_sh, int64_t num_slots,
                          void *stream) {
  int rc;
  if ((rc = check_fp4_scales(k_scale, v_scale))) return rc;
  if (n_tokens < 0 || hkv <= 0 || lk <= 0 || lk % 16 || (v && (lv <= 0 || lv % 16)))
    return set_error(PKX_EINVAL,
                     "set_kv_buffer_fp4: n_tokens >= 0, hkv > 0, lk (and lv) multiples of 16");
  if (num_slots < 0) return set_error(PKX_EINVAL, "set_kv_buffer_fp4: negative num_slots");
  if (n_tokens == 0) return PKX_OK;
  if (!cache_loc || !aligned(cache_loc, 8))
    return set_error(PKX_EINVAL, "set_kv_buffer_fp4: cache_loc null or misaligned");
  if ((rc = check_rows("k", k, k_ts, k_hs))) return rc;
  if ((rc = check_fp4_half("k_buffer", k_buffer, kb_ss, kb_sh, k_block_scale, kbs_ss, kbs_sh, 8,
                           1)))
    return rc;
  if (v) {
    if ((rc = check_rows("v", v, v_ts, v_hs))) return rc;
    if ((rc = check_fp4_half("v_buffer", v_buffer, vb_ss, vb_sh, v_block_scale, vbs_ss, vbs_sh, 8,
                             1)))
      return rc;
  }
  return launch_set_kv_buffer_fp4(k, k_ts, k_hs, v, v_ts, v_hs, cache_loc, n_tokens, hkv, lk, lv,
                                  k_scale, v_scale,
                                  fp4_pool(k_buffer, k_block_scale, v_buffer, v_block_scale, kb_ss,
                                           kb_sh, kbs_ss, kbs_sh, vb_ss, vb_sh, vbs_ss, vbs_sh,
                                           num_slots),
                                  static_cast<cudaStream_t>(stream));
}

int pkx_get_kv_buffer_fp4(const void *k_buffer, int64_t kb_ss, int64_t kb_sh,
                          const void *k_block_scale, int64_t kbs_ss, int64_t kbs_sh,
                          const void *v_buffer, int64_t vb_ss, int64_t vb_sh,
                          const void *v_block_scale, int64_t vbs_ss, int64_t vbs_sh,
                          int64_t num_slots, const int32_t *kv_indices, int64_t n_rows, int hkv,
                          int lk, int lv, float k_scale, float v_scale, void *k, int64_t k_ts,
                          int64_t k_hs, void *v, int64_t v_ts, int64_t v_hs, void *stream) {
  int rc;
  if ((rc = check_fp4_scales(k_scale, v_scale))) return rc;
  if (n_rows < 0 || hkv <= 0 || lk <= 0 || lk % 16 || (v && (lv <= 0 || lv % 16)))
    return set_error(PKX_EINVAL,
                     "get_kv_buffer_fp4: n_rows >= 0, hkv > 0, lk (and lv) multiples of 16");
  if (num_slots < 0) return set_error(PKX_EINVAL, "get_kv_buffer_fp4: negative num_slots");
  if (n_rows == 0) return PKX_OK;
  if (!kv_indices || !aligned(kv_indices, 4))
    return set_error(PKX_EINVAL, "get_kv_buffer_fp4: kv_indices null or misaligned");
  if ((rc = check_rows("k", k, k_ts, k_hs))) return rc;
  if ((rc = check_fp4_half("k_buffer", k_buffer, kb_ss, kb_sh, k_block_scale, kbs_ss, kbs_sh, 8,
                           1)))
    return rc;
  if (v) {
    if ((rc = check_rows("v", v, v_ts, v_hs))) return rc;
    if ((rc = check_fp4_half("v_buffer", v_buffer, vb_ss, vb_sh, v_block_scale, vbs_ss, vbs_sh, 8,
                             1)))
      return rc;
  }
  return launch_get_kv_buffer_fp4(
      fp4_pool(k_buffer, k_block_scale, v_buffer, v_block_scale, kb_ss, kb_sh, kbs_ss, kbs_sh,
               vb_ss, vb_sh, vbs_ss, vbs_sh, num_slots),
      kv_indices, n_rows, hkv, lk, lv, k_scale, v_scale, k, k_ts, k_hs, v, v_ts, v_hs,
      static_cast<cudaStream_t>(stream));
}

size_t pkx_decode_fp4_workspace_size(int batch, int hq, int hkv, int lq, int lv) {
  if (batch < 0 || hkv <= 0 || hq <= 0 || hq % hkv || hq / hkv > kBlockM || lq != lv ||
      (lq != 64 && lq != 128))
    return 0;
  return fp4_decode_workspace(hq, hkv, lq);
}

int pkx_decode_attention_fwd_fp4(
    const void *q, void *o, const void *k_buffer, const void *k_block_scale, const void *v_buffer,
    const void *v_block_scale, const int32_t *kv_indptr, const int32_t *kv_indices, int batch,
    int hq, int hkv, int lq, int lv, int64_t kb_ss, int64_t kb_sh, int64_t kbs_ss, int64_t kbs_sh,
    int64_t vb_ss, int64_t vb_sh, int64_t vbs_ss, int64_t vbs_sh, int64_t num_slots,
    float sm_scale, float logit_cap, int sliding_window, int first_tokens, float k_scale,
    float v_scale, float *lse_out, void *workspace, size_t workspace_bytes, void *stream) {
  Fp4DecodeArgs a{};
  int rc;
  a.pool = fp4_pool(k_buffer, k_block_scale, v_buffer, v_block_scale, kb_ss, kb_sh, kbs_ss,
                    kbs_sh, vb_ss, vb_sh, vbs_ss, vbs_sh, num_slots);
  if (batch < 0) return set_error(PKX_EINVAL, "negative batch");
  if ((rc = check_fp4_attention(hq, hkv, lq, lv, k_scale, v_scale))) return rc;
  if ((rc = check_scalars(sm_scale, logit_cap))) return rc;
  if (first_tokens < 0) return set_error(PKX_EINVAL, "negative first_tokens");
  if (batch == 0) return PKX_OK;
  if ((rc = check_rows("q", q, 8, 8))) return rc;
  if ((rc = check_rows("o", o, 8, 8))) return rc;
  if ((rc = check_fp4_attention_rows(a.pool, lq))) return rc;
  if (!kv_indptr || !aligned(kv_indptr, 4))
    return set_error(PKX_EINVAL, "kv_indptr null or misaligned");
  if (kv_indices && !aligned(kv_indices, 4)) return set_error(PKX_EINVAL, "kv_indices misaligned");
  if (lse_out && !aligned(lse_out, 4)) return set_error(PKX_EINVAL, "lse_out misaligned");
  a.q = q; a.o = o; a.lse = lse_out;
  a.kv_indptr = kv_indptr; a.kv_indices = kv_indices;
  a.batch = batch; a.hq = hq; a.hkv = hkv; a.d = lq;
  a.sm_scale = sm_scale; a.logit_cap = logit_cap;
  a.window = sliding_window; a.first_tokens = first_tokens;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_decode_fp4(a);
}

int pkx_extend_attention_fwd_fp4(
    const void *q_extend, const void *k_extend, const void *v_extend, void *o_extend,
    const void *k_buffer, const void *k_block_scale, const void *v_buffer,
    const void *v_block_scale, const int32_t *qo_indptr, const int32_t *kv_indptr,
    const int32_t *kv_indices, int batch, int num_q_tokens, int hq, int hkv, int lq, int lv,
    int64_t ke_st, int64_t ke_sh, int64_t ve_st, int64_t ve_sh, int64_t kb_ss, int64_t kb_sh,
    int64_t kbs_ss, int64_t kbs_sh, int64_t vb_ss, int64_t vb_sh, int64_t vbs_ss, int64_t vbs_sh,
    int64_t num_slots, float sm_scale, float logit_cap, int sliding_window, int first_tokens,
    const uint8_t *custom_mask, const int32_t *mask_indptr, const float *sinks, float k_scale,
    float v_scale, float *lse_out, void *workspace, size_t workspace_bytes, void *stream) {
  int rc;
  if ((rc = check_fp4_attention(hq, hkv, lq, lv, k_scale, v_scale))) return rc;
  if ((rc = check_first_tokens(first_tokens, sliding_window, custom_mask != nullptr))) return rc;
  AttnArgs a{};
  bool done;
  rc = two_stage_args(a, q_extend, k_extend, v_extend, o_extend, k_buffer, v_buffer, qo_indptr,
                      kv_indptr, kv_indices, batch, num_q_tokens, hq, hkv, lq, lv, ke_st, ke_sh,
                      ve_st, ve_sh, kb_ss, kb_sh, vb_ss, vb_sh, num_slots, sm_scale, logit_cap,
                      sliding_window, custom_mask, mask_indptr, sinks, kKvBf16, 1.f, 1.f, lse_out,
                      &done);
  if (rc != PKX_OK || done) return rc;
  const Fp4Pool pool = fp4_pool(k_buffer, k_block_scale, v_buffer, v_block_scale, kb_ss, kb_sh,
                                kbs_ss, kbs_sh, vb_ss, vb_sh, vbs_ss, vbs_sh, num_slots);
  if ((rc = check_fp4_attention_rows(pool, lq))) return rc;
  a.kv_fmt = kKvFp4;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.k_bscale = k_block_scale; a.v_bscale = v_block_scale;
  a.kbs_ss = kbs_ss; a.kbs_sh = kbs_sh; a.vbs_ss = vbs_ss; a.vbs_sh = vbs_sh;
  a.first_tokens = first_tokens;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attention(a);
}

int pkx_extend_attention_fwd_streaming(
    const void *q_extend, const void *k_extend, const void *v_extend, void *o_extend,
    const void *k_buffer, const void *v_buffer, const int32_t *qo_indptr,
    const int32_t *kv_indptr, const int32_t *kv_indices, int batch, int num_q_tokens, int hq,
    int hkv, int lq, int lv, int64_t ke_st, int64_t ke_sh, int64_t ve_st, int64_t ve_sh,
    int64_t kb_ss, int64_t kb_sh, int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale,
    float logit_cap, int sliding_window, int first_tokens, const float *sinks, float *lse_out,
    void *workspace, size_t workspace_bytes, void *stream) {
  int rc;
  if ((rc = check_streaming(hq, hkv, lq, lv, sliding_window, first_tokens))) return rc;
  AttnArgs a{};
  bool done;
  rc = two_stage_args(a, q_extend, k_extend, v_extend, o_extend, k_buffer, v_buffer, qo_indptr,
                      kv_indptr, kv_indices, batch, num_q_tokens, hq, hkv, lq, lv, ke_st, ke_sh,
                      ve_st, ve_sh, kb_ss, kb_sh, vb_ss, vb_sh, num_slots, sm_scale, logit_cap,
                      sliding_window, nullptr, nullptr, sinks, kKvBf16, 1.f, 1.f, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  a.first_tokens = first_tokens;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attention(a);
}

int pkx_decode_attention_fwd_streaming(
    const void *q, void *o, const void *k_buffer, const void *v_buffer, const int32_t *kv_indptr,
    const int32_t *kv_indices, int batch, int hq, int hkv, int lq, int lv, int64_t kb_ss,
    int64_t kb_sh, int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale,
    float logit_cap, int sliding_window, int first_tokens, float *lse_out, void *workspace,
    size_t workspace_bytes, void *stream) {
  int rc;
  if ((rc = check_streaming(hq, hkv, lq, lv, sliding_window, first_tokens))) return rc;
  AttnArgs a{};
  bool done;
  rc = decode_args(a, q, o, k_buffer, v_buffer, kv_indptr, kv_indices, batch, hq, hkv, lq, lv,
                   kb_ss, kb_sh, vb_ss, vb_sh, num_slots, sm_scale, logit_cap, sliding_window,
                   kKvBf16, 1.f, 1.f, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  a.first_tokens = first_tokens;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_attention(a);
}

}  // extern "C"

// ------------------------------------ a decode step around the paged pool
static int check_pool_format(const char *what, int kv_dtype, float k_scale, float v_scale) {
  if (kv_dtype == kKvBf16) return PKX_OK;
  if (kv_dtype != kKvFp8E4M3 && kv_dtype != kKvFp8E5M2)
    return set_error(PKX_EINVAL, "%s: kv_dtype %d is not a PKX_KV_* value", what, kv_dtype);
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return set_error(PKX_EINVAL, "%s: k_scale and v_scale must be positive and finite", what);
  return PKX_OK;
}

// Heads of the forms built for Lq = Lv = 64 or 128.
static int check_equal_heads(const char *what, int hq, int hkv, int lq, int lv) {
  int rc;
  if ((rc = check_heads(hq, hkv, lq, lv))) return rc;
  if (lq != lv || (lq != 64 && lq != 128))
    return set_error(PKX_EUNSUPPORTED, "%s is built for Lq = Lv = 64 or 128", what);
  return PKX_OK;
}

// Rows of an fp8 pool that are copied 16 bytes at a time.
static int check_fp8_strides(int kv_dtype, int64_t kb_ss, int64_t kb_sh, int64_t vb_ss,
                             int64_t vb_sh) {
  if (kv_dtype != kKvBf16 && ((kb_ss | kb_sh | vb_ss | vb_sh) & 15))
    return set_error(PKX_EINVAL, "the strides of an fp8 pool must be multiples of 16 bytes");
  return PKX_OK;
}

// Pages of one call: a selection fits the listing kernel's shared memory.
constexpr int kMaxTopK = 4096;
static int check_top_k(int top_k) {
  if (top_k <= 0) return set_error(PKX_EINVAL, "top_k must be positive");
  if (top_k > kMaxTopK) return set_error(PKX_EUNSUPPORTED, "top_k %d > %d", top_k, kMaxTopK);
  return PKX_OK;
}

// What the two listed decode forms share, after decode_args().
static ListedArgs listed_args(const AttnArgs &a, void *workspace, size_t workspace_bytes,
                              void *stream) {
  ListedArgs l{};
  l.q = a.q; l.o = a.o; l.lse = a.lse;
  l.k_buf = a.k_buf; l.v_buf = a.v_buf;
  l.kb_ss = a.kb_ss; l.kb_sh = a.kb_sh; l.vb_ss = a.vb_ss; l.vb_sh = a.vb_sh;
  l.num_slots = a.num_slots;
  l.kv_indptr = a.kv_indptr;
  l.kv_indices = static_cast<const int32_t *>(a.kv_indices);
  l.batch = a.batch; l.hq = a.hq; l.hkv = a.hkv; l.d = a.lq;
  l.sm_scale = a.sm_scale; l.logit_cap = a.logit_cap;
  l.kv_fmt = a.kv_fmt; l.k_scale = a.k_scale; l.v_scale = a.v_scale;
  l.workspace = workspace; l.workspace_bytes = workspace_bytes;
  l.stream = static_cast<cudaStream_t>(stream);
  return l;
}

extern "C" {

int pkx_qk_norm_rope(const void *q, int64_t q_ts, int64_t q_hs, const void *k, int64_t k_ts,
                     int64_t k_hs, const void *v, int64_t v_ts, int64_t v_hs, int64_t n_tokens,
                     int hq, int hkv, int d, const int64_t *positions, int num_axes,
                     const uint8_t *pair_axis, const float *cos_sin, int64_t max_position,
                     int rotary_dim, int interleaved, const void *q_weight, const void *k_weight,
                     float eps, float weight_offset, void *q_out, int64_t qo_ts, int64_t qo_hs,
                     void *k_out, int64_t ko_ts, int64_t ko_hs, const int64_t *cache_loc,
                     void *k_buffer, int64_t kb_ss, int64_t kb_sh, void *v_buffer, int64_t vb_ss,
                     int64_t vb_sh, int64_t num_slots, int kv_dtype, float k_scale, float v_scale,
                     void *stream) {
  int rc;
  if (n_tokens < 0 || hq <= 0 || hkv <= 0)
    return set_error(PKX_EINVAL, "qk_norm_rope: n_tokens >= 0, hq > 0 and hkv > 0");
  if (n_tokens >= (1ll << 40) || hq > (1 << 20) || hkv > (1 << 20))
    return set_error(PKX_EUNSUPPORTED, "qk_norm_rope: 2^40 tokens or more than 2^20 heads");
  if (d <= 0 || d % 8) return set_error(PKX_EINVAL, "qk_norm_rope: d must be a multiple of 8");
  if (d > 256) return set_error(PKX_EUNSUPPORTED, "qk_norm_rope: d %d > 256", d);
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 16)
    return set_error(PKX_EINVAL, "qk_norm_rope: rotary_dim must be a multiple of 16 up to d");
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(weight_offset))
    return set_error(PKX_EINVAL, "qk_norm_rope: eps must be finite and not negative, "
                                 "weight_offset finite");
  if (n_tokens == 0) return PKX_OK;
  if (v && !cache_loc)
    return set_error(PKX_EINVAL, "qk_norm_rope: v is only written to the pool: cache_loc is null");
  if (rotary_dim > 0) {
    if (!positions || !aligned(positions, 8))
      return set_error(PKX_EINVAL, "qk_norm_rope: positions null or misaligned");
    if (!cos_sin || !aligned(cos_sin, 16) || max_position <= 0)
      return set_error(PKX_EINVAL, "qk_norm_rope: cos_sin null, misaligned or without rows");
    if (num_axes <= 0 || (num_axes > 1 && !pair_axis))
      return set_error(PKX_EINVAL, "qk_norm_rope: several axes need pair_axis");
  }
  if ((rc = check_rows("q", q, q_ts, q_hs))) return rc;
  if ((rc = check_rows("k", k, k_ts, k_hs))) return rc;
  if ((rc = check_rows("q_out", q_out, qo_ts, qo_hs))) return rc;
  if ((rc = check_rows("k_out", k_out, ko_ts, ko_hs))) return rc;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16))
    return set_error(PKX_EINVAL, "qk_norm_rope: weights must be 16-byte aligned");
  if (cache_loc) {
    if ((rc = check_pool_format("qk_norm_rope", kv_dtype, k_scale, v_scale))) return rc;
    if (!aligned(cache_loc, 8)) return set_error(PKX_EINVAL, "qk_norm_rope: cache_loc misaligned");
    if (num_slots < 0) return set_error(PKX_EINVAL, "qk_norm_rope: negative num_slots");
    if ((rc = check_rows("k_buffer", k_buffer, kb_ss, kb_sh))) return rc;
    if (v) {
      if ((rc = check_rows("v", v, v_ts, v_hs))) return rc;
      if ((rc = check_rows("v_buffer", v_buffer, vb_ss, vb_sh))) return rc;
    }
  }
  RopeArgs a{};
  auto in = [](const void *p) { return static_cast<const uint16_t *>(p); };
  a.q = in(q); a.k = in(k); a.v = in(v);
  a.q_out = static_cast<uint16_t *>(q_out); a.k_out = static_cast<uint16_t *>(k_out);
  a.q_ts = q_ts; a.q_hs = q_hs; a.k_ts = k_ts; a.k_hs = k_hs; a.v_ts = v_ts; a.v_hs = v_hs;
  a.qo_ts = qo_ts; a.qo_hs = qo_hs; a.ko_ts = ko_ts; a.ko_hs = ko_hs;
  a.n_tokens = n_tokens;
  a.hq = hq; a.hkv = hkv; a.d = d; a.rotary = rotary_dim;
  a.positions = positions; a.axes = num_axes;
  a.pair_axis = pair_axis; a.cos_sin = cos_sin; a.max_position = max_position;
  a.interleaved = interleaved;
  a.q_weight = in(q_weight); a.k_weight = in(k_weight);
  a.eps = eps; a.weight_offset = weight_offset;
  a.cache_loc = cache_loc;
  a.k_buffer = k_buffer; a.v_buffer = v_buffer;
  a.kb_ss = kb_ss; a.kb_hs = kb_sh; a.vb_ss = vb_ss; a.vb_hs = vb_sh;
  a.num_slots = num_slots;
  a.kv_fmt = cache_loc ? kv_dtype : kKvBf16;
  a.k_scale = k_scale; a.v_scale = v_scale;
  return launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream));
}

int pkx_update_page_bounds(const void *k_buffer, int64_t kb_ss, int64_t kb_sh, int kv_dtype,
                           int page_size, int64_t num_pages, int hkv, int d,
                           const int32_t *page_ids, const int32_t *page_lens, int64_t n_pages,
                           void *bounds, void *stream) {
  int rc;
  if ((rc = check_pool_format("update_page_bounds", kv_dtype, 1.f, 1.f))) return rc;
  if (page_size <= 0 || num_pages < 0 || n_pages < 0)
    return set_error(PKX_EINVAL, "update_page_bounds: page_size > 0, no negative counts");
  if (hkv <= 0 || d <= 0 || d % 8)
    return set_error(PKX_EINVAL, "update_page_bounds: hkv > 0, d a multiple of 8");
  if (hkv > (1 << 20) || d > (1 << 10))
    return set_error(PKX_EUNSUPPORTED, "update_page_bounds: more than 2^20 heads or d > 1024");
  if (page_size > (1 << 30))
    return set_error(PKX_EUNSUPPORTED, "update_page_bounds: more than 2^30 slots a page");
  if (n_pages == 0) return PKX_OK;
  if ((rc = check_rows("k_buffer", k_buffer, kb_ss, kb_sh))) return rc;
  if (!bounds || !aligned(bounds, 16))
    return set_error(PKX_EINVAL, "update_page_bounds: bounds null or misaligned");
  if (!page_ids || !aligned(page_ids, 4) || !aligned(page_lens, 4))
    return set_error(PKX_EINVAL, "update_page_bounds: page_ids null or misaligned");
  return launch_update_page_bounds(k_buffer, kb_ss, kb_sh, kv_dtype, page_size, num_pages, hkv, d,
                                   page_ids, page_lens, n_pages, bounds,
                                   static_cast<cudaStream_t>(stream));
}

size_t pkx_select_pages_workspace_size(int batch, int hkv, int64_t n_indices) {
  if (batch < 0 || hkv <= 0 || n_indices < 0) return 0;
  return select_pages_workspace(batch, hkv, n_indices);
}

int pkx_select_pages(const void *q, const void *bounds, int64_t num_pages,
                     const int32_t *kv_indptr, const int32_t *kv_indices, int64_t n_indices,
                     int batch, int hq, int hkv, int d, int top_k, int first_pages, int last_pages,
                     int32_t *selected, void *workspace, size_t workspace_bytes, void *stream) {
  int rc;
  if (batch < 0) return set_error(PKX_EINVAL, "negative batch");
  if ((rc = check_equal_heads("select_pages", hq, hkv, d, d))) return rc;
  if ((rc = check_top_k(top_k))) return rc;
  if (first_pages < 0 || last_pages < 0 || (int64_t)first_pages + last_pages > top_k)
    return set_error(PKX_EINVAL, "select_pages: first_pages + last_pages must be in [0, top_k]");
  if (num_pages < 0 || n_indices < 0)
    return set_error(PKX_EINVAL, "select_pages: negative count of pages");
  if (n_indices > (1ll << 30))
    return set_error(PKX_EUNSUPPORTED, "select_pages: more than 2^30 pages in one call");
  if (batch == 0) return PKX_OK;
  if ((rc = check_rows("q", q, 8, 8))) return rc;
  if (num_pages > 0 && (!bounds || !aligned(bounds, 16)))
    return set_error(PKX_EINVAL, "select_pages: bounds null or misaligned");
  if (!kv_indptr || !aligned(kv_indptr, 4))
    return set_error(PKX_EINVAL, "kv_indptr null or misaligned");
  if (n_indices > 0 && (!kv_indices || !aligned(kv_indices, 4)))
    return set_error(PKX_EINVAL, "kv_indices null or misaligned");
  if (!selected || !aligned(selected, 4))
    return set_error(PKX_EINVAL, "select_pages: selected null or misaligned");
  const size_t need = select_pages_workspace(batch, hkv, n_indices);
  if (!workspace || workspace_bytes < need)
    return set_error(PKX_EWORKSPACE, "workspace of %zu bytes given, %zu needed", workspace_bytes,
                     need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return set_error(PKX_EINVAL, "workspace must be 256-byte aligned");
  SelectArgs a{};
  a.q = q; a.bounds = bounds; a.num_pages = num_pages;
  a.kv_indptr = kv_indptr; a.kv_indices = kv_indices; a.n_indices = n_indices;
  a.batch = batch; a.hq = hq; a.hkv = hkv; a.d = d;
  a.top_k = top_k; a.first_pages = first_pages; a.last_pages = last_pages;
  a.selected = selected;
  a.workspace = workspace; a.workspace_bytes = workspace_bytes;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_select_pages(a);
}

size_t pkx_decode_pages_workspace_size(int batch, int hq, int hkv, int lq, int lv, int page_size,
                                       int top_k) {
  if (batch < 0 || hkv <= 0 || hq <= 0 || hq % hkv || hq / hkv > kBlockM || lq != lv ||
      (lq != 64 && lq != 128) || page_size <= 0 || top_k <= 0 || top_k > kMaxTopK ||
      (int64_t)top_k * page_size > kMaxListedKeys)
    return 0;
  return pages_decode_workspace(batch, hq, hkv, lq, page_size, top_k, num_sms_current_device());
}

int pkx_decode_attention_fwd_pages(
    const void *q, void *o, const void *k_buffer, const void *v_buffer, const int32_t *kv_indptr,
    const int32_t *kv_indices, int64_t n_indices, const int32_t *kv_last_page_len, int page_size,
    const int32_t *selected, int top_k, int batch, int hq, int hkv, int lq, int lv, int64_t kb_ss,
    int64_t kb_sh, int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale,
    float logit_cap, int kv_dtype, float k_scale, float v_scale, float *lse_out, void *workspace,
    size_t workspace_bytes, void *stream) {
  int rc;
  if ((rc = check_equal_heads("decode over selected pages", hq, hkv, lq, lv))) return rc;
  if ((rc = check_top_k(top_k))) return rc;
  if (page_size <= 0) return set_error(PKX_EINVAL, "page_size must be positive");
  if (n_indices < 0) return set_error(PKX_EINVAL, "negative n_indices");
  AttnArgs a{};
  bool done;
  rc = decode_args(a, q, o, k_buffer, v_buffer, kv_indptr, kv_indices, batch, hq, hkv, lq, lv,
                   kb_ss, kb_sh, vb_ss, vb_sh, num_slots, sm_scale, logit_cap, -1, kv_dtype,
                   k_scale, v_scale, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  if ((rc = check_fp8_strides(kv_dtype, kb_ss, kb_sh, vb_ss, vb_sh))) return rc;
  if (n_indices > 0 && !kv_indices) return set_error(PKX_EINVAL, "kv_indices is null");
  if (!kv_last_page_len || !aligned(kv_last_page_len, 4))
    return set_error(PKX_EINVAL, "kv_last_page_len null or misaligned");
  if (!selected || !aligned(selected, 4))
    return set_error(PKX_EINVAL, "selected null or misaligned");
  if (num_slots >= INT32_MAX) return set_error(PKX_EUNSUPPORTED, "more than 2^31 pool slots");
  ListedArgs l = listed_args(a, workspace, workspace_bytes, stream);
  l.last_page_len = kv_last_page_len;
  l.selected = selected;
  l.page_size = page_size;
  l.top_k = top_k;
  l.n_indices = n_indices;
  return launch_decode_pages(l);
}

size_t pkx_decode_shared_workspace_size(int batch, int num_groups, int hq, int hkv, int lq,
                                        int lv) {
  if (batch < 0 || num_groups < 0 || hkv <= 0 || hq <= 0 || hq % hkv || hq / hkv > kBlockM ||
      lq != lv || (lq != 64 && lq != 128))
    return 0;
  return shared_decode_workspace(batch, num_groups, hq, hkv, lq, num_sms_current_device());
}

int pkx_decode_attention_fwd_shared(
    const void *q, void *o, const void *k_buffer, const void *v_buffer, const int32_t *kv_indptr,
    const int32_t *kv_indices, int64_t n_indices, const int32_t *group_indptr,
    const int32_t *shared_lens, int num_groups, int batch, int hq, int hkv, int lq, int lv,
    int64_t kb_ss, int64_t kb_sh, int64_t vb_ss, int64_t vb_sh, int64_t num_slots, float sm_scale,
    float logit_cap, int kv_dtype, float k_scale, float v_scale, float *lse_out, void *workspace,
    size_t workspace_bytes, void *stream) {
  int rc;
  if ((rc = check_equal_heads("decode with shared prefixes", hq, hkv, lq, lv))) return rc;
  if (num_groups < 0 || n_indices < 0)
    return set_error(PKX_EINVAL, "negative num_groups or n_indices");
  if (n_indices > kMaxListedKeys)
    return set_error(PKX_EUNSUPPORTED, "more than 2^31 - 4097 entries of kv_indices");
  AttnArgs a{};
  bool done;
  rc = decode_args(a, q, o, k_buffer, v_buffer, kv_indptr, kv_indices, batch, hq, hkv, lq, lv,
                   kb_ss, kb_sh, vb_ss, vb_sh, num_slots, sm_scale, logit_cap, -1, kv_dtype,
                   k_scale, v_scale, lse_out, &done);
  if (rc != PKX_OK || done) return rc;
  if ((rc = check_fp8_strides(kv_dtype, kb_ss, kb_sh, vb_ss, vb_sh))) return rc;
  if (n_indices > 0 && !kv_indices) return set_error(PKX_EINVAL, "kv_indices is null");
  if (num_groups > 0 && (!group_indptr || !shared_lens || !aligned(group_indptr, 4) ||
                         !aligned(shared_lens, 4)))
    return set_error(PKX_EINVAL, "group_indptr or shared_lens null or misaligned");
  if (num_slots >= INT32_MAX) return set_error(PKX_EUNSUPPORTED, "more than 2^31 pool slots");
  ListedArgs l = listed_args(a, workspace, workspace_bytes, stream);
  l.group_indptr = group_indptr;
  l.shared_lens = shared_lens;
  l.num_groups = num_groups;
  l.n_indices = n_indices;
  return launch_decode_shared(l);
}

}  // extern "C"
