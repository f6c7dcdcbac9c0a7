// C ABI of libstatefulconv.so: host-side validation, then one asynchronous
// launch on the caller's stream. Declarations and their defining passages are
// in include/statefulconv.h.
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <unordered_set>
#include <vector>

#include "statefulconv.h"
#include "kernels.hpp"
#include "attn.hpp"
#include "cca.hpp"
#include "gdn.hpp"

namespace {

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool al8(const void* p) { return ((uintptr_t)p & 7u) == 0; }

// Descriptor checks shared by the depthwise entry points. The state-capacity
// rule follows the PLE layer's _short_conv (cache narrower than the window
// raises); a wider state is a buffer sized for speculative rollback.
sc_status check_conv_desc(const sc_conv_desc* d, int* H) {
  if (d->dtype != SC_DTYPE_F32 && d->dtype != SC_DTYPE_BF16) return SC_ERR_DTYPE;
  if (d->channels < 1 || d->width < 1 || d->dilation < 1) return SC_ERR_INVALID_ARG;
  if (d->width > 8) return SC_ERR_UNSUPPORTED;
  if (d->activation != SC_ACT_NONE && d->activation != SC_ACT_SILU) return SC_ERR_INVALID_ARG;
  if (d->x_row_stride < d->channels || d->out_row_stride < d->channels) return SC_ERR_INVALID_ARG;
  if (d->state_indices_stride < 1) return SC_ERR_INVALID_ARG;
  const int64_t h = (int64_t)(d->width - 1) * d->dilation;
  if (h > (1 << 20)) return SC_ERR_INVALID_ARG;
  if (d->state_len < h) return SC_ERR_STATE_CAPACITY;
  if (d->state_len > (1 << 20)) return SC_ERR_INVALID_ARG;
  if (d->state_layout != SC_STATE_DS && d->state_layout != SC_STATE_SD) return SC_ERR_INVALID_ARG;
  *H = (int)h;
  return SC_OK;
}

// Whether every vector access of the fast kernels is 16-byte aligned.
bool conv_aligned(const sc_conv_desc* d, const void* x, const void* out, const void* w,
                  const void* bias, const void* pool) {
  const int64_t es = d->dtype == SC_DTYPE_BF16 ? 2 : 4;
  return al16(x) && al16(out) && al16(w) && (!bias || al16(bias)) && (!pool || al16(pool)) &&
         (d->x_row_stride * es) % 16 == 0 && (d->out_row_stride * es) % 16 == 0;
}

// Descriptor checks of the optional residual fusion / row map.
sc_status check_fuse(const sc_conv_fuse* f, const sc_conv_desc* d) {
  if (!f) return SC_OK;
  if (f->accumulate != 0 && f->accumulate != 1) return SC_ERR_INVALID_ARG;
  if (f->token_indices && f->num_physical_rows < 1) return SC_ERR_INVALID_ARG;
  if (f->outer_residual && f->outer_row_stride < d->channels) return SC_ERR_INVALID_ARG;
  return SC_OK;
}

// Copies the fusion descriptor into the kernel arguments; out must not be the
// outer residual.
sc_status apply_fuse(const sc_conv_fuse* f, const void* out, sc::ConvArgs& a) {
  if (!f) return SC_OK;
  if (f->outer_residual && f->outer_residual == out) return SC_ERR_INVALID_ARG;
  a.tok = f->token_indices;
  a.phys_rows = f->num_physical_rows;
  a.accumulate = f->accumulate;
  a.outer = f->outer_residual;
  a.outer_rs = f->outer_row_stride;
  return SC_OK;
}

sc_status from_hip(hipError_t e) {
  if (e == hipSuccess) return SC_OK;
  if (e == hipErrorNotSupported) return SC_ERR_UNSUPPORTED;
  return SC_ERR_HIP;
}

// host side of sc_validate_metadata: copies the arrays and checks them
sc_status validate_metadata_host(const int32_t* query_start_loc,
                                 const int32_t* state_indices, int64_t idx_stride,
                                 int32_t batch, int64_t num_tokens, int32_t num_slots,
                                 hipStream_t st) {
  if (query_start_loc) {
    std::vector<int32_t> q((size_t)batch + 1);
    if (hipMemcpyAsync(q.data(), query_start_loc, q.size() * sizeof(int32_t),
                       hipMemcpyDeviceToHost, st) != hipSuccess ||
        hipStreamSynchronize(st) != hipSuccess)
      return SC_ERR_HIP;
    if (q[0] != 0 || (int64_t)q[(size_t)batch] != num_tokens) return SC_ERR_INVALID_ARG;
    for (int32_t r = 0; r < batch; ++r)
      if (q[(size_t)r + 1] < q[(size_t)r]) return SC_ERR_INVALID_ARG;
  }
  if (state_indices) {
    if (idx_stride > (INT64_MAX / 4 - 1) / batch) return SC_ERR_INVALID_ARG;
    const size_t n = (size_t)(batch - 1) * (size_t)idx_stride + 1;
    std::vector<int32_t> s(n);
    if (hipMemcpyAsync(s.data(), state_indices, n * sizeof(int32_t), hipMemcpyDeviceToHost,
                       st) != hipSuccess ||
        hipStreamSynchronize(st) != hipSuccess)
      return SC_ERR_HIP;
    std::unordered_set<int32_t> seen;
    for (int32_t r = 0; r < batch; ++r) {
      const int32_t v = s[(size_t)r * (size_t)idx_stride];
      if (v < 0) continue;
      if (v >= num_slots || !seen.insert(v).second) return SC_ERR_INVALID_ARG;
    }
  }
  return SC_OK;
}

// Descriptor checks shared by the gated delta rule entry points.
sc_status check_gdn_desc(const sc_gdn_desc* d) {
  if (d->dtype != SC_DTYPE_BF16) return SC_ERR_DTYPE;
  if (d->gate_dtype != SC_DTYPE_F32 && d->gate_dtype != SC_DTYPE_BF16) return SC_ERR_DTYPE;
  if (d->num_k_heads < 1 || d->num_v_heads < 1 || d->num_v_heads % d->num_k_heads != 0 ||
      d->head_k_dim < 1 || d->head_v_dim < 1)
    return SC_ERR_INVALID_ARG;
  if (d->qk_l2norm != 0 && d->qk_l2norm != 1) return SC_ERR_INVALID_ARG;
  if (!std::isfinite(d->scale)) return SC_ERR_INVALID_ARG;
  const int64_t kw = (int64_t)d->num_k_heads * d->head_k_dim;
  const int64_t vw = (int64_t)d->num_v_heads * d->head_v_dim;
  if (d->q_row_stride < kw || d->k_row_stride < kw || d->v_row_stride < vw ||
      d->out_row_stride < vw || d->a_row_stride < d->num_v_heads ||
      d->b_row_stride < d->num_v_heads || d->state_indices_stride < 1)
    return SC_ERR_INVALID_ARG;
  if ((d->head_k_dim != 64 && d->head_k_dim != 128) || d->head_v_dim % 16 != 0 ||
      d->q_row_stride % 8 != 0 || d->k_row_stride % 8 != 0 || d->v_row_stride % 8 != 0 ||
      d->out_row_stride % 4 != 0)
    return SC_ERR_UNSUPPORTED;
  // 64 rows are addressed with 32-bit byte offsets
  if (d->q_row_stride >= (1 << 24) || d->k_row_stride >= (1 << 24) ||
      d->v_row_stride >= (1 << 24) || d->out_row_stride >= (1 << 24))
    return SC_ERR_UNSUPPORTED;
  return SC_OK;
}

// Chunks of a prefill; SC_ERR_UNSUPPORTED where its launches do not fit.
sc_status gdn_chunks(const sc_gdn_desc* d, int32_t batch, int64_t num_tokens, int64_t* chunks) {
  if (num_tokens > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  *chunks = num_tokens / sc::kGdnChunk + batch;
  return sc::gdn_prefill_fits(*chunks, batch, d->num_k_heads, d->num_v_heads, d->head_v_dim)
             ? SC_OK
             : SC_ERR_UNSUPPORTED;
}

// Pointers and sizes common to the three calls.
sc_status gdn_args(const sc_gdn_desc* d, const void* q, const void* k, const void* v,
                   const void* a, const void* b, const float* A_log, const float* dt_bias,
                   void* out, float* pool, int32_t num_slots, const int32_t* slots,
                   int32_t batch, sc::GdnArgs* g) {
  if (!q || !k || !v || !a || !b || !A_log || !dt_bias || !out || !slots || (!pool && num_slots > 0))
    return SC_ERR_NULL_ARG;
  if (out == q || out == k || out == v) return SC_ERR_INVALID_ARG;
  if (!al16(q) || !al16(k) || !al16(v) || !al8(out) || !al16(pool)) return SC_ERR_UNSUPPORTED;
  *g = sc::GdnArgs{};
  g->q = q;
  g->k = k;
  g->v = v;
  g->a = a;
  g->b = b;
  g->A_log = A_log;
  g->dt_bias = dt_bias;
  g->out = out;
  g->pool = pool;
  g->slots = slots;
  g->q_rs = d->q_row_stride;
  g->k_rs = d->k_row_stride;
  g->v_rs = d->v_row_stride;
  g->a_rs = d->a_row_stride;
  g->b_rs = d->b_row_stride;
  g->out_rs = d->out_row_stride;
  g->slot_stride = d->state_indices_stride;
  g->scale = d->scale;
  g->hk = d->num_k_heads;
  g->hv = d->num_v_heads;
  g->dk = d->head_k_dim;
  g->dv = d->head_v_dim;
  g->l2norm = d->qk_l2norm;
  g->gate_f32 = d->gate_dtype == SC_DTYPE_F32;
  g->num_slots = num_slots;
  g->batch = batch;
  return SC_OK;
}

// Head counts and sizes shared by the norm and attention calls.
sc_status check_heads(int32_t dtype, int32_t nq, int32_t nkv, int32_t hd) {
  if (dtype != SC_DTYPE_BF16) return SC_ERR_DTYPE;
  if (nq < 1 || nkv < 1 || nq % nkv != 0 || hd < 1) return SC_ERR_INVALID_ARG;
  if (hd != 64 && hd != 128 && hd != 256) return SC_ERR_UNSUPPORTED;
  if (nq > (1 << 20)) return SC_ERR_UNSUPPORTED;
  return SC_OK;
}

sc_status check_paged(const sc_paged_cache* c, int32_t block_size, int64_t multiple,
                      sc::PagedCache* out) {
  if (!c->data) return SC_ERR_NULL_ARG;
  if (c->block_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || block_size < 1)
    return SC_ERR_INVALID_ARG;
  if (c->block_stride % multiple != 0 || c->token_stride % multiple != 0 ||
      c->head_stride % multiple != 0 || ((uintptr_t)c->data & (multiple * 2 - 1)) != 0)
    return SC_ERR_UNSUPPORTED;
  *out = sc::PagedCache{c->data, c->block_stride, c->token_stride, c->head_stride};
  return SC_OK;
}

// A quantised cache; `multiple`: bytes that its loads and stores of codes have.
sc_status check_paged_fp8(const sc_paged_cache_fp8* c, int32_t block_size, int64_t multiple,
                          int64_t scale_multiple, sc::PagedCacheFp8* out) {
  if (!c->data || !c->scale) return SC_ERR_NULL_ARG;
  if (c->block_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || block_size < 1 ||
      c->scale_block_stride < 0 || c->scale_head_stride < 0)
    return SC_ERR_INVALID_ARG;
  if (c->block_stride % multiple != 0 || c->token_stride % multiple != 0 ||
      c->head_stride % multiple != 0 || ((uintptr_t)c->data & (multiple - 1)) != 0 ||
      c->scale_block_stride % scale_multiple != 0 || c->scale_head_stride % scale_multiple != 0 ||
      ((uintptr_t)c->scale & (scale_multiple - 1)) != 0)
    return SC_ERR_UNSUPPORTED;
  *out = sc::PagedCacheFp8{c->data, c->block_stride, c->token_stride, c->head_stride,
                           (uint8_t*)c->scale, c->scale_block_stride, c->scale_head_stride};
  return SC_OK;
}

sc_status check_attn_desc(const sc_paged_attn_desc* d) {
  const sc_status st = check_heads(d->dtype, d->num_q_heads, d->num_kv_heads, d->head_dim);
  if (st != SC_OK) return st;
  const int64_t w = (int64_t)d->num_q_heads * d->head_dim;
  if (d->block_size < 1 || d->num_blocks < 0 || !std::isfinite(d->scale) ||
      d->q_row_stride < w || d->out_row_stride < w || d->block_table_row_stride < 1)
    return SC_ERR_INVALID_ARG;
  if (d->block_size % 16 != 0 || d->q_row_stride % 8 != 0 || d->out_row_stride % 4 != 0)
    return SC_ERR_UNSUPPORTED;
  return SC_OK;
}

void attn_fill(const sc_paged_attn_desc* d, int32_t batch, int32_t q_len, int32_t max_seq_len,
               sc::PagedAttnArgs* a) {
  a->q_rs = d->q_row_stride;
  a->out_rs = d->out_row_stride;
  a->table_rs = d->block_table_row_stride;
  a->scale = d->scale;
  a->batch = batch;
  a->nq_tok = q_len;
  a->nq = d->num_q_heads;
  a->nkv = d->num_kv_heads;
  a->hd = d->head_dim;
  a->block_size = d->block_size;
  a->num_blocks = d->num_blocks;
  a->max_len = max_seq_len;
}

// Sizes of an attention call and its split; workspace bytes through *need.
sc_status attn_sizes(const sc_paged_attn_desc* d, int32_t batch, int32_t q_len,
                     int32_t max_seq_len, sc::PagedAttnArgs* a, int64_t* need, bool fp8 = false) {
  if (batch < 0 || q_len < 0 || max_seq_len < 0) return SC_ERR_INVALID_ARG;
  // rows, row groups and the ends of splits are counted with 32 bits
  if ((int64_t)batch * q_len * d->num_q_heads > 0x7FFFFFFFLL || max_seq_len > (1 << 30))
    return SC_ERR_UNSUPPORTED;
  *a = sc::PagedAttnArgs{};
  *need = 0;
  if (batch == 0 || q_len == 0) return SC_OK;
  attn_fill(d, batch, q_len, max_seq_len, a);
  *need = fp8 ? sc::plan_paged_attn_fp8(a) : sc::plan_paged_attn(a);
  return SC_OK;
}

// The same of an attention call with shared prefixes.
sc_status prefix_sizes(const sc_paged_attn_desc* d, int32_t batch, int32_t q_len,
                       int32_t max_seq_len, int32_t num_groups, int32_t max_prefix_len,
                       bool fp8, sc::PagedAttnArgs* a, int64_t* need) {
  if (batch < 0 || q_len < 0 || max_seq_len < 0 || num_groups < 0 || max_prefix_len < 0 ||
      max_prefix_len > max_seq_len)
    return SC_ERR_INVALID_ARG;
  if ((int64_t)batch * q_len * d->num_q_heads > 0x7FFFFFFFLL || max_seq_len > (1 << 30) ||
      num_groups > (1 << 30))
    return SC_ERR_UNSUPPORTED;
  *a = sc::PagedAttnArgs{};
  *need = 0;
  if (batch == 0 || q_len == 0) return SC_OK;
  attn_fill(d, batch, q_len, max_seq_len, a);
  a->groups = num_groups;
  a->max_prefix = num_groups > 0 ? max_prefix_len : 0;
  const int64_t bytes = sc::plan_paged_attn_prefix(a, fp8);
  if (bytes < 0) return SC_ERR_UNSUPPORTED;
  *need = bytes;
  return SC_OK;
}

sc_status attn_caches(const sc_paged_cache* k, const sc_paged_cache* v, int32_t block_size,
                      sc::PagedAttnArgs* a) {
  const sc_status st = check_paged(k, block_size, 8, &a->kc);
  return st != SC_OK ? st : check_paged(v, block_size, 8, &a->vc);
}
sc_status attn_caches(const sc_paged_cache_fp8* k, const sc_paged_cache_fp8* v, int32_t block_size,
                      sc::PagedAttnArgs* a) {
  const sc_status st = check_paged_fp8(k, block_size, 16, 4, &a->kc8);
  return st != SC_OK ? st : check_paged_fp8(v, block_size, 16, 4, &a->vc8);
}
sc_status norm_caches(const sc_paged_cache* k, const sc_paged_cache* v, int32_t block_size,
                      sc::QkNormArgs* a) {
  const sc_status st = check_paged(k, block_size, 4, &a->kc);
  return st != SC_OK ? st : check_paged(v, block_size, 4, &a->vc);
}
sc_status norm_caches(const sc_paged_cache_fp8* k, const sc_paged_cache_fp8* v, int32_t block_size,
                      sc::QkNormArgs* a) {
  const sc_status st = check_paged_fp8(k, block_size, 4, 1, &a->kc8);
  return st != SC_OK ? st : check_paged_fp8(v, block_size, 4, 1, &a->vc8);
}

// What the attention calls have in common, from their sizes on.
template <class Cache>
sc_status attn_args(const sc_paged_attn_desc* d, const void* q, void* out, const Cache* k_cache,
                    const Cache* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                    int32_t max_seq_len, void* workspace, int64_t workspace_bytes, int64_t need,
                    sc::PagedAttnArgs* a) {
  // no cached token anywhere: the rows are zeros, and no table is needed
  if (!q || !out || !seq_lens || (max_seq_len > 0 && (!block_table || !k_cache || !v_cache)) ||
      (need > 0 && !workspace))
    return SC_ERR_NULL_ARG;
  if (out == q || workspace_bytes < need || (need > 0 && !al16(workspace)))
    return SC_ERR_INVALID_ARG;
  if (max_seq_len > 0) {
    const sc_status st = attn_caches(k_cache, v_cache, d->block_size, a);
    if (st != SC_OK) return st;
    if (d->num_blocks < 1) return SC_ERR_INVALID_ARG;
  }
  if (!al16(q) || !al8(out)) return SC_ERR_UNSUPPORTED;
  a->q = q;
  a->out = out;
  a->table = block_table;
  a->lens = seq_lens;
  a->ws = (float*)workspace;
  return SC_OK;
}

sc_status attn_bounds(const sc_paged_attn_desc* d, int32_t max_blocks, int32_t max_seq_len,
                      int64_t workspace_bytes) {
  return max_blocks < 0 || workspace_bytes < 0 || d->block_table_row_stride < max_blocks ||
                 max_seq_len > (int64_t)max_blocks * d->block_size
             ? SC_ERR_INVALID_ARG
             : SC_OK;
}

// Whether a lane's offset in 16 tokens has 31 bits.
bool tokens_near(const sc::PagedAttnArgs& a) {
  return std::max({a.kc.token_s, a.vc.token_s, a.kc8.token_s, a.vc8.token_s}) < (1 << 26);
}

template <class Cache>
sc_status attn_prefix_call(const sc_paged_attn_desc* desc, const void* q, void* out,
                           const Cache* k_cache, const Cache* v_cache, const int32_t* block_table,
                           int32_t max_blocks, const int32_t* seq_lens,
                           const int32_t* group_start_loc, const int32_t* prefix_lens,
                           int32_t num_groups, int32_t batch, int32_t q_len, int32_t max_seq_len,
                           int32_t max_prefix_len, void* workspace, int64_t workspace_bytes,
                           bool fp8, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  sc_status st = check_attn_desc(desc);
  if (st != SC_OK) return st;
  sc::PagedAttnArgs a;
  int64_t need = 0;
  st = prefix_sizes(desc, batch, q_len, max_seq_len, num_groups, max_prefix_len, fp8, &a, &need);
  if (st != SC_OK) return st;
  if ((st = attn_bounds(desc, max_blocks, max_seq_len, workspace_bytes)) != SC_OK) return st;
  if (batch == 0 || q_len == 0) return SC_OK;
  if (num_groups > 0 && (!group_start_loc || !prefix_lens)) return SC_ERR_NULL_ARG;
  st = attn_args(desc, q, out, k_cache, v_cache, block_table, seq_lens, max_seq_len, workspace,
                 workspace_bytes, need, &a);
  if (st != SC_OK) return st;
  if (!tokens_near(a)) return SC_ERR_UNSUPPORTED;
  a.group_starts = group_start_loc;
  a.prefix_lens = prefix_lens;
  return from_hip(sc::launch_paged_attn_prefix(a, fp8, (hipStream_t)stream));
}

// Norms with either cache: the checks and arguments that both have; with no tokens
// SC_OK and no arguments.
template <class Cache>
sc_status norm_args(const sc_qk_norm_desc* desc, const void* q, const void* k, const void* v,
                    void* q_out, void* k_out, const void* q_weight, const void* k_weight,
                    const void* cos_sin, const int64_t* positions, const int64_t* slots,
                    const Cache* k_cache, const Cache* v_cache, int64_t num_tokens,
                    sc::QkNormArgs* a) {
  const int nq = desc->num_q_heads, nkv = desc->num_kv_heads, hd = desc->head_dim;
  const sc_status st = check_heads(desc->dtype, nq, nkv, hd);
  if (st != SC_OK) return st;
  if (desc->table_dtype != SC_DTYPE_F32 && desc->table_dtype != SC_DTYPE_BF16)
    return SC_ERR_DTYPE;
  const int rot = desc->rotary_dim;
  if (rot < 0 || rot > hd || (desc->interleaved != 0 && desc->interleaved != 1) ||
      !(desc->eps >= 0) || num_tokens < 0 || desc->num_blocks < 0)
    return SC_ERR_INVALID_ARG;
  if (rot % 8 != 0) return SC_ERR_UNSUPPORTED;
  const int64_t qw = (int64_t)nq * hd, kw = (int64_t)nkv * hd;
  if (desc->q_row_stride < qw || desc->k_row_stride < kw || desc->q_out_row_stride < qw ||
      (k_out && desc->k_out_row_stride < kw) || (k_cache && desc->v_row_stride < kw) ||
      (rot > 0 && (desc->table_row_stride < rot || desc->max_position < 1)))
    return SC_ERR_INVALID_ARG;
  if (!k_cache != !v_cache) return SC_ERR_NULL_ARG;
  if (num_tokens == 0) return SC_OK;
  if (!q || !k || !q_out || (rot > 0 && (!cos_sin || !positions)) || (k_cache && (!v || !slots)))
    return SC_ERR_NULL_ARG;
  // in place only on the same rows: a lane then rewrites what it alone has read
  if ((q_out == q && desc->q_out_row_stride != desc->q_row_stride) ||
      (k_out && k_out == k && desc->k_out_row_stride != desc->k_row_stride) || q_out == k ||
      q_out == k_out || k_out == q)
    return SC_ERR_INVALID_ARG;
  if (k_cache) {
    const sc_status bad = norm_caches(k_cache, v_cache, desc->block_size, a);
    if (bad != SC_OK) return bad;
  }
  if (!al8(q) || !al8(k) || !al8(q_out) || !al8(k_out) || !al8(q_weight) || !al8(k_weight) ||
      (k_cache && (!al8(v) || desc->v_row_stride % 4 != 0)) || desc->q_row_stride % 4 != 0 ||
      desc->k_row_stride % 4 != 0 || desc->q_out_row_stride % 4 != 0 ||
      (k_out && desc->k_out_row_stride % 4 != 0))
    return SC_ERR_UNSUPPORTED;
  a->q = q;
  a->k = k;
  a->v = v;
  a->q_out = q_out;
  a->k_out = k_out;
  a->q_w = q_weight;
  a->k_w = k_weight;
  a->table = cos_sin;
  a->positions = positions;
  a->slots = k_cache ? slots : nullptr;
  a->q_rs = desc->q_row_stride;
  a->k_rs = desc->k_row_stride;
  a->v_rs = desc->v_row_stride;
  a->qo_rs = desc->q_out_row_stride;
  a->ko_rs = desc->k_out_row_stride;
  a->table_rs = desc->table_row_stride;
  a->max_pos = desc->max_position;
  a->num_tokens = num_tokens;
  a->eps = desc->eps;
  a->nq = nq;
  a->nkv = nkv;
  a->hd = hd;
  a->rot = rot;
  a->interleaved = desc->interleaved;
  a->table_f32 = desc->table_dtype == SC_DTYPE_F32;
  a->block_size = desc->block_size;
  a->num_blocks = desc->num_blocks;
  return SC_OK;
}

}  // namespace

extern "C" {

int32_t sc_abi_version(void) { return SC_ABI_VERSION; }

sc_status sc_validate_metadata(const int32_t* query_start_loc, const int32_t* state_indices,
                               int64_t idx_stride, int32_t batch, int64_t num_tokens,
                               int32_t num_slots, void* stream) {
  if (batch < 0 || num_tokens < 0 || num_slots < 0 || idx_stride < 1) return SC_ERR_INVALID_ARG;
  if (batch == 0) return SC_OK;
  // the host copies below must not let an allocation failure leave the C ABI
  try {
    return validate_metadata_host(query_start_loc, state_indices, idx_stride, batch,
                                  num_tokens, num_slots, (hipStream_t)stream);
  } catch (const std::bad_alloc&) {
    return SC_ERR_INVALID_ARG;
  }
}


const char* sc_status_string(sc_status s) {
  switch (s) {
    case SC_OK: return "ok";
    case SC_ERR_NULL_ARG: return "a required pointer is NULL";
    case SC_ERR_INVALID_ARG: return "invalid size, stride, enum or grid";
    case SC_ERR_DTYPE: return "unsupported dtype";
    case SC_ERR_STATE_CAPACITY: return "state_len smaller than (width-1)*dilation";
    case SC_ERR_UNSUPPORTED: return "configuration not supported by this library";
    case SC_ERR_HIP: return "HIP runtime error (launch or copy)";
  }
  return "unknown status";
}

sc_status sc_conv_prefill_varlen(const sc_conv_desc* desc, const void* x, void* out,
                                 const void* weight, const void* bias, void* state_pool,
                                 int32_t num_slots, const int32_t* query_start_loc,
                                 const int32_t* state_indices,
                                 const uint8_t* has_initial_state, int32_t batch,
                                 int64_t num_tokens, const sc_ckpt_desc* ckpt,
                                 const sc_conv_fuse* fuse, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  int H = 0;
  sc_status st = check_conv_desc(desc, &H);
  if (st != SC_OK) return st;
  if ((st = check_fuse(fuse, desc)) != SC_OK) return st;
  if (batch < 0 || num_tokens < 0 || num_slots < 0) return SC_ERR_INVALID_ARG;
  int32_t grid = 0;
  if (ckpt && ckpt->grid != 0) {
    // the PLE layer asserts grid >= conv_state_len: a window holds inputs only
    if (ckpt->grid < 0 || ckpt->grid < H) return SC_ERR_INVALID_ARG;
    grid = ckpt->grid;
  }
  // zero work is a no-op before any pointer is required (empty tensors may
  // carry NULL data pointers), as the GDN core returns early on zero tokens
  if (batch == 0 || num_tokens == 0) return SC_OK;
  if (!x || !out || !weight || !query_start_loc || !state_indices || !has_initial_state)
    return SC_ERR_NULL_ARG;
  if (!state_pool && num_slots > 0 && H > 0) return SC_ERR_NULL_ARG;
  if (grid && !ckpt->cu_ckpt) return SC_ERR_NULL_ARG;
  // no destination slots (an empty array: no request is long enough to reach a
  // checkpoint) means nothing to export
  if (grid && !ckpt->ckpt_slots) grid = 0;
  if (x == out) return SC_ERR_INVALID_ARG;
  if (num_tokens > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  sc::ConvArgs a{};
  a.x = x;
  a.out = out;
  a.w = weight;
  a.bias = bias;
  a.pool = state_pool;
  a.qsl = query_start_loc;
  a.slots = state_indices;
  a.has_init = has_initial_state;
  a.cu_ckpt = grid ? ckpt->cu_ckpt : nullptr;
  a.ckpt_slots = grid ? ckpt->ckpt_slots : nullptr;
  a.x_rs = desc->x_row_stride;
  a.out_rs = desc->out_row_stride;
  a.slot_stride = desc->state_indices_stride;
  a.num_tokens = num_tokens;
  a.C = desc->channels;
  a.num_slots = (H > 0) ? num_slots : 0;
  a.batch = batch;
  a.q = 0;
  a.ckpt_grid = grid;
  a.S = desc->state_len;
  a.sd = desc->state_layout == SC_STATE_SD ? 1 : 0;
  if ((st = apply_fuse(fuse, out, a)) != SC_OK) return st;
  const bool aligned = conv_aligned(desc, x, out, weight, bias, state_pool) &&
                       (!a.outer || al16(a.outer));
  return from_hip(sc::launch_conv(a, desc->dtype, desc->width, desc->dilation,
                                  desc->activation == SC_ACT_SILU, aligned,
                                  (hipStream_t)stream, nullptr));
}

sc_status sc_conv_update(const sc_conv_desc* desc, const void* x, void* out,
                         const void* weight, const void* bias, void* state_pool,
                         int32_t num_slots, const int32_t* state_indices,
                         const uint8_t* has_initial_state, int32_t batch, int32_t q,
                         const sc_conv_fuse* fuse, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  int H = 0;
  sc_status st = check_conv_desc(desc, &H);
  if (st != SC_OK) return st;
  if ((st = check_fuse(fuse, desc)) != SC_OK) return st;
  if (batch < 0 || q < 0 || num_slots < 0) return SC_ERR_INVALID_ARG;
  if (batch == 0 || q == 0) return SC_OK;
  if (!x || !out || !weight || !state_indices) return SC_ERR_NULL_ARG;
  if (!state_pool && num_slots > 0 && H > 0) return SC_ERR_NULL_ARG;
  if (x == out) return SC_ERR_INVALID_ARG;
  const int64_t T = (int64_t)batch * q;
  if (T > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  sc::ConvArgs a{};
  a.x = x;
  a.out = out;
  a.w = weight;
  a.bias = bias;
  a.pool = state_pool;
  a.qsl = nullptr;
  a.slots = state_indices;
  a.has_init = has_initial_state;
  a.x_rs = desc->x_row_stride;
  a.out_rs = desc->out_row_stride;
  a.slot_stride = desc->state_indices_stride;
  a.num_tokens = T;
  a.C = desc->channels;
  a.num_slots = (H > 0) ? num_slots : 0;
  a.batch = batch;
  a.q = q;
  a.ckpt_grid = 0;
  a.S = desc->state_len;
  a.sd = desc->state_layout == SC_STATE_SD ? 1 : 0;
  if ((st = apply_fuse(fuse, out, a)) != SC_OK) return st;
  const bool aligned = conv_aligned(desc, x, out, weight, bias, state_pool) &&
                       (!a.outer || al16(a.outer));
  return from_hip(sc::launch_conv(a, desc->dtype, desc->width, desc->dilation,
                                  desc->activation == SC_ACT_SILU, aligned,
                                  (hipStream_t)stream, nullptr));
}

sc_status sc_conv_update_spec(const sc_conv_desc* desc, const void* x, void* out,
                              const void* weight, const void* bias, void* state_pool,
                              int32_t num_slots, const int32_t* state_indices,
                              const int32_t* num_accepted_tokens, int32_t batch, int32_t q,
                              const sc_conv_fuse* fuse, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  int H = 0;
  sc_status st = check_conv_desc(desc, &H);
  if (st != SC_OK) return st;
  if ((st = check_fuse(fuse, desc)) != SC_OK) return st;
  if (batch < 0 || q < 0 || num_slots < 0) return SC_ERR_INVALID_ARG;
  // the rolled buffer keeps S - q old entries: q drafts must fit in it
  if (q > desc->state_len) return SC_ERR_INVALID_ARG;
  if (batch == 0 || q == 0) return SC_OK;
  if (!x || !out || !weight || !state_indices || !num_accepted_tokens) return SC_ERR_NULL_ARG;
  if (!state_pool && num_slots > 0) return SC_ERR_NULL_ARG;
  if (x == out) return SC_ERR_INVALID_ARG;
  const int64_t T = (int64_t)batch * q;
  if (T > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  sc::ConvArgs a{};
  a.x = x;
  a.out = out;
  a.w = weight;
  a.bias = bias;
  a.pool = state_pool;
  a.qsl = nullptr;
  a.slots = state_indices;
  a.has_init = nullptr;
  a.num_acc = num_accepted_tokens;
  a.x_rs = desc->x_row_stride;
  a.out_rs = desc->out_row_stride;
  a.slot_stride = desc->state_indices_stride;
  a.num_tokens = T;
  a.C = desc->channels;
  a.num_slots = num_slots;
  a.batch = batch;
  a.q = q;
  a.ckpt_grid = 0;
  a.S = desc->state_len;
  a.sd = desc->state_layout == SC_STATE_SD ? 1 : 0;
  if ((st = apply_fuse(fuse, out, a)) != SC_OK) return st;
  const bool aligned = conv_aligned(desc, x, out, weight, bias, state_pool) &&
                       (!a.outer || al16(a.outer));
  return from_hip(sc::launch_conv_spec(a, desc->dtype, desc->width, desc->dilation,
                                       desc->activation == SC_ACT_SILU, aligned,
                                       (hipStream_t)stream));
}

sc_status sc_conv_update_spec_varlen(const sc_conv_desc* desc, const void* x, void* out,
                                     const void* weight, const void* bias, void* state_pool,
                                     int32_t num_slots, const int32_t* state_indices,
                                     const int32_t* num_accepted_tokens,
                                     const int32_t* query_start_loc, int32_t batch,
                                     int64_t num_tokens, int32_t max_query_len,
                                     const sc_conv_fuse* fuse, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  int H = 0;
  sc_status st = check_conv_desc(desc, &H);
  if (st != SC_OK) return st;
  if ((st = check_fuse(fuse, desc)) != SC_OK) return st;
  if (batch < 0 || num_tokens < 0 || max_query_len < 0 || num_slots < 0)
    return SC_ERR_INVALID_ARG;
  // the rolled buffer keeps S - q old entries: every request's drafts must fit
  if (max_query_len > desc->state_len) return SC_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0 || max_query_len == 0) return SC_OK;
  if (!x || !out || !weight || !state_indices || !num_accepted_tokens || !query_start_loc)
    return SC_ERR_NULL_ARG;
  if (!state_pool && num_slots > 0) return SC_ERR_NULL_ARG;
  if (x == out) return SC_ERR_INVALID_ARG;
  if (num_tokens > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  sc::ConvArgs a{};
  a.x = x;
  a.out = out;
  a.w = weight;
  a.bias = bias;
  a.pool = state_pool;
  a.qsl = query_start_loc;
  a.slots = state_indices;
  a.has_init = nullptr;
  a.num_acc = num_accepted_tokens;
  a.x_rs = desc->x_row_stride;
  a.out_rs = desc->out_row_stride;
  a.slot_stride = desc->state_indices_stride;
  a.num_tokens = num_tokens;
  a.C = desc->channels;
  a.num_slots = num_slots;
  a.batch = batch;
  a.q = max_query_len;
  a.ckpt_grid = 0;
  a.S = desc->state_len;
  a.sd = desc->state_layout == SC_STATE_SD ? 1 : 0;
  if ((st = apply_fuse(fuse, out, a)) != SC_OK) return st;
  const bool aligned = conv_aligned(desc, x, out, weight, bias, state_pool) &&
                       (!a.outer || al16(a.outer));
  return from_hip(sc::launch_conv_spec(a, desc->dtype, desc->width, desc->dilation,
                                       desc->activation == SC_ACT_SILU, aligned,
                                       (hipStream_t)stream));
}

sc_status sc_state_gather(const void* pool, int32_t num_slots, int64_t row_bytes,
                          const int32_t* idx, int64_t idx_stride, int32_t n, void* dense,
                          void* stream) {
  if (num_slots < 0 || row_bytes < 1 || idx_stride < 1 || n < 0) return SC_ERR_INVALID_ARG;
  if (n == 0) return SC_OK;
  if (!idx || !dense || (!pool && num_slots > 0)) return SC_ERR_NULL_ARG;
  return from_hip(sc::launch_state_copy(true, pool, dense, row_bytes, num_slots, idx,
                                        idx_stride, n, (hipStream_t)stream));
}

sc_status sc_state_scatter(const void* dense, int64_t row_bytes, const int32_t* idx,
                           int64_t idx_stride, int32_t n, void* pool, int32_t num_slots,
                           void* stream) {
  if (num_slots < 0 || row_bytes < 1 || idx_stride < 1 || n < 0) return SC_ERR_INVALID_ARG;
  if (n == 0) return SC_OK;
  if (!idx || !dense || (!pool && num_slots > 0)) return SC_ERR_NULL_ARG;
  return from_hip(sc::launch_state_copy(false, dense, pool, row_bytes, num_slots, idx,
                                        idx_stride, n, (hipStream_t)stream));
}

sc_status sc_cca_qk_conv(const sc_cca_desc* desc, const void* q, const void* k,
                         const void* v_cur, const void* v_del, void* out, const void* w_dw,
                         const void* b_dw, const void* w_gr, const void* b_gr,
                         const void* delayed_init, void* conv_state, void* delayed_state,
                         int32_t num_slots, int32_t num_decodes,
                         const int32_t* decode_slots, int32_t num_prefills,
                         const int32_t* prefill_qsl, const int32_t* prefill_slots,
                         const uint8_t* prefill_has_initial_state, int64_t num_tokens,
                         void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  if (desc->dtype != SC_DTYPE_BF16) return SC_ERR_DTYPE;
  const int nq = desc->num_q_heads, nkv = desc->num_kv_heads, hd = desc->head_dim;
  if (nq < 1 || nkv < 1 || hd < 2 || nq % nkv != 0 || hd % 2 != 0 || desc->t0 < 1 ||
      desc->t1 < 1)
    return SC_ERR_INVALID_ARG;
  if (num_slots < 0 || num_decodes < 0 || num_prefills < 0 || num_tokens < 0)
    return SC_ERR_INVALID_ARG;
  const int64_t C = (int64_t)(nq + nkv) * hd, vd = (int64_t)nkv * hd / 2;
  const int64_t W = (int64_t)(nq + 2 * nkv) * hd;
  if (desc->q_row_stride < (int64_t)nq * hd || desc->k_row_stride < (int64_t)nkv * hd ||
      desc->v_cur_row_stride < vd || desc->v_del_row_stride < vd || desc->out_row_stride < W)
    return SC_ERR_INVALID_ARG;
  if (desc->decode_slot_stride < 1 || desc->prefill_slot_stride < 1) return SC_ERR_INVALID_ARG;
  if (num_tokens < num_decodes) return SC_ERR_INVALID_ARG;
  if (num_tokens == 0 || (num_decodes == 0 && num_prefills == 0)) return SC_OK;
  if (!q || !k || !v_cur || !v_del || !out || !w_dw || !b_dw || !w_gr || !b_gr)
    return SC_ERR_NULL_ARG;
  if (num_decodes > 0 && !decode_slots) return SC_ERR_NULL_ARG;
  if (num_prefills > 0 && (!prefill_qsl || !prefill_slots || !prefill_has_initial_state))
    return SC_ERR_NULL_ARG;
  // with t0 = t1 = 1 there is no conv history (an empty, possibly NULL, pool)
  const bool has_history = desc->t0 + desc->t1 - 2 > 0;
  if (num_slots > 0 && ((has_history && !conv_state) || !delayed_state)) return SC_ERR_NULL_ARG;
  if (num_tokens > 0x7FFFFFFFLL || C > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  sc::CcaArgs a{};
  a.q = q;
  a.k = k;
  a.v_cur = v_cur;
  a.v_del = v_del;
  a.out = out;
  a.w_dw = w_dw;
  a.b_dw = b_dw;
  a.w_gr = w_gr;
  a.b_gr = b_gr;
  a.delayed_init = delayed_init;
  a.conv_state = conv_state;
  a.delayed_state = delayed_state;
  a.decode_slots = decode_slots;
  a.prefill_qsl = prefill_qsl;
  a.prefill_slots = prefill_slots;
  a.prefill_h = prefill_has_initial_state;
  a.q_rs = desc->q_row_stride;
  a.k_rs = desc->k_row_stride;
  a.vc_rs = desc->v_cur_row_stride;
  a.vd_rs = desc->v_del_row_stride;
  a.out_rs = desc->out_row_stride;
  a.dslot_stride = desc->decode_slot_stride;
  a.pslot_stride = desc->prefill_slot_stride;
  a.num_tokens = num_tokens;
  a.nq = nq;
  a.nkv = nkv;
  a.hd = hd;
  a.t0 = desc->t0;
  a.t1 = desc->t1;
  a.num_slots = num_slots;
  a.num_decodes = num_decodes;
  a.num_prefills = num_prefills;
  return from_hip(sc::launch_cca(a, (hipStream_t)stream));
}

sc_status sc_gdn_workspace_bytes(const sc_gdn_desc* desc, int32_t batch, int64_t num_tokens,
                                 int64_t* bytes) {
  if (!desc || !bytes) return SC_ERR_NULL_ARG;
  sc_status st = check_gdn_desc(desc);
  if (st != SC_OK) return st;
  if (batch < 0 || num_tokens < 0) return SC_ERR_INVALID_ARG;
  int64_t chunks = 0;
  st = gdn_chunks(desc, batch, num_tokens, &chunks);
  const bool empty = batch == 0 || num_tokens == 0;     // a no-op, whatever the other size
  if (st != SC_OK && !empty) return st;
  *bytes = empty ? 0
                 : sc::GdnWorkspace::bytes(chunks, desc->num_k_heads, desc->num_v_heads,
                                           desc->head_k_dim, batch);
  return SC_OK;
}

sc_status sc_gdn_prefill_varlen(const sc_gdn_desc* desc, const void* q, const void* k,
                                const void* v, const void* a, const void* b,
                                const float* A_log, const float* dt_bias, void* out,
                                float* state_pool, int32_t num_slots,
                                const int32_t* query_start_loc, const int32_t* state_indices,
                                const uint8_t* has_initial_state, int32_t batch,
                                int64_t num_tokens, void* workspace, int64_t workspace_bytes,
                                void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  sc_status st = check_gdn_desc(desc);
  if (st != SC_OK) return st;
  if (batch < 0 || num_tokens < 0 || num_slots < 0 || workspace_bytes < 0)
    return SC_ERR_INVALID_ARG;
  if (batch == 0 || num_tokens == 0) return SC_OK;
  int64_t chunks = 0;
  if ((st = gdn_chunks(desc, batch, num_tokens, &chunks)) != SC_OK) return st;
  if (!query_start_loc || !has_initial_state || !workspace) return SC_ERR_NULL_ARG;
  sc::GdnArgs g;
  st = gdn_args(desc, q, k, v, a, b, A_log, dt_bias, out, state_pool, num_slots, state_indices,
                batch, &g);
  if (st != SC_OK) return st;
  if (!al16(workspace) ||
      workspace_bytes < sc::GdnWorkspace::bytes(chunks, g.hk, g.hv, g.dk, batch))
    return SC_ERR_INVALID_ARG;
  g.qsl = query_start_loc;
  g.has_init = has_initial_state;
  g.num_tokens = num_tokens;
  g.ws = (char*)workspace;
  g.n_chunks = (int32_t)chunks;
  return from_hip(sc::launch_gdn_prefill(g, (hipStream_t)stream));
}

sc_status sc_gdn_update(const sc_gdn_desc* desc, const void* q, const void* k, const void* v,
                        const void* a, const void* b, const float* A_log, const float* dt_bias,
                        void* out, float* state_pool, int32_t num_slots,
                        const int32_t* state_indices, const uint8_t* has_initial_state,
                        int32_t batch, int32_t q_len, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  sc_status st = check_gdn_desc(desc);
  if (st != SC_OK) return st;
  if (batch < 0 || q_len < 0 || num_slots < 0) return SC_ERR_INVALID_ARG;
  if (batch == 0 || q_len == 0) return SC_OK;
  if ((int64_t)batch * q_len > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  sc::GdnArgs g;
  st = gdn_args(desc, q, k, v, a, b, A_log, dt_bias, out, state_pool, num_slots, state_indices,
                batch, &g);
  if (st != SC_OK) return st;
  g.has_init = has_initial_state;
  g.nq = q_len;
  return from_hip(sc::launch_gdn_update(g, (hipStream_t)stream));
}

sc_status sc_gdn_update_spec(const sc_gdn_desc* desc, const void* q, const void* k,
                             const void* v, const void* a, const void* b, const float* A_log,
                             const float* dt_bias, void* out, float* state_pool,
                             int32_t num_slots, const int32_t* state_indices,
                             const int32_t* num_accepted_tokens, int32_t batch, int32_t q_len,
                             void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  sc_status st = check_gdn_desc(desc);
  if (st != SC_OK) return st;
  if (batch < 0 || q_len < 0 || num_slots < 0) return SC_ERR_INVALID_ARG;
  // a row of slots per request, one for each draft
  if (desc->state_indices_stride < q_len) return SC_ERR_INVALID_ARG;
  if (batch == 0 || q_len == 0) return SC_OK;
  if ((int64_t)batch * q_len > 0x7FFFFFFFLL) return SC_ERR_UNSUPPORTED;
  if (!num_accepted_tokens) return SC_ERR_NULL_ARG;
  sc::GdnArgs g;
  st = gdn_args(desc, q, k, v, a, b, A_log, dt_bias, out, state_pool, num_slots, state_indices,
                batch, &g);
  if (st != SC_OK) return st;
  g.num_acc = num_accepted_tokens;
  g.nq = q_len;
  return from_hip(sc::launch_gdn_update(g, (hipStream_t)stream));
}

sc_status sc_qk_norm_rope(const sc_qk_norm_desc* desc, const void* q, const void* k,
                          const void* v, void* q_out, void* k_out, const void* q_weight,
                          const void* k_weight, const void* cos_sin, const int64_t* positions,
                          const int64_t* slots, const sc_paged_cache* k_cache,
                          const sc_paged_cache* v_cache, int64_t num_tokens, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  sc::QkNormArgs a{};
  const sc_status st = norm_args(desc, q, k, v, q_out, k_out, q_weight, k_weight, cos_sin, positions,
                                 slots, k_cache, v_cache, num_tokens, &a);
  if (st != SC_OK || num_tokens == 0) return st;
  return from_hip(sc::launch_qk_norm(a, (hipStream_t)stream));
}

sc_status sc_qk_norm_rope_fp8(const sc_qk_norm_desc* desc, const void* q, const void* k,
                              const void* v, void* q_out, void* k_out, const void* q_weight,
                              const void* k_weight, const void* cos_sin, const int64_t* positions,
                              const int64_t* slots, const sc_paged_cache_fp8* k_cache,
                              const sc_paged_cache_fp8* v_cache, int64_t num_tokens,
                              void* stream) {
  if (!desc || !k_cache || !v_cache) return SC_ERR_NULL_ARG;
  sc::QkNormArgs a{};
  const sc_status st = norm_args(desc, q, k, v, q_out, k_out, q_weight, k_weight, cos_sin, positions,
                                 slots, k_cache, v_cache, num_tokens, &a);
  if (st != SC_OK || num_tokens == 0) return st;
  return from_hip(sc::launch_qk_norm_fp8(a, (hipStream_t)stream));
}

sc_status sc_paged_cache_read_fp8(const sc_cache_read_desc* desc, const sc_paged_cache_fp8* k_cache,
                                  const sc_paged_cache_fp8* v_cache, void* k_out, void* v_out,
                                  const int32_t* block_table, int32_t max_blocks,
                                  const int32_t* start_loc, const int32_t* first_tokens,
                                  int32_t batch, int64_t num_rows, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  const int nkv = desc->num_kv_heads, hd = desc->head_dim;
  sc_status st = check_heads(SC_DTYPE_BF16, nkv, nkv, hd);
  if (st != SC_OK) return st;
  const int64_t w = (int64_t)nkv * hd;
  if (desc->block_size < 1 || desc->num_blocks < 0 || desc->k_row_stride < w ||
      desc->v_row_stride < w || max_blocks < 0 || batch < 0 || num_rows < 0 ||
      desc->block_table_row_stride < std::max(max_blocks, 1))
    return SC_ERR_INVALID_ARG;
  if (desc->k_row_stride % 8 != 0 || desc->v_row_stride % 8 != 0 || num_rows > 0x7FFFFFFFLL)
    return SC_ERR_UNSUPPORTED;
  if (batch == 0 || num_rows == 0) return SC_OK;
  if (!k_cache || !v_cache || !k_out || !v_out || !start_loc || (!block_table && max_blocks > 0))
    return SC_ERR_NULL_ARG;
  if (k_out == v_out) return SC_ERR_INVALID_ARG;
  sc::CacheReadArgs a{};
  if ((st = check_paged_fp8(k_cache, desc->block_size, 16, 1, &a.kc)) != SC_OK) return st;
  if ((st = check_paged_fp8(v_cache, desc->block_size, 16, 1, &a.vc)) != SC_OK) return st;
  if (!al16(k_out) || !al16(v_out)) return SC_ERR_UNSUPPORTED;
  a.k_out = k_out;
  a.v_out = v_out;
  a.table = block_table;
  a.starts = start_loc;
  a.first = first_tokens;
  a.k_rs = desc->k_row_stride;
  a.v_rs = desc->v_row_stride;
  a.table_rs = desc->block_table_row_stride;
  a.num_rows = num_rows;
  a.batch = batch;
  a.nkv = nkv;
  a.hd = hd;
  a.block_size = desc->block_size;
  a.num_blocks = desc->num_blocks;
  a.max_blocks = max_blocks;
  return from_hip(sc::launch_cache_read_fp8(a, (hipStream_t)stream));
}

sc_status sc_paged_attn_workspace_bytes(const sc_paged_attn_desc* desc, int32_t batch,
                                        int32_t q_len, int32_t max_seq_len, int64_t* bytes) {
  if (!desc || !bytes) return SC_ERR_NULL_ARG;
  sc_status st = check_attn_desc(desc);
  if (st != SC_OK) return st;
  sc::PagedAttnArgs a;
  return attn_sizes(desc, batch, q_len, max_seq_len, &a, bytes);
}

sc_status sc_paged_attn_fp8_workspace_bytes(const sc_paged_attn_desc* desc, int32_t batch,
                                            int32_t q_len, int32_t max_seq_len, int64_t* bytes) {
  if (!desc || !bytes) return SC_ERR_NULL_ARG;
  const sc_status st = check_attn_desc(desc);
  if (st != SC_OK) return st;
  sc::PagedAttnArgs a;
  return attn_sizes(desc, batch, q_len, max_seq_len, &a, bytes, true);
}

sc_status sc_paged_attn_decode(const sc_paged_attn_desc* desc, const void* q, void* out,
                               const sc_paged_cache* k_cache, const sc_paged_cache* v_cache,
                               const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seq_lens, int32_t batch, int32_t q_len,
                               int32_t max_seq_len, void* workspace, int64_t workspace_bytes,
                               void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  sc_status st = check_attn_desc(desc);
  if (st != SC_OK) return st;
  sc::PagedAttnArgs a;
  int64_t need = 0;
  if ((st = attn_sizes(desc, batch, q_len, max_seq_len, &a, &need)) != SC_OK) return st;
  if ((st = attn_bounds(desc, max_blocks, max_seq_len, workspace_bytes)) != SC_OK) return st;
  if (batch == 0 || q_len == 0) return SC_OK;
  st = attn_args(desc, q, out, k_cache, v_cache, block_table, seq_lens, max_seq_len, workspace,
                 workspace_bytes, need, &a);
  if (st != SC_OK) return st;
  return from_hip(sc::launch_paged_attn(a, (hipStream_t)stream));
}

sc_status sc_paged_attn_decode_fp8(const sc_paged_attn_desc* desc, const void* q, void* out,
                                   const sc_paged_cache_fp8* k_cache,
                                   const sc_paged_cache_fp8* v_cache, const int32_t* block_table,
                                   int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                   int32_t q_len, int32_t max_seq_len, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  if (!desc) return SC_ERR_NULL_ARG;
  sc_status st = check_attn_desc(desc);
  if (st != SC_OK) return st;
  sc::PagedAttnArgs a;
  int64_t need = 0;
  if ((st = attn_sizes(desc, batch, q_len, max_seq_len, &a, &need, true)) != SC_OK) return st;
  if ((st = attn_bounds(desc, max_blocks, max_seq_len, workspace_bytes)) != SC_OK) return st;
  if (batch == 0 || q_len == 0) return SC_OK;
  st = attn_args(desc, q, out, k_cache, v_cache, block_table, seq_lens, max_seq_len, workspace,
                 workspace_bytes, need, &a);
  if (st != SC_OK) return st;
  if (!tokens_near(a)) return SC_ERR_UNSUPPORTED;
  return from_hip(sc::launch_paged_attn_fp8(a, (hipStream_t)stream));
}

sc_status sc_paged_attn_prefix_workspace_bytes(const sc_paged_attn_desc* desc, int32_t batch,
                                               int32_t q_len, int32_t max_seq_len,
                                               int32_t num_groups, int32_t max_prefix_len,
                                               int64_t* bytes) {
  if (!desc || !bytes) return SC_ERR_NULL_ARG;
  sc_status st = check_attn_desc(desc);
  if (st != SC_OK) return st;
  // what either cache needs
  sc::PagedAttnArgs a;
  int64_t need[2];
  for (int fp8 = 0; fp8 < 2; ++fp8) {
    st = prefix_sizes(desc, batch, q_len, max_seq_len, num_groups, max_prefix_len, fp8 != 0, &a, &need[fp8]);
    if (st != SC_OK) return st;
  }
  *bytes = std::max(need[0], need[1]);
  return SC_OK;
}

sc_status sc_paged_attn_prefix(const sc_paged_attn_desc* desc, const void* q, void* out,
                               const sc_paged_cache* k_cache, const sc_paged_cache* v_cache,
                               const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seq_lens, const int32_t* group_start_loc,
                               const int32_t* prefix_lens, int32_t num_groups, int32_t batch,
                               int32_t q_len, int32_t max_seq_len, int32_t max_prefix_len,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  return attn_prefix_call(desc, q, out, k_cache, v_cache, block_table, max_blocks, seq_lens,
                          group_start_loc, prefix_lens, num_groups, batch, q_len, max_seq_len,
                          max_prefix_len, workspace, workspace_bytes, false, stream);
}

sc_status sc_paged_attn_prefix_fp8(const sc_paged_attn_desc* desc, const void* q, void* out,
                                   const sc_paged_cache_fp8* k_cache,
                                   const sc_paged_cache_fp8* v_cache, const int32_t* block_table,
                                   int32_t max_blocks, const int32_t* seq_lens,
                                   const int32_t* group_start_loc, const int32_t* prefix_lens,
                                   int32_t num_groups, int32_t batch, int32_t q_len,
                                   int32_t max_seq_len, int32_t max_prefix_len, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  return attn_prefix_call(desc, q, out, k_cache, v_cache, block_table, max_blocks, seq_lens,
                          group_start_loc, prefix_lens, num_groups, batch, q_len, max_seq_len,
                          max_prefix_len, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
