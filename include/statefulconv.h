/*
 * statefulconv.h — C ABI of the MI355X (gfx950) stateful causal short
 * convolution library (libstatefulconv.so).
 *
 * The operation: a per-channel (depthwise) causal conv1d over variable-length
 * token batches, optionally dilated, with bias and SiLU, whose per-request
 * history of the last (width-1)*dilation raw inputs lives in a slot-indexed
 * state pool; plus the CCA variant (depthwise then per-head grouped conv, a
 * residual mix and a one-token-delayed value). And the operators that take the
 * convs' outputs: the gated delta rule on a pool of matrix states, and for CCA
 * the head norms with rotation and cache write and the attention of new tokens
 * over that paged cache.
 *
 * Defining passages (page title, section):
 *  - "vllm.model_executor.layers.mamba.ops.cpu.gdn_attention":
 *    _spec_aware_nonspec (decode conv update, then varlen prefill conv with
 *    query_start_loc / cache_indices / has_initial_state, bias, SiLU),
 *    _conv_buffer_view (state as (num_slots, dim, state_len)),
 *    cpu_gdn_attention_core (zero tokens is a no-op; state_len vs width-1).
 *  - "vllm.models.qwen4_exp.nvidia.ple_layer", Qwen4ExpPLELayer:
 *    conv_state_len = (kernel-1)*dilation, dilated depthwise Conv1d,
 *    _short_conv (state capacity check, weights cast to the input dtype),
 *    _short_conv_dilated_dispatch (decode call, then prefill call, then the
 *    prefill checkpoint export), get_kv_cache_spec (checkpoint grid >= state
 *    length, so a checkpoint window holds inputs only).
 *  - "vllm.model_executor.models.zaya", ZayaCCA: the two Conv1d modules,
 *    project (residual mix, output layout) and _mix_with_state (decodes first,
 *    then prefills; history masked by has-state; new history = last n inputs;
 *    delayed value shifted by one token).
 *
 * Conventions for every entry point:
 *  - Pointers marked (device) are device pointers; (host) are host pointers,
 *    read during the call only. The library never allocates or frees device
 *    memory: the caller owns every buffer.
 *  - Calls are asynchronous on `stream` (a hipStream_t passed as void*; NULL
 *    is the default stream). No call synchronises with the host or reads
 *    device memory from the host, so calls may be captured in a HIP graph.
 *  - Arguments are validated on the host before any launch; an error status
 *    means nothing was launched. A launch failure returns SC_ERR_HIP.
 *  - Device-side metadata is trusted but never dereferenced out of bounds:
 *    a slot outside [0, num_slots) is a padding row (zero history, no state
 *    read or write); token rows are clamped to [0, num_tokens).
 *  - Documented, unchecked preconditions (checking needs a host sync):
 *    query_start_loc is non-decreasing with first entry 0 and last entry
 *    num_tokens; slots (and checkpoint slots) are distinct within one call;
 *    `out` does not overlap `x` (exact aliasing is rejected).
 *  - Zero tokens or zero requests: SC_OK, nothing launched; descriptor and
 *    size arguments are still validated, but no pointer is required then
 *    (empty tensors may carry NULL data pointers).
 */
#ifndef STATEFULCONV_H
#define STATEFULCONV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SC_ABI_VERSION 3

typedef enum {
  SC_OK = 0,
  SC_ERR_NULL_ARG = -1,        /* a required pointer is NULL */
  SC_ERR_INVALID_ARG = -2,     /* a size, stride, enum or grid is out of range */
  SC_ERR_DTYPE = -3,           /* dtype not supported by this entry point */
  SC_ERR_STATE_CAPACITY = -4,  /* state_len < (width-1)*dilation */
  SC_ERR_UNSUPPORTED = -5,     /* valid but not built here (e.g. width > 8) */
  SC_ERR_HIP = -6              /* the HIP runtime reported a launch error */
} sc_status;

typedef enum { SC_DTYPE_F32 = 0, SC_DTYPE_BF16 = 1 } sc_dtype;
typedef enum { SC_ACT_NONE = 0, SC_ACT_SILU = 1 } sc_activation;
/* State pool layout (GDN and PLE pages, `is_conv_state_dim_first`): DS =
 * (num_slots, C, S), a channel's entries adjacent (GDN `_conv_buffer_view`);
 * SD = (num_slots, S, C), the cache viewed transposed. Entries are oldest
 * first in both. */
typedef enum { SC_STATE_DS = 0, SC_STATE_SD = 1 } sc_state_layout;

/* Depthwise conv descriptor (host struct, read during the call only).
 * x, out, weight, bias and the state pool share `dtype` (the PLE layer casts
 * its weights to the input dtype); accumulation is fp32. */
typedef struct {
  int32_t channels;       /* C >= 1 */
  int32_t width;          /* K in [1, 8] */
  int32_t dilation;       /* d >= 1 */
  int32_t state_len;      /* S, entries per channel of a state row; S < H = (K-1)*d
                             -> SC_ERR_STATE_CAPACITY; S > 2^20 -> SC_ERR_INVALID_ARG.
                             S > H is a buffer sized for speculative rollback
                             (GDN page, _spec_forward: width-1 + num_spec); the
                             non-speculative calls keep their window in entries
                             [0, H) of each row and leave [H, S) untouched (GDN
                             page, _spec_aware_nonspec, first width-1 columns). */
  int32_t dtype;          /* sc_dtype */
  int32_t activation;     /* sc_activation */
  int64_t x_row_stride;   /* elements between token rows of x, >= C */
  int64_t out_row_stride; /* elements between token rows of out, >= C */
  int64_t state_indices_stride; /* >= 1; row stride of a 2-D index tensor whose
                                   column 0 holds the slot */
  int32_t state_layout;   /* sc_state_layout of every state pool the call touches */
} sc_conv_desc;

/* Prefill checkpoint export (optional). For prefill request r, the m-th
 * checkpoint (m = 1 .. cu_ckpt[r+1]-cu_ckpt[r], and m*grid <= L_r) writes the
 * state window ending at token offset p = m*grid of this chunk — the raw inputs
 * x_r[p-H .. p) — into pool slot ckpt_slots[cu_ckpt[r] + m - 1]. */
typedef struct {
  int32_t grid;              /* g; 0 = no export; else g >= H required */
  const int32_t* cu_ckpt;    /* (device) B+1 exclusive prefix of checkpoint counts */
  const int32_t* ckpt_slots; /* (device) destination slots, flat; NULL (an empty
                                array: no request reaches a checkpoint) exports
                                nothing */
} sc_ckpt_desc;

/* Residual fusion and row mapping, optional on every depthwise call (PLE page
 * "vllm.models.qwen4_exp.nvidia.ple_layer", _short_conv: the conv result is
 * accumulated into `residual`, optionally adding `outer_residual` in the same
 * pass; the dispatch's token_indices let the calls address the speculative and
 * non-speculative rows of a mixed batch in place). NULL = plain call
 * (out = conv). With a descriptor, logical row j of the call (the row the
 * plain call would use) lives at physical row
 *   p = token_indices ? token_indices[j] : j
 * of x, out and outer_residual, and the stored value is, in fp32,
 *   out[p] = (accumulate ? out[p] : 0) + conv_j (+ outer_residual[p])
 * with one final rounding (the additions follow the conv's activation).
 *   token_indices     (device) int32 per logical row, or NULL; entries must be
 *                     distinct rows in [0, num_physical_rows) (an entry outside
 *                     is clamped: no memory fault, that row's results unspecified)
 *   num_physical_rows rows of x / out / outer_residual; required with token_indices
 *   accumulate        0 or 1: out holds the residual on entry (read, then written)
 *   outer_residual    (device) rows like out, or NULL; must not alias out
 *   outer_row_stride  elements between its rows (>= C) */
typedef struct {
  const int32_t* token_indices;
  int64_t num_physical_rows;
  int32_t accumulate;
  const void* outer_residual;
  int64_t outer_row_stride;
} sc_conv_fuse;

/* Varlen prefill: for request r (token rows [qsl[r], qsl[r+1]) of x), slot
 * s = state_indices[r*stride], flag h = has_initial_state[r]:
 *   ext = [h ? pool[s][c][0 .. H) : zeros (oldest first), x_r]
 *   out[t, c] = act(bias[c] + sum_k weight[c, k] * ext[c, H + t - (K-1-k)*d])
 *   pool[s][c][0 .. H) = last H entries of ext (bit-exact copies)
 * A zero-length request produces nothing and leaves its slot untouched.
 *   x                 (device) (num_tokens, C) rows of x_row_stride elements
 *   out               (device) (num_tokens, C) rows of out_row_stride
 *   weight            (device) (C, K) row-major
 *   bias              (device) (C) or NULL
 *   state_pool        (device) (num_slots, C, S) contiguous
 *   query_start_loc   (device) int32 (batch+1)
 *   state_indices     (device) int32, entry r at r*state_indices_stride
 *   has_initial_state (device) uint8 (batch), required (the PLE page raises
 *                     without it)
 *   ckpt              (host) NULL or a checkpoint descriptor */
sc_status sc_conv_prefill_varlen(const sc_conv_desc* desc, const void* x, void* out,
                                 const void* weight, const void* bias,
                                 void* state_pool, int32_t num_slots,
                                 const int32_t* query_start_loc,
                                 const int32_t* state_indices,
                                 const uint8_t* has_initial_state, int32_t batch,
                                 int64_t num_tokens, const sc_ckpt_desc* ckpt,
                                 const sc_conv_fuse* fuse, void* stream);

/* Decode / multi-token update: `batch` requests of exactly q tokens each,
 * request r owning rows [r*q, (r+1)*q) of x (x viewed as (batch, q, C)), all q
 * tokens consumed. Same arithmetic and state rule as the prefill call.
 *   has_initial_state (device) uint8 (batch) or NULL = every request continues
 *                     its saved state (decodes always do). */
sc_status sc_conv_update(const sc_conv_desc* desc, const void* x, void* out,
                         const void* weight, const void* bias, void* state_pool,
                         int32_t num_slots, const int32_t* state_indices,
                         const uint8_t* has_initial_state, int32_t batch,
                         int32_t q, const sc_conv_fuse* fuse, void* stream);

/* Speculative multi-token update on a rolling buffer (GDN page
 * "vllm.model_executor.layers.mamba.ops.cpu.gdn_attention", _spec_forward,
 * per-sequence rolling buffer; PLE page "vllm.models.qwen4_exp.nvidia.ple_layer",
 * ple_conv mode "spec" with num_accepted_tokens and spec_query_len).
 * `batch` requests of exactly q tokens (request r owns rows [r*q, (r+1)*q)),
 * pool rows of S = desc->state_len >= H entries. With slot s and
 *   a = num_accepted_tokens[r] clamped to [1, min(q, S-H+1)]
 * (the range in which the page's slices are well formed; values outside it
 * act as the nearest bound):
 *   ext      = [pool[s][c][a-1 .. a-1+H), x_r]
 *   out[t,c] = act(bias[c] + sum_k weight[c,k] * ext[c, H + t - (K-1-k)*d])
 *   pool[s]  = [pool[s][c][a .. a+S-q), x_r]   (length S, bit-exact copies)
 * A slot outside [0, num_slots) is a padding row: zero history, no write.
 * q > S -> SC_ERR_INVALID_ARG (the drafts would not fit the buffer).
 *   num_accepted_tokens (device) int32 (batch), required.
 * Other arguments as for sc_conv_update (no has_initial_state: speculative
 * requests always continue their buffer). */
sc_status sc_conv_update_spec(const sc_conv_desc* desc, const void* x, void* out,
                              const void* weight, const void* bias, void* state_pool,
                              int32_t num_slots, const int32_t* state_indices,
                              const int32_t* num_accepted_tokens, int32_t batch,
                              int32_t q, const sc_conv_fuse* fuse, void* stream);

/* Speculative update with a draft count per request (GDN page
 * "vllm.model_executor.layers.mamba.ops.cpu.gdn_attention", _spec_forward,
 * the per-sequence loop over spec_query_start_loc that serves batches whose
 * requests draft different numbers of tokens). Request r owns rows
 * [query_start_loc[r], query_start_loc[r+1]) of x and out; with
 * q_r = query_start_loc[r+1] - query_start_loc[r], the rule of
 * sc_conv_update_spec applies to it with q = q_r (a clamped to
 * [1, min(q_r, S-H+1)]). A request with q_r = 0 is skipped (the page's loop
 * continues past it): nothing is read or written for it.
 *   query_start_loc (device) int32 (batch+1), non-decreasing,
 *                   query_start_loc[0] >= 0, query_start_loc[batch] <= num_tokens.
 *   max_query_len   (host) a bound on every q_r; must be <= S
 *                   (SC_ERR_INVALID_ARG otherwise). A request that breaks
 *                   the bound, or whose rows leave [0, num_tokens), is
 *                   skipped whole (its rows and slot are left as they were).
 *   num_tokens      (host) rows of x and out.
 * Other arguments as for sc_conv_update_spec. batch = 0, num_tokens = 0 or
 * max_query_len = 0: no-op. */
sc_status sc_conv_update_spec_varlen(const sc_conv_desc* desc, const void* x, void* out,
                                     const void* weight, const void* bias, void* state_pool,
                                     int32_t num_slots, const int32_t* state_indices,
                                     const int32_t* num_accepted_tokens,
                                     const int32_t* query_start_loc, int32_t batch,
                                     int64_t num_tokens, int32_t max_query_len,
                                     const sc_conv_fuse* fuse, void* stream);

/* Row copies between a slot pool and a dense buffer; each row is row_bytes.
 * They are the state gather and write-back of "vllm.model_executor.models.zaya",
 * ZayaCCA._mix_with_state, on their own: that method reads each request's
 * history as the pool row its slot index names, masked to zeros when the
 * request has no initial state, and afterwards writes the new history back to
 * the same row; the GDN page ("vllm.model_executor.layers.mamba.ops.cpu.
 * gdn_attention", _spec_forward) indexes its conv-state cache by slot in the
 * same way. Byte copies, so bit-exact for any dtype and either layout.
 * gather: dense[i] = pool[idx[i*idx_stride]], or zeros when that index is
 *         outside [0, num_slots) (a padding row has no history).
 * scatter: pool[idx[i*idx_stride]] = dense[i]; out-of-range indices skipped;
 *          two equal in-range indices race (a documented precondition:
 *          distinct indices, as sc_validate_metadata checks).
 *   pool, dense, idx (device, caller-owned); n rows; row_bytes >= 1.
 * Errors: NULL pointer with n > 0 -> SC_ERR_NULL_ARG; negative n or
 * num_slots, row_bytes < 1 or idx_stride < 1 -> SC_ERR_INVALID_ARG;
 * launch failure -> SC_ERR_HIP. n = 0: no-op. Asynchronous on `stream`. */
sc_status sc_state_gather(const void* pool, int32_t num_slots, int64_t row_bytes,
                          const int32_t* idx, int64_t idx_stride, int32_t n,
                          void* dense, void* stream);
sc_status sc_state_scatter(const void* dense, int64_t row_bytes,
                           const int32_t* idx, int64_t idx_stride, int32_t n,
                           void* pool, int32_t num_slots, void* stream);

/* CCA q/k conv descriptor (host struct). bf16 only (SC_ERR_DTYPE otherwise). */
typedef struct {
  int32_t num_q_heads;    /* nq */
  int32_t num_kv_heads;   /* nkv; nq % nkv == 0 */
  int32_t head_dim;       /* hd */
  int32_t t0;             /* depthwise kernel size */
  int32_t t1;             /* grouped kernel size */
  int32_t dtype;          /* SC_DTYPE_BF16 */
  int64_t q_row_stride, k_row_stride, v_cur_row_stride, v_del_row_stride;
  int64_t out_row_stride;
  int64_t decode_slot_stride, prefill_slot_stride;
} sc_cca_desc;

/* CCA q/k conv with per-request state (ZayaCCA.project + _mix_with_state).
 * Tokens: num_decodes one-token decode rows first (always continuing their
 * state), then prefill rows with offsets prefill_qsl (rebased to 0).
 * With C = (nq+nkv)*hd raw channels [q | k] and n = t0+t1-2:
 *   dw   = depthwise conv (t0 taps, bias) of [history, raw], materialised in
 *          bf16: summed in fp32 from the bias (hd = 128, t1 = 2: taps in
 *          pairs on the two-term bf16 dot product; other shapes: a fused
 *          multiply-add chain in tap order) and rounded to bf16, which is the
 *          exact value rounded once except where the fp32 sum's own rounding
 *          moves it across a bf16 midpoint (a few values in 10^7 on normally
 *          distributed data)
 *   yg   = grouped conv (nq+nkv groups of hd, t1 taps, bias) of dw, fp32 acc.
 *   out row = [yg_q + 0.5(q + k of the head's kv group) |
 *              yg_k + mean over the group's q heads of that residual |
 *              v_cur | previous token's v_del (first token: saved delayed
 *              value if it has state, else delayed_init, NULL = zeros)]
 *   conv_state[s] = last n raw inputs; delayed_state[s] = last v_del row.
 *   q (T, nq*hd), k (T, nkv*hd), v_cur, v_del (T, nkv*hd/2), out
 *   (T, (nq+2*nkv)*hd); w_dw (C, t0), b_dw (C), w_gr (C, hd, t1), b_gr (C),
 *   delayed_init (nkv*hd/2) or NULL; conv_state (num_slots, C, n; may be NULL
 *   when n = 0),
 *   delayed_state (num_slots, nkv*hd/2); slot arrays int32, has-state uint8.
 *   All (device). num_tokens must equal num_decodes + prefill_qsl[last]. */
sc_status sc_cca_qk_conv(const sc_cca_desc* desc, const void* q, const void* k,
                         const void* v_cur, const void* v_del, void* out,
                         const void* w_dw, const void* b_dw, const void* w_gr,
                         const void* b_gr, const void* delayed_init,
                         void* conv_state, void* delayed_state, int32_t num_slots,
                         int32_t num_decodes, const int32_t* decode_slots,
                         int32_t num_prefills, const int32_t* prefill_qsl,
                         const int32_t* prefill_slots,
                         const uint8_t* prefill_has_initial_state,
                         int64_t num_tokens, void* stream);

/* Gated delta rule (GDN page "vllm.model_executor.layers.mamba.ops.cpu.
 * gdn_attention": it hands the mixed-qkv conv's output to this recurrence, as
 * decode, speculative decode and varlen prefill, with gates from A_log, a, b and
 * dt_bias; the arithmetic is not on the page, and is the rule's usual one). Per
 * value head, with a state S (DV x DK) that lives in a slot pool next to the
 * conv state:
 *   g = -exp(A_log) * softplus(a + dt_bias),  beta = sigmoid(b)
 *   q^, k^ = q, k scaled by 1/sqrt(sum of squares + 1e-6) (qk_l2norm = 1), or as they are
 *   S <- exp(g) S;  S <- S + beta (v - S k^) k^T;  out = scale * S q^
 * Value head h reads key head h / (num_v_heads / num_k_heads). q, k, v and out
 * are bf16 (the page's core rejects other inputs); the state, the gates and
 * every sum are fp32, whose range a head's sum of squares must not pass.
 *   q, k    (T, num_k_heads * DK), v, out (T, num_v_heads * DV): rows of their
 *           strides, e.g. the column blocks of the conv's output rows; q, k and
 *           v 16-byte aligned with strides a multiple of 8, out 8-byte
 *           aligned with a stride a multiple of 4
 *   a, b    (T, num_v_heads), gate_dtype; A_log, dt_bias (num_v_heads) fp32
 *   state   (num_slots, num_v_heads, DV, DK) fp32, contiguous, 16-byte aligned
 * DK is 64 or 128, DV a multiple of 16 (SC_ERR_UNSUPPORTED otherwise; also
 * for rows that break the alignment above). `out` overlaps no input; two
 * requests of a call share no slot. */
typedef struct {
  int32_t num_k_heads;   /* HK >= 1 */
  int32_t num_v_heads;   /* HV, a multiple of HK */
  int32_t head_k_dim;    /* DK */
  int32_t head_v_dim;    /* DV */
  int32_t dtype;         /* SC_DTYPE_BF16 */
  int32_t gate_dtype;    /* sc_dtype of a and b */
  int32_t qk_l2norm;     /* 0 or 1 */
  float scale;           /* finite; the usual choice is 1/sqrt(DK) */
  int64_t q_row_stride, k_row_stride, v_row_stride;   /* elements */
  int64_t a_row_stride, b_row_stride, out_row_stride;
  int64_t state_indices_stride;                       /* >= 1 */
} sc_gdn_desc;

/* Bytes of workspace sc_gdn_prefill_varlen needs for these sizes (host only). */
sc_status sc_gdn_workspace_bytes(const sc_gdn_desc* desc, int32_t batch, int64_t num_tokens,
                                 int64_t* bytes);

/* Varlen prefill: request r owns token rows [qsl[r], qsl[r+1]), starts from
 * state[slot] if has_initial_state[r] (zeros otherwise, and for a slot outside
 * the pool) and leaves its final state there. A zero-length request leaves
 * its slot untouched. Tokens are taken 64 at a time; a non-finite input can
 * reach earlier rows of its own request's group of 64, and no other request.
 *   workspace (device) 16-byte aligned, at least sc_gdn_workspace_bytes; its
 *             contents are scratch, so two calls that may run at once (two
 *             streams, two captured graphs) need one each. */
sc_status sc_gdn_prefill_varlen(const sc_gdn_desc* desc, const void* q, const void* k,
                                const void* v, const void* a, const void* b,
                                const float* A_log, const float* dt_bias, void* out,
                                float* state_pool, int32_t num_slots,
                                const int32_t* query_start_loc, const int32_t* state_indices,
                                const uint8_t* has_initial_state, int32_t batch,
                                int64_t num_tokens, void* workspace, int64_t workspace_bytes,
                                void* stream);

/* Decode / multi-token update: `batch` requests of exactly q_len tokens,
 * request r owning rows [r*q_len, (r+1)*q_len). has_initial_state NULL = every
 * request continues its state. */
sc_status sc_gdn_update(const sc_gdn_desc* desc, const void* q, const void* k, const void* v,
                        const void* a, const void* b, const float* A_log, const float* dt_bias,
                        void* out, float* state_pool, int32_t num_slots,
                        const int32_t* state_indices, const uint8_t* has_initial_state,
                        int32_t batch, int32_t q_len, void* stream);

/* Speculative update: request r has q_len drafts and q_len state slots,
 * state_indices[r*stride .. r*stride + q_len) (stride >= q_len). It starts from
 * the slot of its last accepted draft, entry num_accepted_tokens[r] - 1
 * (clamped to [0, q_len)), and leaves the state after draft t in entry t's
 * slot, so that the next call can roll back to any of them. */
sc_status sc_gdn_update_spec(const sc_gdn_desc* desc, const void* q, const void* k,
                             const void* v, const void* a, const void* b, const float* A_log,
                             const float* dt_bias, void* out, float* state_pool,
                             int32_t num_slots, const int32_t* state_indices,
                             const int32_t* num_accepted_tokens, int32_t batch, int32_t q_len,
                             void* stream);

/* A paged cache of keys or values: (num_blocks, block_size, num_kv_heads,
 * head_dim) bf16 with a unit stride in head_dim; element strides of the other
 * three dimensions (so heads before tokens, or keys and values in one
 * allocation, are the caller's choice). Token s of the cache is row
 * s % block_size of block s / block_size. */
typedef struct {
  void* data;              /* (device) */
  int64_t block_stride, token_stride, head_stride;
} sc_paged_cache;

/* Norms of query and key heads, position rotation and cache write, for the
 * [query | key | value] rows that sc_cca_qk_conv writes. The four pages end
 * before this step: these are the usual root-mean-square norm and rotation, not
 * a form that they print. Per head x of head_dim values, with one weight for all
 * query heads and one for all key heads:
 *   x^ = weight * x / sqrt(mean(x^2) + eps)           (weight NULL: 1)
 *   pair i of the first rotary_dim values turns by the table's angle i:
 *   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin), the pair being values
 *   (i, i + rotary_dim/2), or (2i, 2i + 1) with interleaved = 1
 * in fp32 with one rounding at the store (a head whose sum of squares passes
 * fp32's range, from values near 2^60 on, comes out as zeros). Values are copied. */
typedef struct {
  int32_t num_q_heads, num_kv_heads;
  int32_t head_dim;        /* 64, 128 or 256 (SC_ERR_UNSUPPORTED otherwise) */
  int32_t rotary_dim;      /* 0 (no rotation) .. head_dim, a multiple of 8 */
  int32_t interleaved;     /* 0 or 1 */
  int32_t dtype;           /* SC_DTYPE_BF16 */
  int32_t table_dtype;     /* sc_dtype of cos_sin */
  float eps;               /* >= 0 */
  int32_t block_size, num_blocks;                   /* of the caches */
  int64_t q_row_stride, k_row_stride, v_row_stride; /* elements */
  int64_t q_out_row_stride, k_out_row_stride, table_row_stride;
  int64_t max_position;    /* rows of cos_sin */
} sc_qk_norm_desc;

/*   q, k, v   (device) (T, heads * head_dim) rows, 8-byte aligned, strides a
 *             multiple of 4 (e.g. column blocks of the CCA output rows)
 *   q_out     (device) (T, num_q_heads * head_dim); k_out the same for keys, or
 *             NULL; q_out == q and k_out == k (the same stride) work in place,
 *             other overlaps are not allowed
 *   q_weight, k_weight (device) bf16 (head_dim) or NULL
 *   cos_sin   (device) (max_position, rotary_dim): cos of the rotary_dim/2
 *             angles, then sin; NULL with rotary_dim = 0
 *   positions (device) int64 (T), clamped to [0, max_position); NULL with
 *             rotary_dim = 0
 *   slots     (device) int64 (T): the cache row of each token; a row outside
 *             the cache (-1: padding) is not written. Required with a cache.
 *   k_cache, v_cache (host) NULL or a cache, both or neither; v may be NULL
 *             without them. Rows must be distinct within one call. */
sc_status sc_qk_norm_rope(const sc_qk_norm_desc* desc, const void* q, const void* k,
                          const void* v, void* q_out, void* k_out, const void* q_weight,
                          const void* k_weight, const void* cos_sin, const int64_t* positions,
                          const int64_t* slots, const sc_paged_cache* k_cache,
                          const sc_paged_cache* v_cache, int64_t num_tokens, void* stream);

/* Attention of the newest tokens over a paged cache (the attention that reads
 * what sc_qk_norm_rope wrote; the usual softmax form, as none of the pages prints
 * it). `batch` requests of exactly q_len new tokens,
 * request r owning rows [r*q_len, (r+1)*q_len) of q and out; its cache holds
 * seq_lens[r] tokens, the new ones last, so new token j sees positions
 * [0, seq_lens[r] - q_len + j]. Query head h reads key/value head
 * h / (num_q_heads / num_kv_heads).
 *   out = sum_t softmax_t(scale q.k_t) v_t
 * A row that sees nothing, or only scores of minus infinity, is zeros. Scores,
 * weights and sums are fp32, the scores in base 2: one of a size above 2.3e38
 * counts as infinite. `out` overlaps no input. */
typedef struct {
  int32_t num_q_heads, num_kv_heads;
  int32_t head_dim;        /* 64, 128 or 256 (SC_ERR_UNSUPPORTED otherwise) */
  int32_t dtype;           /* SC_DTYPE_BF16 */
  int32_t block_size;      /* a multiple of 16 (SC_ERR_UNSUPPORTED otherwise) */
  int32_t num_blocks;
  float scale;             /* finite */
  int64_t q_row_stride, out_row_stride;   /* elements, multiples of 8 and 4 */
  int64_t block_table_row_stride;         /* >= max_blocks */
} sc_paged_attn_desc;

/* Bytes of workspace for these sizes on the current device (host only; 0 when
 * the cache's length is not split). */
sc_status sc_paged_attn_workspace_bytes(const sc_paged_attn_desc* desc, int32_t batch,
                                        int32_t q_len, int32_t max_seq_len, int64_t* bytes);

/*   block_table (device) int32 (batch, max_blocks): block of each block_size
 *               tokens; entries behind a request's last token may hold
 *               anything; a block outside the cache holds no visible token
 *   seq_lens    (device) int32 (batch), clamped to [0, max_seq_len]
 *   max_seq_len (host) <= max_blocks * block_size and <= 2^30; the split
 *               follows from it
 *   workspace   (device) 16-byte aligned, or NULL if none is needed; scratch:
 *               calls that may run at once need one each
 * Cache pointers 16-byte aligned, strides a multiple of 8. */
sc_status sc_paged_attn_decode(const sc_paged_attn_desc* desc, const void* q, void* out,
                               const sc_paged_cache* k_cache, const sc_paged_cache* v_cache,
                               const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seq_lens, int32_t batch, int32_t q_len,
                               int32_t max_seq_len, void* workspace, int64_t workspace_bytes,
                               void* stream);

/* A quantised paged cache: the codes, 8-bit floats of four significant bits (e4m3, no
 * infinities, largest 448), laid out as sc_paged_cache (strides in codes), and one
 * scale for each token's head, 2^(byte - 127) in a byte (e8m0): (num_blocks,
 * num_kv_heads, block_size) with a unit stride over a block's tokens. A value is its
 * code times its scale. The library writes bytes 1 .. 247; 0 counts as 2^-127, and
 * rows that see a token with a byte of 255 are undefined. A bf16 value of 248 * 2^120
 * or more is nearest to the code 256 under 247, which is 2^128: infinite in bf16. */
typedef struct {
  void* data;              /* (device) */
  int64_t block_stride, token_stride, head_stride;
  void* scale;             /* (device) */
  int64_t scale_block_stride, scale_head_stride;
} sc_paged_cache_fp8;

/* sc_qk_norm_rope into a quantised cache (required here). The scale of a head is the
 * smallest power of two, from 2^-126 on, that brings its largest finite value to 448
 * or less; values over it are rounded to the nearest code, ties to even, keys
 * straight from fp64. Infinities, keys past fp32's range among them, and NaN become
 * NaN codes and leave the scale to the others. Codes 4-byte aligned, strides a
 * multiple of 4. */
sc_status sc_qk_norm_rope_fp8(const sc_qk_norm_desc* desc, const void* q, const void* k,
                              const void* v, void* q_out, void* k_out, const void* q_weight,
                              const void* k_weight, const void* cos_sin, const int64_t* positions,
                              const int64_t* slots, const sc_paged_cache_fp8* k_cache,
                              const sc_paged_cache_fp8* v_cache, int64_t num_tokens,
                              void* stream);

typedef struct {
  int32_t num_kv_heads;
  int32_t head_dim;        /* 64, 128 or 256 (SC_ERR_UNSUPPORTED otherwise) */
  int32_t block_size, num_blocks;
  int64_t k_row_stride, v_row_stride;     /* elements, multiples of 8 */
  int64_t block_table_row_stride;         /* >= max_blocks, >= 1 */
} sc_cache_read_desc;

/* Reads tokens of a quantised cache back as bf16 rows, exactly but for values
 * outside bf16's range (below 2^-126 to the nearest 2^-133, 2^128 as infinity): row
 * start_loc[r] + i is token first_tokens[r] + i of request r, for start_loc[r] <= row <
 * start_loc[r + 1]. Tokens outside the block table or in a block outside the cache read
 * as zeros; other rows are left as they were.
 *   k_out, v_out (device) (num_rows, num_kv_heads * head_dim) bf16, 16-byte aligned
 *   block_table  (device) int32 (batch, max_blocks)
 *   start_loc    (device) int32 (batch + 1), non-decreasing
 *   first_tokens (device) int32 (batch), or NULL: every request from its first on
 * Codes 16-byte aligned, strides a multiple of 16. */
sc_status sc_paged_cache_read_fp8(const sc_cache_read_desc* desc, const sc_paged_cache_fp8* k_cache,
                                  const sc_paged_cache_fp8* v_cache, void* k_out, void* v_out,
                                  const int32_t* block_table, int32_t max_blocks,
                                  const int32_t* start_loc, const int32_t* first_tokens,
                                  int32_t batch, int64_t num_rows, void* stream);

/* sc_paged_attn_decode over quantised caches: the same rows, visibility and
 * arguments, scores and weights in fp32. Codes 16-byte aligned, strides a multiple of
 * 16 and of tokens below 2^26; scales 4-byte aligned, strides a multiple of 4. The
 * workspace is its own function's. */
sc_status sc_paged_attn_fp8_workspace_bytes(const sc_paged_attn_desc* desc, int32_t batch,
                                            int32_t q_len, int32_t max_seq_len, int64_t* bytes);
sc_status sc_paged_attn_decode_fp8(const sc_paged_attn_desc* desc, const void* q, void* out,
                                   const sc_paged_cache_fp8* k_cache,
                                   const sc_paged_cache_fp8* v_cache, const int32_t* block_table,
                                   int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                   int32_t q_len, int32_t max_seq_len, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/* Attention of the newest tokens of requests that share the beginning of their
 * caches: the rows of sc_paged_attn_decode, with each group's prefix read once for
 * all of its requests. Requests [group_start_loc[g], group_start_loc[g + 1]) hold the
 * same keys and values in their first prefix_lens[g] tokens, in the same blocks or
 * copies of them: they are read where the first such request has them whose new
 * tokens all see the whole prefix. Requests whose new tokens do not (short ones,
 * rows that pad a captured batch) and those of no group are taken by themselves, as
 * in sc_paged_attn_decode, whatever the others hold. Into how many parts a request's
 * own tokens are split follows from the sizes alone: from max_seq_len where few rows
 * share long prefixes, else from max_seq_len - max_prefix_len. Requests with many
 * thousand tokens of their own beside large groups end sooner in a call without
 * groups.
 *   group_start_loc (device) int32 (num_groups + 1), non-decreasing, in [0, batch]
 *   prefix_lens     (device) int32 (num_groups), clamped to [0, max_prefix_len]; any
 *                   length, in whole blocks or not
 *   num_groups      (host) >= 0; with 0 both arrays may be NULL
 *   max_prefix_len  (host) <= max_seq_len; the split of the prefixes follows from it
 * block_table rows hold a request's whole cache, its prefix first. Over the prefix,
 * weights enter the second product as two bf16 parts (2^-15); everything else is
 * as in sc_paged_attn_decode and sc_paged_attn_decode_fp8. Other arguments, limits
 * and alignment are theirs, and token strides are below 2^26; one workspace function
 * serves both caches. Quantised keys and values of a prefix enter as bf16, as
 * sc_paged_cache_read_fp8 reads them: below 2^-126 to the nearest 2^-133, 2^128 as
 * infinity. */
sc_status sc_paged_attn_prefix_workspace_bytes(const sc_paged_attn_desc* desc, int32_t batch,
                                               int32_t q_len, int32_t max_seq_len,
                                               int32_t num_groups, int32_t max_prefix_len,
                                               int64_t* bytes);
sc_status sc_paged_attn_prefix(const sc_paged_attn_desc* desc, const void* q, void* out,
                               const sc_paged_cache* k_cache, const sc_paged_cache* v_cache,
                               const int32_t* block_table, int32_t max_blocks,
                               const int32_t* seq_lens, const int32_t* group_start_loc,
                               const int32_t* prefix_lens, int32_t num_groups, int32_t batch,
                               int32_t q_len, int32_t max_seq_len, int32_t max_prefix_len,
                               void* workspace, int64_t workspace_bytes, void* stream);
sc_status sc_paged_attn_prefix_fp8(const sc_paged_attn_desc* desc, const void* q, void* out,
                                   const sc_paged_cache_fp8* k_cache,
                                   const sc_paged_cache_fp8* v_cache, const int32_t* block_table,
                                   int32_t max_blocks, const int32_t* seq_lens,
                                   const int32_t* group_start_loc, const int32_t* prefix_lens,
                                   int32_t num_groups, int32_t batch, int32_t q_len,
                                   int32_t max_seq_len, int32_t max_prefix_len, void* workspace,
                                   int64_t workspace_bytes, void* stream);

/* Checks the device-side preconditions the calls above document but cannot
 * check without a host sync (a debugging and test aid, not for the hot path):
 * waits for `stream`, copies the metadata to the host and returns
 * SC_ERR_INVALID_ARG if
 *   query_start_loc (device, batch+1, or NULL to skip) is not non-decreasing
 *                   from query_start_loc[0] = 0 to query_start_loc[batch] = num_tokens;
 *   state_indices   (device, batch rows of idx_stride, or NULL to skip) has an
 *                   entry >= num_slots, or two equal non-negative entries
 *                   (negative entries are padding rows);
 * else SC_OK. It allocates no device memory and launches nothing. batch = 0:
 * SC_OK without touching the pointers; a HIP error while copying: SC_ERR_HIP;
 * negative sizes, idx_stride < 1, or arrays too large to copy to the host:
 * SC_ERR_INVALID_ARG. */
sc_status sc_validate_metadata(const int32_t* query_start_loc, const int32_t* state_indices,
                               int64_t idx_stride, int32_t batch, int64_t num_tokens,
                               int32_t num_slots, void* stream);

/* Static string for a status code. */
const char* sc_status_string(sc_status status);

/* SC_ABI_VERSION of the built library. */
int32_t sc_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* STATEFULCONV_H */
