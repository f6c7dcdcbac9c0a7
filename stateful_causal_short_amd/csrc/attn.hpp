// Argument blocks and launchers of the head norms with rotation, of the quantised
// cache's read and of attention over paged caches, shared by their kernels and abi.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sc {

// A paged cache of keys or values: (num_blocks, block_size, heads, head_dim),
// element strides of the first three dimensions.
struct PagedCache {
  void* p;
  int64_t block_s, token_s, head_s;
};

// A quantised cache: e4m3 codes laid out as above, and a scale 2^(byte - 127) for each
// (block, head, token), tokens adjacent, at strides of the first two.
struct PagedCacheFp8 {
  void* p;
  int64_t block_s, token_s, head_s;
  uint8_t* scale;
  int64_t scale_block_s, scale_head_s;
};

struct QkNormArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_out;               // nullable
  const void* q_w;           // nullable: no weight
  const void* k_w;
  const void* table;         // cos | sin rows, nullable with rot = 0
  const int64_t* positions;
  const int64_t* slots;      // nullable without caches
  PagedCache kc, vc;         // p nullable: no write
  int64_t q_rs, k_rs, v_rs, qo_rs, ko_rs, table_rs, max_pos;
  int64_t num_tokens;
  float eps;
  int32_t nq, nkv, hd, rot, interleaved, table_f32, block_size, num_blocks;
  PagedCacheFp8 kc8, vc8;    // quantised caches in place of kc and vc; last, bf16 calls do not fetch them
};

struct PagedAttnArgs {
  const void* q;
  void* out;
  PagedCache kc, vc;
  const int32_t* table;      // (batch, max_blocks) at table_rs
  const int32_t* lens;
  float* ws;                 // partial results when split, else nullptr
  int64_t q_rs, out_rs, table_rs;
  float scale;
  int32_t batch, nq_tok, nq, nkv, hd, block_size, num_blocks, max_len;
  int32_t splits, split_len, sorted; // set by the plans
  // requests [group_starts[g], group_starts[g + 1]) share prefix_lens[g] leading tokens
  const int32_t* group_starts;
  const int32_t* prefix_lens;
  int32_t groups, max_prefix;
  int32_t prefix_splits, prefix_split_len, waves, row_tiles, whole;   // set by plan_paged_attn_prefix
  PagedCacheFp8 kc8, vc8;    // quantised caches in place of kc and vc; last, bf16 calls do not fetch them
};

struct CacheReadArgs {
  PagedCacheFp8 kc, vc;
  void* k_out;
  void* v_out;
  const int32_t* table;      // (batch, max_blocks) at table_rs
  const int32_t* starts;     // (batch + 1): rows of each request
  const int32_t* first;      // nullable: first token of each request
  int64_t k_rs, v_rs, table_rs, num_rows;
  int32_t batch, nkv, hd, block_size, num_blocks, max_blocks;
};

// What a call's workgroups of single requests are: all of it, the parts of requests behind
// their shared prefixes, or those with the prefixes' parts taken in.
enum class After { kNo, kParts, kWhole };

// Splits of the cache's length and the workspace they need (bytes).
int64_t plan_paged_attn(PagedAttnArgs* a);
int64_t plan_paged_attn_fp8(PagedAttnArgs* a);
int64_t plan_paged_attn_prefix(PagedAttnArgs* a, bool fp8);   // -1: more workgroups than a launch has
// Workgroups of the requests' own tokens.
int64_t own_attn_grid(const PagedAttnArgs& a);

hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t stream);
hipError_t launch_qk_norm_fp8(const QkNormArgs& a, hipStream_t stream);
hipError_t launch_cache_read_fp8(const CacheReadArgs& a, hipStream_t stream);
hipError_t launch_paged_attn(const PagedAttnArgs& a, hipStream_t stream);
hipError_t launch_paged_attn_fp8(const PagedAttnArgs& a, hipStream_t stream);
// Requests' own tokens behind their shared prefix.
hipError_t launch_paged_attn_after(const PagedAttnArgs& a, hipStream_t stream);
hipError_t launch_paged_attn_after_fp8(const PagedAttnArgs& a, hipStream_t stream);
hipError_t launch_attn_join(const PagedAttnArgs& a, hipStream_t stream);
hipError_t launch_paged_attn_prefix(const PagedAttnArgs& a, bool fp8, hipStream_t stream);

}  // namespace sc
