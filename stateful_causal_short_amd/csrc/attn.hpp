// Argument blocks and launchers of the head norms with rotation and of the
// paged decode attention, shared by qk_norm.hip, attn.hip and abi.hip.
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
  int32_t splits, split_len, sorted; // set by plan_paged_attn
};

// Splits of the cache's length and the workspace they need (bytes).
int64_t plan_paged_attn(PagedAttnArgs* a);

hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t stream);
hipError_t launch_paged_attn(const PagedAttnArgs& a, hipStream_t stream);

}  // namespace sc
