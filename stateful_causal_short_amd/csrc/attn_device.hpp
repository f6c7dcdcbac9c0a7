// Device helpers shared by the attention kernels over a paged cache: the order of
// requests, the range of the cache that a call's own splits cover, and where the
// parts of a row lie in the workspace.
#pragma once

#include "attn.hpp"
#include "common.hpp"

namespace sc {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 16;        // cached tokens per tile
constexpr int kRows = 16;        // query rows per workgroup of a split
constexpr int kMaxSplits = 64;
constexpr int kSortMax = 512;    // requests put in order by their workgroups
constexpr float kNone = -3.402823466e38f;   // running maximum before any token, the lowest value

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// The i-th request in order of falling length, in 64 steps of max_len and by
// index within a step; a batch of up to kSortMax, its lengths spread over the
// lanes. The step of the i-th is found bit by bit, then its place in the step.
__device__ __forceinline__ int by_length(const PagedAttnArgs& a, int i) {
  const int lane = (int)(threadIdx.x & 63);
  const int drop = max(26 - __builtin_clz(a.max_len | 1), 0);   // 6 bits are left
  int key[kSortMax / 64];
#pragma unroll
  for (int u = 0; u < kSortMax / 64; ++u) {
    const int r = u * 64 + lane;
    key[u] = r < a.batch ? min(max(a.lens[r], 0), a.max_len) >> drop : -1;
  }
  int step = 0;                     // the highest with more than i requests at or above it
#pragma unroll
  for (int bit = 32; bit > 0; bit >>= 1) {
    int n = 0;
#pragma unroll
    for (int u = 0; u < kSortMax / 64; ++u) n += __popcll(__ballot(key[u] >= (step | bit)));
    if (n > i) step |= bit;
  }
  int at = 0;
#pragma unroll
  for (int u = 0; u < kSortMax / 64; ++u) i -= __popcll(__ballot(key[u] > step));
#pragma unroll
  for (int u = 0; u < kSortMax / 64; ++u) {
    const uint64_t in = __ballot(key[u] == step);
    const int n = __popcll(in);
    if (i >= 0 && i < n) {
      const int below = __builtin_amdgcn_mbcnt_hi((uint32_t)(in >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in, 0));
      at = u * 64 + __ffsll(__ballot(key[u] == step && below == i)) - 1;
    }
    i -= n;
  }
  return at;
}

// Workspace: the maximum and the sum of each (query row, split), then, 16-byte
// aligned, its hd values. The float at which those begin, for n of them:
__host__ __device__ inline int64_t values_at(int64_t n) { return (n * 2 + 3) & ~(int64_t)3; }

// Leading tokens of request r that attn_prefix takes for its whole group: those of
// the group, if each of its new tokens sees all of them; else none.
__device__ __forceinline__ int shared_tokens(const PagedAttnArgs& a, int r, int len) {
  const int lane = (int)(threadIdx.x & 63);
  int g = 0;                        // groups that end at or before r
  if (a.groups > 1)
    for (int u = 0; u < a.groups; u += 64) {
      const int64_t in = __ballot(u + lane < a.groups && a.group_starts[u + lane + 1] <= r);
      g += __popcll(in);
    }
  if (g >= a.groups || a.group_starts[g] > r || a.group_starts[g + 1] <= r) return 0;
  const int n = min(max(a.prefix_lens[g], 0), a.max_prefix);
  return n <= len - a.nq_tok + 1 ? n : 0;
}

// Tokens [lo, hi) of a split of a request's own part, which begins at `start`:
// equal parts of whole turns of `unit` tokens, from a multiple of 16 on.
__device__ __forceinline__ int own_split_len(const PagedAttnArgs& a, int start, int len, int unit) {
  const int units = (max(len - (start & ~15), 0) + unit - 1) / unit;
  return max(1, (units + a.splits - 1) / a.splits) * unit;
}

}  // namespace sc
