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
constexpr int kOwnLeast = 256;   // tokens behind a prefix, a multiple of both kernels' turns
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

// Lane n's value, for all lanes.
__device__ __forceinline__ int64_t lane_of(int64_t x, int n) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, n);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), n);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

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

// Tokens of a split of a request's own part, which begins at `start`: equal parts of
// whole turns of `unit` tokens, from a multiple of 16 on, kOwnLeast or more.
__device__ __forceinline__ int own_split_len(const PagedAttnArgs& a, int start, int len, int unit) {
  const int units = (max(len - (start & ~15), 0) + unit - 1) / unit;
  return max((units + a.splits - 1) / a.splits * unit, kOwnLeast);
}

// What the attn_prefix workgroups left of rows whose own tokens a workgroup of four waves
// has gone through: wave w takes every fourth part into its maximum m, sum l and
// outputs O of the 16 rows from row0 on, as if it were a tile of its own. O[u VR + e] of a
// lane is value (16 u + l16) VR + e of rows 4 lg + i; m belongs to row l16, and of l the
// four lanes of a row have a share each.
template <int HD, int VR, int VW>
__device__ __forceinline__ void take_prefix(const PagedAttnArgs& a, int r, int kvh, int row0, int w,
                                            int n_parts, float& m, float& l, f32x4* O) {
  const int lane = (int)(threadIdx.x & 63), l16 = lane & 15, lg = lane >> 4;
  const int group = a.nq / a.nkv, rows = group * a.nq_tok;
  const int row_parts = a.prefix_splits + a.splits;
  const int64_t n_rows = (int64_t)a.batch * a.nq_tok * a.nq;
  auto first_part = [&](int row) {
    const int j = row / group;
    return (((int64_t)r * a.nq_tok + j) * a.nq + kvh * group + row - j * group) * row_parts;
  };
  const bool ok = row0 + l16 < rows;
  const float* const ml = a.ws + first_part(ok ? row0 + l16 : 0) * 2;
  const float* from[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + lg * 4 + i;
    from[i] = row < rows ? a.ws + values_at(n_rows * row_parts) + first_part(row) * HD + l16 * VR : nullptr;
  }
  for (int p = w; p < n_parts; p += 4) {
    f32x4 x[4][VW * VR / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < VW * VR / 4; ++u) {
        x[i][u] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (from[i]) x[i][u] = *(const f32x4*)(from[i] + (int64_t)p * HD + u / (VR / 4) * 16 * VR + u % (VR / 4) * 4);
      }
    const float mp = ok ? ml[p * 2] : kNone, lp = ok && lg == 0 ? ml[p * 2 + 1] : 0.f;
    const float mn = fmaxf(m, mp);
    const float f = exp2_(m - mn), fp = exp2_(mp - mn);
    m = mn;
    l = l * f + lp * fp;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float fi = __shfl(f, lg * 4 + i), fpi = __shfl(fp, lg * 4 + i);
#pragma unroll
      for (int u = 0; u < VW * VR / 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[u * 4 + e][i] = O[u * 4 + e][i] * fi + x[i][u][e] * fpi;
    }
  }
}

}  // namespace sc
