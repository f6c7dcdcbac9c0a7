// Attention of one or a few new tokens per request over a paged cache.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - max)
//
// over the positions a token sees. The bytes of the cache bound it: a group of
// up to 16 rows (the query heads of one key/value head, times the request's new
// tokens) reads keys and values once from HBM straight into registers, as MFMA
// operands. More rows are more groups, in workgroups of their own, and each
// reads the cache again.
//
// The rows of a group share each key: scores of 16 cached tokens x 16 rows
// are one 16x16x32 bf16 product per 32 values of a head, with the keys as the
// left operand as they lie in the cache. A score tile then has row n = lane %
// 16 and tokens 4 (lane / 16) + i in register i, which is how the fp32
// 16x16x4 product wants its left operand when product i sums over tokens
// 4 g + i, g = 0..3. So p goes from the softmax to the second product in its
// registers, in fp32, and the values are read 16 lanes to a token's row.
//
// Work split: a workgroup has one (request, key/value head, row group, split of
// the cache's length); its four waves take 16-token tiles in turn, each with a
// running maximum and sum, and join in LDS at the end. With more than one split
// the parts go to the workspace and attn_join adds them.
//
// 16 query and 4 key/value heads x 128, pages of 16: three requests of 131,071
// tokens 155 + 7 us (805 MB, 5.2 TB/s in the first); 512 requests of up to
// 2,048 tokens 208 us (1,078 MB, 5.2 TB/s; 5.5 with even lengths); 64 x 4 drafts
// over up to 8,192 tokens 116-135 + 9 us, where uneven splits and the start and
// end of each workgroup show; one request of 300 tokens 10.8 us: a wave's five
// tiles in turn, each page -> key -> softmax -> values, on four CUs, and the join.
#include "attn.hpp"
#include "common.hpp"

#include <algorithm>

namespace sc {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

namespace {

constexpr int kTile = 16;        // cached tokens per tile
constexpr int kRows = 16;        // query rows per workgroup
constexpr int kMaxSplits = 64;
constexpr int kSortMax = 512;    // requests put in order by their workgroups
constexpr float kNone = -3.402823466e38f;   // running maximum before any token, the lowest value

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Two bf16 values, infinities and NaN replaced by zero.
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {
  const uint32_t lo = (x & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu;
  return ((x & 0x7F800000u) == 0x7F800000u ? 0u : x & 0xFFFF0000u) | lo;
}

// N adjacent bf16 values (4 or 8), one load.
template <int N>
using ValueRun = uint32_t __attribute__((ext_vector_type(N / 2)));

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

}  // namespace

template <int HD>
__global__ __launch_bounds__(kBlock, HD == 256 ? 2 : 4) void attn_split(PagedAttnArgs a) {
  constexpr int KS = HD / 32;               // score products per tile
  constexpr int VPL = HD / 16;              // values of a token's row per lane
  constexpr int VR = VPL < 8 ? VPL : 8;     // ... in runs of one load, 16 VR apart
  constexpr int VW = VPL / VR;
  __shared__ __align__(16) float Ol[3][kRows * HD];
  __shared__ float ml[3][kRows], ll[3][kRows];

  const int group = a.nq / a.nkv, rows = group * a.nq_tok;
  const int row_groups = (rows + kRows - 1) / kRows;
  unsigned id = blockIdx.x;
  const int kvh = (int)(id % (unsigned)a.nkv);
  id /= (unsigned)a.nkv;
  int r = (int)(id % (unsigned)a.batch);
  id /= (unsigned)a.batch;
  const int rg = (int)(id % (unsigned)row_groups);
  const int split = (int)(id / (unsigned)row_groups);
  if (a.sorted) r = by_length(a, r);

  const int lane = (int)(threadIdx.x & 63);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l16 = lane & 15, lg = lane >> 4;
  const int t_lo = split * a.split_len;
  // Page ids run two tiles ahead of their use: a load that waits for another
  // load waits for the memory queue twice. They do not wait for the length
  // either: a tile below max_len has an entry in the table.
  const int32_t* const table = a.table + (int64_t)r * a.table_rs;
  auto page_of = [&](int t) { return t < a.max_len ? table[t / a.block_size] : -1; };
  int t0 = t_lo + w * kTile;
  int page = page_of(t0), page_next = page_of(t0 + 4 * kTile);
  const int len = min(max(a.lens[r], 0), a.max_len);
  const int t_hi = min(len, t_lo + a.split_len);
  if (split > 0 && t_lo >= len) return;      // the join does not read such a split

  // this lane's query row: head kvh * group + g of new token j
  const int row = rg * kRows + l16;
  const bool row_ok = row < rows;
  const int j = row_ok ? row / group : 0, g = row_ok ? row - j * group : 0;
  const int64_t q_row = (int64_t)r * a.nq_tok + j;
  const int head = kvh * group + g;
  const int limit = row_ok ? len - a.nq_tok + j : -1;   // last visible position
  u32x4 qf[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    qf[s] = u32x4{0, 0, 0, 0};
    if (row_ok)
      qf[s] = ld16((const uint16_t*)a.q + q_row * a.q_rs + (int64_t)head * HD + s * 32 + lg * 8);
  }

  const int first_new = len - a.nq_tok + 1;    // from here on only later drafts see
  bool odd = false;                            // a non-finite value was among those
  float m = kNone, l = 0.f;
  f32x4 O[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) O[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float c = a.scale * 1.4426950408889634f;
  const uint16_t* const kbase = (const uint16_t*)a.kc.p + (int64_t)kvh * a.kc.head_s;
  const uint16_t* const vbase = (const uint16_t*)a.vc.p + (int64_t)kvh * a.vc.head_s;

  // A tile lies in one page (pages are multiples of 16 tokens). A page id
  // outside the cache makes the tile invisible.
  auto load_k = [&](u32x4* k, int64_t pg, int in) {
    const uint16_t* kp = kbase + pg * a.kc.block_s + (int64_t)(in + l16) * a.kc.token_s + lg * 8;
#pragma unroll
    for (int s = 0; s < KS; ++s) k[s] = ld16(kp + s * 32);
  };
  auto load_v = [&](ValueRun<VR> (*v)[VW], int64_t pg, int in) {
    const uint16_t* vp = vbase + pg * a.vc.block_s + (int64_t)(in + lg * 4) * a.vc.token_s + l16 * VR;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < VW; ++u)
        v[i][u] = *(const ValueRun<VR>*)(vp + (int64_t)i * a.vc.token_s + u * 16 * VR);
  };
  // The next tile's keys and values are loaded as soon as this one's have been
  // used; four workgroups a CU (128 registers) hide what is left of the latency.
  struct {
    u32x4 k[KS];
    ValueRun<VR> v[4][VW];
    bool ok;
  } cur;
  auto in_cache = [&](int pg) { return pg >= 0 && pg < a.num_blocks; };
  int64_t pg = in_cache(page) ? page : 0;
  if (t0 < t_hi) {
    cur.ok = in_cache(page);
    load_k(cur.k, pg, t0 % a.block_size);
    load_v(cur.v, pg, t0 % a.block_size);
  }
  for (; t0 < t_hi; t0 += 4 * kTile) {
    const bool more = t0 + 4 * kTile < t_hi;
    const bool next_ok = in_cache(page_next);
    const int in = (t0 + 4 * kTile) % a.block_size;
    pg = next_ok ? page_next : 0;
    page_next = page_of(t0 + 8 * kTile);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, cur.k[ks]),
                                                  __builtin_bit_cast(bf16x8, qf[ks]), s, 0, 0, 0);
    if (more) load_k(cur.k, pg, in);
    float top = kNone;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + lg * 4 + i;
      // positions behind the tile's last visible one hold anything, NaN included
      s[i] = cur.ok && t <= limit && t < t_hi ? s[i] * c : -INFINITY;
      top = fmaxf(top, s[i]);
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    // the accumulators are rescaled only when some row's maximum grows
    if (__any(top > m)) {
      const float mn = fmaxf(m, top);
      const float f = exp2_(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float fi = __shfl(f, lg * 4 + i);
#pragma unroll
        for (int d = 0; d < VPL; ++d) O[d][i] *= fi;
      }
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = exp2_(s[i] - m);
      l += p[i];
    }
    // Value rows behind the visible ones hold anything, NaN included, which a
    // weight of 0 would not undo: they count as zeros. So do non-finite values
    // that only later drafts see; they are added after the loop, to those alone.
    if (a.nq_tok > 1 && t0 + kTile > first_new) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < VW; ++u)
#pragma unroll
          for (int e = 0; e < VR / 2; ++e) {
            const uint32_t x = cur.v[i][u][e], y = finite_pair(x);
            if (y != x && t0 + lg * 4 + i >= first_new && t0 + lg * 4 + i < t_hi && cur.ok) {
              cur.v[i][u][e] = y;
              odd = true;
            }
          }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool live = cur.ok && t0 + lg * 4 + i < t_hi;
#pragma unroll
      for (int u = 0; u < VW; ++u) {
#pragma unroll
        for (int e = 0; e < VR / 2; ++e) {
          const uint32_t x = live ? cur.v[i][u][e] : 0u;
          O[u * VR + 2 * e] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              p[i], __uint_as_float(x << 16), O[u * VR + 2 * e], 0, 0, 0);
          O[u * VR + 2 * e + 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              p[i], __uint_as_float(x & 0xFFFF0000u), O[u * VR + 2 * e + 1], 0, 0, 0);
        }
      }
    }
    if (more) load_v(cur.v, pg, in);
    cur.ok = next_ok;
  }
  if (__any(odd)) {
#pragma unroll 1
    for (int t = max(first_new, t_lo); t < t_hi; ++t) {
      if ((((t - t_lo) / kTile) & 3) != w) continue;
      const int b = t / a.block_size, page = table[b];
      if (page < 0 || page >= a.num_blocks) continue;
      const uint16_t* vp = vbase + page * a.vc.block_s + (int64_t)(t - b * a.block_size) * a.vc.token_s + l16 * VR;
      bool sees[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sees[i] = __shfl(limit, lg * 4 + i) >= t;
#pragma unroll
      for (int u = 0; u < VW; ++u) {
        const ValueRun<VR> run = *(const ValueRun<VR>*)(vp + u * 16 * VR);
#pragma unroll
        for (int e = 0; e < VR; ++e) {
          const uint32_t x = run[e / 2];
          const float y = __uint_as_float(e & 1 ? x & 0xFFFF0000u : x << 16);
          const bool add = !(fabsf(y) < INFINITY);
#pragma unroll
          for (int i = 0; i < 4; ++i) O[u * VR + e][i] += add && sees[i] ? y : 0.f;
        }
      }
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  // join the four waves: wave 0 takes in the others' parts. O[u VR + e] of a
  // lane is value (16 u + l16) VR + e of rows 4 lg + i; F: in fours.
  constexpr int F = VR / 4;
  if (w > 0) {
    if (lg == 0) {
      ml[w - 1][l16] = m;
      ll[w - 1][l16] = l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < VW * F; ++u)
        *(f32x4*)&Ol[w - 1][(lg * 4 + i) * HD + (u / F * 16 + l16) * VR + u % F * 4] =
            f32x4{O[u * 4][i], O[u * 4 + 1][i], O[u * 4 + 2][i], O[u * 4 + 3][i]};
  }
  __syncthreads();
  if (w > 0) return;
  float mt = m;
#pragma unroll
  for (int x = 0; x < 3; ++x) mt = fmaxf(mt, ml[x][l16]);
  const float f0 = exp2_(m - mt);
  float lt = l * f0, fx[3];
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    fx[x] = exp2_(ml[x][l16] - mt);
    lt += ll[x][l16] * fx[x];
  }
  const float inv = a.splits > 1 ? 1.f : (lt > 0.f ? 1.f / lt : 0.f);
  const int64_t n_rows = (int64_t)a.batch * a.nq_tok * a.nq;
  float* const wo = a.ws + values_at(n_rows * a.splits);
  const int64_t part = (q_row * a.nq + head) * a.splits + split;
  if (a.splits > 1 && row_ok && lg == 0) {
    a.ws[part * 2] = mt;
    a.ws[part * 2 + 1] = lt;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int src = lg * 4 + i;             // the row held in register i
    const float g0 = __shfl(f0, src), gi = __shfl(inv, src);
    const float g1 = __shfl(fx[0], src), g2 = __shfl(fx[1], src), g3 = __shfl(fx[2], src);
    const int rr = rg * kRows + src;
    const int jj = rr / group, hh = kvh * group + rr - jj * group;
    const int64_t qr = (int64_t)r * a.nq_tok + jj;
#pragma unroll
    for (int u = 0; u < VW * F; ++u) {
      const int col = (u / F * 16 + l16) * VR + u % F * 4, at = src * HD + col;
      const f32x4 a1 = *(const f32x4*)&Ol[0][at], a2 = *(const f32x4*)&Ol[1][at],
                  a3 = *(const f32x4*)&Ol[2][at];
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] = (O[u * 4 + e][i] * g0 + a1[e] * g1 + a2[e] * g2 + a3[e] * g3) * gi;
      if (rr < rows) {
        if (a.splits > 1) {
          *(f32x4*)(wo + ((qr * a.nq + hh) * a.splits + split) * HD + col) = y;
        } else {
          f32x2 y0 = {y[0], y[1]}, y1 = {y[2], y[3]};
          *(uint2*)((uint16_t*)a.out + qr * a.out_rs + (int64_t)hh * HD + col) =
              uint2{__builtin_bit_cast(uint32_t, __builtin_convertvector(y0, bf16x2)),
                    __builtin_bit_cast(uint32_t, __builtin_convertvector(y1, bf16x2))};
        }
      }
    }
  }
}

// Adds the splits of a query row: a workgroup per row, its waves take splits in
// turn, hd/64 values a lane. Up to 16 loads one after another in a wave: 7 us for
// 64 splits of 48 rows, 9 us for 16 of 4,096.
template <int HD>
__global__ __launch_bounds__(kBlock) void attn_join(PagedAttnArgs a) {
  constexpr int N = HD / 64;
  __shared__ float part_s[3][HD];
  const int64_t n_rows = (int64_t)a.batch * a.nq_tok * a.nq;
  const int64_t row = blockIdx.x;
  const int lane = (int)(threadIdx.x & 63);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t q_row = row / a.nq;
  const int head = (int)(row - q_row * a.nq);
  const int r = (int)(q_row / a.nq_tok);
  const int len = min(max(a.lens[r], 0), a.max_len);
  const int n = max(1, min(a.splits, (len + a.split_len - 1) / a.split_len));
  const float* ml = a.ws + row * a.splits * 2;
  const float* part = a.ws + values_at(n_rows * a.splits) + row * a.splits * HD + lane * N;
  const float mine = lane < n ? ml[lane * 2] : kNone;
  float lt = lane < n ? ml[lane * 2 + 1] : 0.f;
  float y[N];
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = 0.f;
  float mt = mine;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d));
  const float f = lane < n ? exp2_(mine - mt) : 0.f;
  lt *= f;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) lt += __shfl_xor(lt, d);
  for (int s = w; s < n; s += 4) {
    const float fs = __shfl(f, s);
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = fmaf(part[(int64_t)s * HD + e], fs, y[e]);
  }
  if (w > 0) {
#pragma unroll
    for (int e = 0; e < N; ++e) part_s[w - 1][lane * N + e] = y[e];
  }
  __syncthreads();
  if (w > 0) return;
  const float inv = lt > 0.f ? 1.f / lt : 0.f;
  uint16_t* o = (uint16_t*)a.out + q_row * a.out_rs + (int64_t)head * HD + lane * N;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float t = (y[e] + part_s[0][lane * N + e]) + (part_s[1][lane * N + e] + part_s[2][lane * N + e]);
    f32x2 p = {t * inv, 0.f};
    o[e] = (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
  }
}

int64_t plan_paged_attn(PagedAttnArgs* a) {
  const int64_t rows = (int64_t)(a->nq / a->nkv) * a->nq_tok;
  const int64_t base = (int64_t)a->batch * a->nkv * ((rows + kRows - 1) / kRows);
  const int64_t unit = 4 * kTile;            // tokens of one turn of the four waves
  const int64_t units = std::max<int64_t>(1, (a->max_len + unit - 1) / unit);
  // Eight workgroups a CU, or sixteen where they come from the split alone
  // (lengths differ, and a short request's splits end at once: 64 x 4 drafts
  // over up to 8,192 tokens took 159 us with eight, 140 with sixteen or more).
  // Not more than one for each 512 tokens or part of them: a length just above
  // 512 is two splits of 320.
  const int64_t cus = device_cus(), want = base >= 4 * cus ? 8 * cus : 16 * cus;
  int64_t splits = std::min<int64_t>({(want + base - 1) / base, (units + 7) / 8, kMaxSplits});
  splits = std::max<int64_t>(splits, 1);
  const int64_t per = (units + splits - 1) / splits;
  splits = (units + per - 1) / per;
  a->splits = (int32_t)splits;
  // Where workgroups wait for a CU, the longest requests go first and the last to
  // start are short. As they come / so, 16 query and 4 key/value heads x 128: 512
  // requests of up to 2,048 tokens 233 / 208 us, 1,000 tokens 123 / 110, 400 tokens
  // 55 / 55, 200 tokens 27 / 32 and 100 tokens 20 / 25, where each workgroup's look
  // at all lengths outweighs it; 400 x 4 drafts of up to 1,000 tokens 136 / 129; 64 x 4
  // of up to 8,192 127-130 / 116-129. Hence 512 tokens or more. With 1,000 requests, twice
  // the lengths to look at, 2,048 tokens 422 / 398 and 200 tokens 54 / 74: kSortMax
  // stays at 512. A CU holds four workgroups, or two of 256-wide heads; the order
  // made no difference between two and four there (300 requests x 2 heads, 146 us).
  a->sorted = base * splits > 4 * cus && a->batch > 1 && a->batch <= kSortMax && a->max_len >= 512;
  a->split_len = (int32_t)(per * unit);
  if (splits == 1) return 0;
  const int64_t parts = (int64_t)a->batch * a->nq_tok * a->nq * splits;
  return (values_at(parts) + parts * a->hd) * (int64_t)sizeof(float);
}

namespace {
template <int HD>
hipError_t launch_hd(const PagedAttnArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)(a.nq / a.nkv) * a.nq_tok;
  const int64_t grid = (int64_t)a.batch * a.nkv * ((rows + kRows - 1) / kRows) * a.splits;
  if (grid > 0x7FFFFFFFLL) return hipErrorNotSupported;
  hipLaunchKernelGGL((attn_split<HD>), dim3((unsigned)grid), dim3(kBlock), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t n_rows = (int64_t)a.batch * a.nq_tok * a.nq;
  hipLaunchKernelGGL((attn_join<HD>), dim3((unsigned)n_rows), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_paged_attn(const PagedAttnArgs& a, hipStream_t s) {
  switch (a.hd) {
    case 64: return launch_hd<64>(a, s);
    case 128: return launch_hd<128>(a, s);
    case 256: return launch_hd<256>(a, s);
  }
  return hipErrorNotSupported;
}

}  // namespace sc
