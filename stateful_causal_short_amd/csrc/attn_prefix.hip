// Attention of many requests over a prefix that they share.
//
// The requests of a group have the same leading P tokens in their caches. All rows of
// the group (requests x new tokens x query heads of a key/value head) then share
// each of those keys, and the prefix is read for all at once:
//
//   (m, l, O)_prefix = max, sum and sum_t p_t v_t over [0, P)       attn_prefix
//   (m, l, O)_own    = the same over [P, len), request by request   attn_split
//   out = sum_x 2^(m_x - m) O_x / sum_x 2^(m_x - m) l_x             attn_prefix_join
//
// One request reads P tokens for a handful of rows; a group does 4 P head_dim
// operations a row and reads P tokens once for 32 rows a wave, so matrix products
// bound it from about 200 rows on and bytes below.
//
// A wave owns 32 rows; up to eight waves of a workgroup share tiles of 32 or 64 keys and
// values in LDS, double buffered, on their way through registers (quantised
// caches are widened there). Scores are taken transposed, keys as the left operand
// of 32x32x16 bf16 products: a lane then has 16 scores of one row per 32 tokens,
// its maximum and sum need one exchange with the other half-wave, and rescaling the
// output is a product by a lane's own factor. The same registers, rounded to bf16,
// are the right operand of the second product, values transposed x weights, whose
// inner index counts the tokens in the order in which they lie there; the transposing
// LDS read brings the values' columns in that order.
//
// Weights are rounded to bf16 (by 2^-8 of each at most), and the sum is taken of the rounded ones, so
// that their mean stays one of the values: the error is that of the values' spread,
// averaged over the tokens, beside 2^-8 for the output's own rounding. Scores,
// maxima, sums and outputs are fp32.
#include "attn_device.hpp"
#include "fp8_device.hpp"

#include <algorithm>

namespace sc {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

namespace {

constexpr int kWaveRows = 32;
constexpr int kMaxPrefixSplits = 96;
constexpr int kMaxOwnSplits = 32;
// A row's maximum may pass the one that its weights refer to by 2^kSlack before the
// outputs are rescaled: weights then reach 256, far from any limit of bf16 or fp32.
constexpr float kSlack = 8.f;

// Tokens of a tile.
constexpr int tile_tokens(int hd, int waves) { return hd == 64 || (hd == 128 && waves >= 4) ? 64 : 32; }

// Where 16-byte chunk c of a tile's row lies in it: chunks are dealt so that eight rows'
// same chunk (a key read) and four rows' same pair of chunks (a transposing read)
// fall into different banks.
template <int HD>
__device__ __forceinline__ int chunk_at(int row, int c) {
  return c ^ (HD == 64 ? (row >> 1 & 3) * 2 : (row & 7) * 2);
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  f32x2 p = {x, y};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}

// The group of a row tile and the tile's number in it (-1: there is no such tile).
__device__ __forceinline__ int group_of_tile(const PagedAttnArgs& a, int rows_each, int tile_rows, int* tile) {
  const int lane = (int)(threadIdx.x & 63);
  int left = *tile;
  for (int u = 0; u < a.groups; u += 64) {
    int n = 0;
    if (u + lane < a.groups) {
      const int lo = min(max(a.group_starts[u + lane], 0), a.batch);
      const int hi = min(max(a.group_starts[u + lane + 1], lo), a.batch);
      n = (int)(((int64_t)(hi - lo) * rows_each + tile_rows - 1) / tile_rows);
    }
    int end = n;                      // tiles up to and with this lane's group
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int x = __shfl_up(end, d);
      end += lane >= d ? x : 0;
    }
    const uint64_t before = __ballot(end <= left);
    if (~before) {
      const int at = __ffsll((unsigned long long)~before) - 1;
      *tile = left - (at > 0 ? __shfl(end, at > 0 ? at - 1 : 0) : 0);
      return u + at;
    }
    left -= __shfl(end, 63);
  }
  return -1;
}

}  // namespace

template <int HD, int WAVES, bool FP8>
__global__ __launch_bounds__(WAVES * 64, HD == 256 || WAVES == 1 ? 1 : 2) void attn_prefix(PagedAttnArgs a) {
  constexpr int TN = tile_tokens(HD, WAVES);
  constexpr int NT = WAVES * 64;
  constexpr int M = WAVES * kWaveRows;
  constexpr int RC = HD / 8;                  // 16-byte chunks of a row
  constexpr int CH = TN * RC / NT;            // ... of a tile, per thread
  constexpr int KS = HD / 16, DB = HD / 32, TB = TN / 32;
  static_assert(TN * RC % NT == 0 && 64 % RC == 0, "a thread's chunks, a wave's rows");
  __shared__ __align__(16) uint16_t Kl[2][TN * HD], Vl[2][TN * HD];
  __shared__ int live_s[2][TN / kTile];

  // A key/value head's split of the prefix is read by all its row tiles: neighbours in
  // this order, which is dealt to the XCDs in eight pieces.
  const unsigned total = (unsigned)a.row_tiles * (unsigned)a.nkv * (unsigned)a.prefix_splits;
  const unsigned piece = (total + kXcds - 1) / kXcds;
  const unsigned id = (blockIdx.x % kXcds) * piece + blockIdx.x / kXcds;
  if (id >= total) return;
  int tile = (int)(id % (unsigned)a.row_tiles);
  const unsigned pair = id / (unsigned)a.row_tiles;
  const int kvh = (int)(pair % (unsigned)a.nkv), split = (int)(pair / (unsigned)a.nkv);

  const int lane = (int)(threadIdx.x & 63);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l32 = lane & 31, half = lane >> 5;
  const int group = a.nq / a.nkv, rows_each = group * a.nq_tok;
  const int g = __builtin_amdgcn_readfirstlane(group_of_tile(a, rows_each, M, &tile));
  if (g < 0) return;
  const int r_lo = min(max(a.group_starts[g], 0), a.batch);
  const int r_hi = min(max(a.group_starts[g + 1], r_lo), a.batch);
  const int P = min(max(a.prefix_lens[g], 0), a.max_prefix);
  const int t_lo = split * a.prefix_split_len, t_hi = min(P, t_lo + a.prefix_split_len);
  if (t_lo >= t_hi) return;
  // the pages are those of the first request that sees the whole prefix
  int r_first = -1;
  for (int u = r_lo; u < r_hi; u += 64) {
    const uint64_t in = __ballot(u + lane < r_hi && min(a.lens[u + lane], a.max_len) - a.nq_tok + 1 >= P);
    if (in) {
      r_first = u + __ffsll((unsigned long long)in) - 1;
      break;
    }
  }
  if (r_first < 0) return;
  const int32_t* const table = a.table + (int64_t)r_first * a.table_rs;

  // this lane's query row: head kvh * group + gi of new token j of request r
  const int64_t row = (int64_t)tile * M + w * kWaveRows + l32;
  bool row_ok = row < (int64_t)(r_hi - r_lo) * rows_each;
  const int rr = row_ok ? (int)row : 0;
  const int r = r_lo + rr / rows_each, in_r = rr % rows_each;
  const int j = in_r / group, head = kvh * group + in_r - j * group;
  row_ok = row_ok && min(a.lens[r], a.max_len) - a.nq_tok + 1 >= P;
  const bool busy = __any(row_ok);
  const int64_t q_row = (int64_t)r * a.nq_tok + j;
  // the maximum is taken of unscaled scores: their factor is made positive
  const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
  u32x4 qf[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    qf[s] = u32x4{0, 0, 0, 0};
    if (row_ok && a.scale != 0.f)
      qf[s] = ld16((const uint16_t*)a.q + q_row * a.q_rs + (int64_t)head * HD + s * 16 + half * 8);
    if (a.scale < 0.f) qf[s] ^= 0x80008000u;
  }

  // Tile to registers, registers to LDS. A thread's chunks lie one after another in
  // rows of the tile, a wave's in whole rows of one 16-token piece and so of one page.
  const int c0 = (int)threadIdx.x % RC;
  u32x4 kr[CH], vr[CH];
  uint32_t ks[CH], vs[CH];
  bool live[CH];
  auto load_tile = [&](int t) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int row = (i * NT + (int)threadIdx.x) / RC;                  // in the tile
      const int piece16 = ((i * NT + w * 64) / RC) & ~(kTile - 1);       // uniform
      const int tp = t + piece16;
      const int b = tp / a.block_size;
      const int pg = tp < t_hi ? table[b] : -1;
      const bool ok = pg >= 0 && pg < a.num_blocks;
      live[i] = ok && t + row < t_hi;
      const int64_t page = ok ? pg : 0;
      const int in = tp - b * a.block_size + (row & (kTile - 1));
      if constexpr (FP8) {
        const uint8_t* kp = (const uint8_t*)a.kc8.p + (int64_t)kvh * a.kc8.head_s + page * a.kc8.block_s;
        const uint8_t* vp = (const uint8_t*)a.vc8.p + (int64_t)kvh * a.vc8.head_s + page * a.vc8.block_s;
        const uint2 x = *(const uint2*)(kp + (int64_t)in * a.kc8.token_s + c0 * 8);
        const uint2 y = *(const uint2*)(vp + (int64_t)in * a.vc8.token_s + c0 * 8);
        kr[i] = u32x4{x.x, x.y, 0, 0};
        vr[i] = u32x4{y.x, y.y, 0, 0};
        ks[i] = a.kc8.scale[page * a.kc8.scale_block_s + kvh * a.kc8.scale_head_s + in];
        vs[i] = a.vc8.scale[page * a.vc8.scale_block_s + kvh * a.vc8.scale_head_s + in];
      } else {
        const uint16_t* kp = (const uint16_t*)a.kc.p + (int64_t)kvh * a.kc.head_s + page * a.kc.block_s;
        const uint16_t* vp = (const uint16_t*)a.vc.p + (int64_t)kvh * a.vc.head_s + page * a.vc.block_s;
        kr[i] = ld16(kp + (int64_t)in * a.kc.token_s + c0 * 8);
        vr[i] = ld16(vp + (int64_t)in * a.vc.token_s + c0 * 8);
      }
    }
  };
  auto store_tile = [&](int buf, int t) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int row = (i * NT + (int)threadIdx.x) / RC;
      u32x4 k = kr[i], v = vr[i];
      if constexpr (FP8) {
        k = fp8_to_bf16(k[0], k[1], scale_float(ks[i]));
        v = fp8_to_bf16(v[0], v[1], scale_float(vs[i]));
      }
      // values of tokens that no row sees count as zeros: a weight of 0 would not
      // undo an infinity or a NaN
      if (!live[i]) v = u32x4{0, 0, 0, 0};
      const int at = row * HD + chunk_at<HD>(row, c0) * 8;
      st16(&Kl[buf][at], k);
      st16(&Vl[buf][at], v);
      if ((row & (kTile - 1)) == 0 && c0 == 0) live_s[buf][row / kTile] = live[i];
    }
  };

  float m = kNone, l = 0.f;
  f32x16 O[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) O[d][i] = 0.f;

  // where this lane reads: keys by row, values four tokens by sixteen columns
  int k_at[KS], v_at[DB];
#pragma unroll
  for (int s = 0; s < KS; ++s) k_at[s] = l32 * HD + chunk_at<HD>(l32, 2 * s + half) * 8;
  const int v_row = half * 4 + (lane >> 2 & 3);
#pragma unroll
  for (int d = 0; d < DB; ++d)
    v_at[d] = v_row * HD + chunk_at<HD>(v_row, d * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1)) * 8 + (lane & 1) * 4;

  auto compute = [&](int buf, int t) {
    const uint16_t* const K = Kl[buf];
    const uint16_t* const V = Vl[buf];
    bool whole = t + TN <= t_hi;
    uint32_t seen = 0;
#pragma unroll
    for (int x = 0; x < TN / kTile; ++x) seen |= (live_s[buf][x] ? 1u : 0u) << x;
    seen = __builtin_amdgcn_readfirstlane((int)seen);
    whole = whole && seen == (1u << (TN / kTile)) - 1;
    f32x16 s[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
    for (int x = 0; x < KS; ++x)
#pragma unroll
      for (int b = 0; b < TB; ++b)
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, ld16(K + k_at[x] + b * 32 * HD)),
            __builtin_bit_cast(bf16x8, qf[x]), s[b], 0, 0, 0);
    if (!whole) {
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int at = b * 32 + (i >> 2) * 8 + half * 4 + (i & 3);
          if (t + at >= t_hi || !(seen >> (at / kTile) & 1)) s[b][i] = -INFINITY;
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    top = fmaxf(top, __shfl_xor(top, 32)) * c;
    if (__any(top > m + kSlack)) {
      const float mn = fmaxf(m, top);
      const float f = exp2_(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[d][i] *= f;
    }
    uint32_t p[TB * 8];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[b * 8 + i] = pack_bf16(exp2_(fmaf(s[b][2 * i], c, -m)), exp2_(fmaf(s[b][2 * i + 1], c, -m)));
        l += __uint_as_float(p[b * 8 + i] << 16) + __uint_as_float(p[b * 8 + i] & 0xFFFF0000u);
      }
#pragma unroll
    for (int x = 0; x < TN / 16; ++x) {
      const u32x4 pf = {p[x * 4], p[x * 4 + 1], p[x * 4 + 2], p[x * 4 + 3]};
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(V + v_at[d] + x * 16 * HD));
        const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(V + v_at[d] + (x * 16 + 8) * HD));
        struct { s16x4 a, b; } v = {v0, v1};
        O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v),
                                                       __builtin_bit_cast(bf16x8, pf), O[d], 0, 0, 0);
      }
    }
  };

  load_tile(t_lo);
  store_tile(0, t_lo);
  __syncthreads();
  int buf = 0;
  for (int t = t_lo; t < t_hi; t += TN, buf ^= 1) {
    const bool more = t + TN < t_hi;
    if (more) load_tile(t + TN);
    if (busy) compute(buf, t);
    if (more) store_tile(buf ^ 1, t + TN);
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (!row_ok) return;
  const int row_parts = a.prefix_splits + a.splits;
  const int64_t n_rows = (int64_t)a.batch * a.nq_tok * a.nq;
  const int64_t part = (q_row * a.nq + head) * row_parts + split;
  if (half == 0) {
    a.ws[part * 2] = m;
    a.ws[part * 2 + 1] = l;
  }
  float* const wo = a.ws + values_at(n_rows * row_parts) + part * HD + half * 4;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(f32x4*)(wo + d * 32 + i * 8) = f32x4{O[d][i * 4], O[d][i * 4 + 1], O[d][i * 4 + 2], O[d][i * 4 + 3]};
}

// Adds a query row's parts, those of the prefix and of its own tokens. WPR waves of
// a workgroup per row take parts in turn, hd/64 values a lane.
template <int HD, int WPR>
__global__ __launch_bounds__(kBlock) void attn_prefix_join(PagedAttnArgs a, int unit) {
  constexpr int N = HD / 64, PER = 4 / WPR;
  constexpr int NP = (kMaxPrefixSplits + kMaxOwnSplits) / 64;
  __shared__ float part_s[4][HD];
  const int64_t n_rows = (int64_t)a.batch * a.nq_tok * a.nq;
  const int lane = (int)(threadIdx.x & 63);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t row = (int64_t)blockIdx.x * PER + w / WPR;
  const bool ok = row < n_rows;
  float y[N], lt = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = 0.f;
  if (ok) {
    const int r = (int)(row / a.nq / a.nq_tok);
    const int len = min(max(a.lens[r], 0), a.max_len);
    const int start = shared_tokens(a, r, len);
    const int split_len = own_split_len(a, start, len, unit);
    const int n1 = start > 0 ? (start + a.prefix_split_len - 1) / a.prefix_split_len : 0;
    const int n2 = max(1, (max(len - (start & ~(kTile - 1)), 0) + split_len - 1) / split_len);
    const int row_parts = a.prefix_splits + a.splits;
    const float* ml = a.ws + row * row_parts * 2;
    const float* part = a.ws + values_at(n_rows * row_parts) + row * row_parts * HD + lane * N;
    float mi[NP], f[NP], mt = kNone;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int x = u * 64 + lane;
      const bool in = x < n1 || (x >= a.prefix_splits && x < a.prefix_splits + n2);
      mi[u] = in ? ml[x * 2] : kNone;
      f[u] = in ? ml[x * 2 + 1] : 0.f;
      mt = fmaxf(mt, mi[u]);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) mt = fmaxf(mt, __shfl_xor(mt, d));
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const float e = exp2_(mi[u] - mt);
      lt += f[u] * e;
      f[u] = e;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) lt += __shfl_xor(lt, d);
    // the i-th part there is
    for (int i = w % WPR; i < n1 + n2; i += WPR) {
      const int x = i < n1 ? i : a.prefix_splits + i - n1;
      float fx = __shfl(f[0], x & 63);
#pragma unroll
      for (int u = 1; u < NP; ++u) {
        const float z = __shfl(f[u], x & 63);
        fx = x >= u * 64 ? z : fx;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = fmaf(part[(int64_t)x * HD + e], fx, y[e]);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < N; ++e) part_s[w][lane * N + e] = y[e];
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int e = 0; e < N; ++e)
      y[e] = (y[e] + part_s[1][lane * N + e]) + (part_s[2][lane * N + e] + part_s[3][lane * N + e]);
  }
  if (!ok) return;
  const float inv = lt > 0.f ? 1.f / lt : 0.f;
  uint16_t* o = (uint16_t*)a.out + row / a.nq * a.out_rs + row % a.nq * HD + lane * N;
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = (uint16_t)pack_bf16(y[e] * inv, 0.f);
}

int64_t plan_paged_attn_prefix(PagedAttnArgs* a) {
  const int64_t rows_each = (int64_t)(a->nq / a->nkv) * a->nq_tok;
  const int64_t rows = a->batch * rows_each;
  const int64_t groups = std::max<int64_t>(1, std::min(a->groups, a->batch));
  const int64_t cus = device_cus();
  // as many waves as an average group has rows for; 256-wide heads leave registers for
  // four, and a tile of them is too much for one wave to move
  const int most = a->hd == 256 ? 4 : 8;
  a->waves = a->hd == 256 ? 2 : 1;
  while (a->waves < most && (int64_t)a->waves * kWaveRows * groups < rows) a->waves *= 2;
  const int64_t m = (int64_t)a->waves * kWaveRows, tn = tile_tokens(a->hd, a->waves);
  const int64_t tiles = (rows - groups) / m + groups;   // the groups' last tiles may be part
  const int64_t each = tiles * a->nkv;                  // workgroups of a split
  const int64_t units = (a->max_prefix + tn - 1) / tn;
  // Splits of the prefix: those for which rounds of workgroups on the chip, each as long as
  // its tiles and about 4 us of start and end, and the join's traffic come out shortest.
  const int64_t per_cu = a->waves == 8 ? 1 : a->waves == 4 ? 2 : 4;
  const double tile_us = per_cu * std::max(m * tn * a->hd * 4 / 3.0e6, tn * a->hd * 4 / 2.0e4);
  const double part_us = (double)rows * a->nkv * a->hd * 8 / 4.0e6;
  int64_t best = 1;
  double best_us = 0;
  for (int64_t s = 1; s <= std::min<int64_t>(units, kMaxPrefixSplits); ++s) {
    const int64_t rounds = (each * s + per_cu * cus - 1) / (per_cu * cus);
    const double us = rounds * ((units + s - 1) / s * tile_us + 4) + s * part_us;
    if (s == 1 || us < best_us) best = s, best_us = us;
  }
  const int64_t per = std::max<int64_t>(1, (units + best - 1) / best);
  a->prefix_splits = (int32_t)((units + per - 1) / per);
  a->prefix_split_len = (int32_t)(per * tn);
  a->row_tiles = (int32_t)std::min<int64_t>(tiles, 0x7FFFFFFF);
  // Splits of the requests' own tokens: as in plan_paged_attn, for the length that is
  // left behind the longest prefix. A longer rest is cut into as many, longer, parts.
  const int64_t base = (int64_t)a->batch * a->nkv * ((rows_each + kRows - 1) / kRows);
  const int64_t left = a->max_len - a->max_prefix + kTile;
  const int64_t want = base >= 4 * cus ? 8 * cus : 16 * cus;
  a->splits = (int32_t)std::max<int64_t>(
      1, std::min<int64_t>({(want + base - 1) / base, (left + 511) / 512, kMaxOwnSplits}));
  a->sorted = 0;
  if (tiles * a->nkv * std::max(a->prefix_splits, 1) > 0x7FFFFFF0LL) return -1;
  const int64_t parts = (int64_t)a->batch * a->nq_tok * a->nq * (a->prefix_splits + a->splits);
  return (values_at(parts) + parts * a->hd) * (int64_t)sizeof(float);
}

namespace {
template <int HD, int WAVES, bool FP8>
void launch_prefix(const PagedAttnArgs& a, hipStream_t s) {
  const unsigned total = (unsigned)a.row_tiles * (unsigned)a.nkv * (unsigned)a.prefix_splits;
  const unsigned grid = (total + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((attn_prefix<HD, WAVES, FP8>), dim3(grid), dim3(WAVES * 64), 0, s, a);
}

template <int HD, bool FP8>
hipError_t launch_hd(const PagedAttnArgs& a, hipStream_t s) {
  if (a.prefix_splits > 0) {
    if (a.waves == 2) launch_prefix<HD, 2, FP8>(a, s);
    else if (a.waves == 4) launch_prefix<HD, 4, FP8>(a, s);
    else if constexpr (HD != 256) {
      if (a.waves == 1) launch_prefix<HD, 1, FP8>(a, s);
      else launch_prefix<HD, 8, FP8>(a, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const hipError_t e = FP8 ? launch_paged_attn_after_fp8(a, s) : launch_paged_attn_after(a, s);
  if (e != hipSuccess) return e;
  // a workgroup per row until rows alone fill the chip
  const int64_t rows = (int64_t)a.batch * a.nq_tok * a.nq;
  const int unit = FP8 ? 128 : 64;
  if (rows < 8 * device_cus())
    hipLaunchKernelGGL((attn_prefix_join<HD, 4>), dim3((unsigned)rows), dim3(kBlock), 0, s, a, unit);
  else
    hipLaunchKernelGGL((attn_prefix_join<HD, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(kBlock), 0, s, a, unit);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_paged_attn_prefix(const PagedAttnArgs& a, bool fp8, hipStream_t s) {
  switch (a.hd) {
    case 64: return fp8 ? launch_hd<64, true>(a, s) : launch_hd<64, false>(a, s);
    case 128: return fp8 ? launch_hd<128, true>(a, s) : launch_hd<128, false>(a, s);
    case 256: return fp8 ? launch_hd<256, true>(a, s) : launch_hd<256, false>(a, s);
  }
  return hipErrorNotSupported;
}

}  // namespace sc
