// Attention of one or a few new tokens per request over a quantised paged cache.
//
//   o = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q.k_t - max)
//   k_t = 2^(kb_t - 127) K_t,  v_t = 2^(vb_t - 127) V_t   (K, V: rows of codes)
//
// A token's scales leave both products: they multiply its score and its weight, exactly
// as powers of two do, and the codes become bf16 as they are.
//
// As in the attention over bf16 caches, the bytes of the cache bound it, up to 16 rows
// share each key, and a workgroup has one (request, key/value head, row group, split).
// A wave's turn is 32 tokens, two tiles of 16 that may lie in two pages. A tile's
// scores are a 16x16 bf16 product with the keys as the left operand; its inner index
// runs over a head's values in the order in which 16-byte loads bring the codes. The
// two score tiles then are the left operand of a 16x16x32 product with the values, if
// its inner index counts a lane's four tokens of the first tile, then of the second.
// For that product a lane's values are turned from rows into columns, two tokens to a
// register, by byte permutes before the codes are widened. The weights enter as three
// bf16 parts, all of an fp32 value's bits: 118.3 us for 117.8 with two, 2^-16 of each
// weight (512 requests below), 89.5 for 89.0 (drafts).
//
// 16 query and 4 key/value heads x 128: 512 requests of up to 2,048 tokens, 545 MB, 114 to
// 121 us (4.6 TB/s); 3 of 131,071, 406 MB, 82 to 92 (4.4 to 4.9) and the join's 6; 64 x 4
// drafts of up to 8,192, 273 MB, 68 to 82 and 7; sessions differ. In one session the same
// loads without the products and sums took 112, 78 and 66: neither 32-byte runs of a key per
// lane nor streaming loads changed that. Registers are loaded again right after their last
// use; 164 of them let three waves run on a SIMD.
#include "attn_device.hpp"
#include "fp8_device.hpp"

#include <algorithm>

namespace sc {

namespace {

constexpr int kTurn = 2 * kTile;   // tokens of a wave's turn
// Key codes enter the product times 2^-9, none above 1, and scores get it back with
// the scale: large queries on small keys do not pass fp32's range in between.
constexpr int kKeyExp = 9;
constexpr float kKeyUnit = 1.f / (1 << kKeyExp);

// N codes (4, 8 or 16), one load.
template <int N>
using CodeRun = uint32_t __attribute__((ext_vector_type(N / 4)));

// The scale in byte i of a word, as a factor (2^-127 has no exponent of its own).
__device__ __forceinline__ float scale_of(uint32_t w, int i) {
  const uint32_t x = (i == 3 ? w >> 1 : w << (23 - 8 * i)) & 0x7F800000u;
  return __uint_as_float(x > 0x00400000u ? x : 0x00400000u);
}

__device__ __forceinline__ uint32_t byte_of(uint32_t w, int i) { return (w >> (8 * i)) & 0xFFu; }

// NaN codes (0x7F and 0xFF) of a word replaced by zeros.
__device__ __forceinline__ uint32_t finite_codes(uint32_t w) {
  uint32_t y = w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((byte_of(w, i) & 0x7Fu) == 0x7Fu) y &= ~(0xFFu << (8 * i));
  return y;
}

}  // namespace

// AFTER: as in attn.hip, the call's second half behind attn_prefix.
template <int HD, After AFTER>
__global__ __launch_bounds__(kBlock, HD == 256 ? 2 : HD == 128 ? 3 : 4) void attn_split_fp8(PagedAttnArgs a) {
  constexpr int KC = HD / 64;               // 16-byte loads of a key row per lane
  constexpr int VPL = HD / 16;              // values of a token's row per lane
  constexpr int VC = VPL / 4;               // ... in words
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
  if (AFTER == After::kNo && a.sorted) r = by_length(a, r);

  const int lane = (int)(threadIdx.x & 63);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l16 = lane & 15, lg = lane >> 4;
  int start = 0, split_len = a.split_len;
  if constexpr (AFTER != After::kNo) {
    const int len = min(max(a.lens[r], 0), a.max_len);
    start = shared_tokens(a, r, len);
    split_len = own_split_len(a, start, len, 4 * kTurn);
  }
  const int t_lo = (start & ~(kTile - 1)) + split * split_len;
  // The wave's n-th tile is at t_mine(n). Its place in the caches is kept in lane n, for 64
  // tiles at a time, so that a tile costs a few lane reads, and its page's id is there
  // long before. A tile lies in one page; below max_len it has an entry in the table.
  const int32_t* const table = a.table + (int64_t)r * a.table_rs;
  auto t_mine = [&](int n) { return (uint32_t)(t_lo + w * kTurn) + (n >> 1) * 4 * kTurn + (n & 1) * kTile; };
  auto page_of = [&](int n) {
    const uint32_t t = t_mine(n + lane);
    return t < (uint32_t)a.max_len ? table[t / a.block_size] : -1;
  };
  auto in_cache = [&](int pg) { return pg >= 0 && pg < a.num_blocks; };
  struct Places {
    int64_t k, v, ks, vs;
    uint64_t ok;           // a page id outside the cache makes the tile invisible
  };
  auto places = [&](int n, int page) {
    const int in = t_mine(n + lane) % a.block_size;
    const int64_t b = in_cache(page) ? page : 0;
    return Places{kvh * a.kc8.head_s + b * a.kc8.block_s + in * a.kc8.token_s,
                  kvh * a.vc8.head_s + b * a.vc8.block_s + in * a.vc8.token_s,
                  kvh * a.kc8.scale_head_s + b * a.kc8.scale_block_s + in,
                  kvh * a.vc8.scale_head_s + b * a.vc8.scale_block_s + in, __ballot(in_cache(page))};
  };
  int page = page_of(0);
  const int len = min(max(a.lens[r], 0), a.max_len);
  const int t_hi = min(len, t_lo + split_len);
  if (split > 0 && t_lo >= len) return;      // the join does not read such a split
  int t0 = t_lo + w * kTurn;
  const int n_tiles = t0 < t_hi ? (t_hi - t0 + 4 * kTurn - 1) / (4 * kTurn) * 2 : 0;

  // this lane's query row: head kvh * group + g of new token j
  const int row = rg * kRows + l16;
  const bool row_ok = row < rows;
  const int j = row_ok ? row / group : 0, g = row_ok ? row - j * group : 0;
  const int64_t q_row = (int64_t)r * a.nq_tok + j;
  const int head = kvh * group + g;
  const int limit = row_ok ? len - a.nq_tok + j : -1;   // last visible position
  // the columns of step (c, e): 64 c + 16 lg + 8 e, as the codes lie in the loads
  u32x4 qf[KC * 2];
#pragma unroll
  for (int s = 0; s < KC * 2; ++s) {
    qf[s] = u32x4{0, 0, 0, 0};
    if (row_ok)
      qf[s] = ld16((const uint16_t*)a.q + q_row * a.q_rs + (int64_t)head * HD + (s / 2) * 64 +
                   lg * 16 + (s & 1) * 8);
  }

  const int first_new = len - a.nq_tok + 1;    // from here on only later drafts see
  bool odd = false;                            // a NaN code was among those
  float m = kNone, l = 0.f;
  f32x4 O[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) O[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float c = a.scale * 1.4426950408889634f * (1 << kKeyExp);
  // a lane's own offsets in a tile (token strides are checked to leave 32 bits)
  const uint32_t k_lane = (uint32_t)l16 * (uint32_t)a.kc8.token_s + lg * 16;
  uint32_t v_lane[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v_lane[i] = (uint32_t)(lg * 4 + i) * (uint32_t)a.vc8.token_s + l16 * VPL;

  struct {
    u32x4 k[2][KC];
    CodeRun<VPL> v[2][4];
    uint32_t ks[2], vs[2];
  } cur;
  auto load_k = [&](const Places& x, int n) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* kp = (const uint8_t*)a.kc8.p + lane_of(x.k, n + u);
#pragma unroll
      for (int s = 0; s < KC; ++s) cur.k[u][s] = ld16(kp + k_lane + s * 64);
      cur.ks[u] = *(const uint32_t*)(a.kc8.scale + lane_of(x.ks, n + u) + lg * 4u);
    }
  };
  auto load_v = [&](const Places& x, int n) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* vp = (const uint8_t*)a.vc8.p + lane_of(x.v, n + u);
#pragma unroll
      for (int i = 0; i < 4; ++i) cur.v[u][i] = *(const CodeRun<VPL>*)(vp + v_lane[i]);
      cur.vs[u] = *(const uint32_t*)(a.vc8.scale + lane_of(x.vs, n + u) + lg * 4u);
    }
  };
  Places at = places(0, page);
  if (n_tiles > 64) page = page_of(64);
  uint32_t ok = 0;
  if (n_tiles > 0) {
    load_k(at, 0);
    load_v(at, 0);
    ok = (uint32_t)at.ok & 3;
  }
  for (int n = 0; n < n_tiles; n += 2, t0 += 4 * kTurn) {
    const bool more = n + 2 < n_tiles;
    if (more && (n + 2) % 64 == 0) {
      at = places(n + 2, page);
      if (n_tiles > n + 66) page = page_of(n + 66);
    }
    // every row sees every token of the turn
    const bool plain = ok == 3 && t0 + kTurn <= min(first_new, t_hi) && (AFTER == After::kNo || t0 >= start);
    f32x4 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < KC * 2; ++x)
        s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8, fp8_to_bf16(cur.k[u][x / 2][(x & 1) * 2], cur.k[u][x / 2][(x & 1) * 2 + 1], kKeyUnit)),
            __builtin_bit_cast(bf16x8, qf[x]), s[u], 0, 0, 0);
    }
    float top = kNone;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u][i] = s[u][i] * scale_of(cur.ks[u], i) * c;
    if (!plain) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + u * kTile + lg * 4 + i;
          // positions behind the tile's last visible one hold anything, NaN included
          if (!(ok >> u & 1) || t > limit || t >= t_hi || (AFTER != After::kNo && t < start)) {
            s[u][i] = -INFINITY;
            cur.vs[u] &= ~(0xFFu << i * 8);
          }
        }
    }
    if (more) load_k(at, (n + 2) & 63);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[u][i]);
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
    // the weights times the values' scales, in three parts
    u32x4 part[3];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float p0 = exp2_(s[u][i] - m), p1 = exp2_(s[u][i + 1] - m);
        l += p0;
        l += p1;
        f32x2 y = {p0 * scale_of(cur.vs[u], i), p1 * scale_of(cur.vs[u], i + 1)};
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          const uint32_t h = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
          part[x][u * 2 + i / 2] = h;
          y = f32x2{y[0] - __uint_as_float(h << 16), y[1] - __uint_as_float(h & 0xFFFF0000u)};
        }
      }
    // Value rows that no row of the tile sees hold anything, NaN codes included,
    // which a weight of 0 would not undo: they count as zeros. So do NaN codes that
    // only later drafts see; they are added after the loop, to those alone.
    if (!plain) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + u * kTile + lg * 4 + i;
          const bool live = (ok >> u & 1) && t < t_hi && (AFTER == After::kNo || t >= start);
#pragma unroll
          for (int x = 0; x < VC; ++x) cur.v[u][i][x] = live ? cur.v[u][i][x] : 0u;
        }
    }
    if (a.nq_tok > 1 && t0 + kTurn > first_new) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < VC; ++x) {
            const uint32_t y = cur.v[u][i][x], f = finite_codes(y);
            if (y != f && t0 + u * kTile + lg * 4 + i >= first_new) {
              cur.v[u][i][x] = f;
              odd = true;
            }
          }
    }
#pragma unroll
    for (int x = 0; x < VC; ++x) {
      uint32_t even[4], uneven[4];           // columns 4x, 4x + 1 and 4x + 2, 4x + 3 of token pairs
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t t_a = cur.v[y / 2][(y & 1) * 2][x], t_b = cur.v[y / 2][(y & 1) * 2 + 1][x];
        even[y] = __builtin_amdgcn_perm(t_b, t_a, 0x05010400u);
        uneven[y] = __builtin_amdgcn_perm(t_b, t_a, 0x07030602u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t* col = e < 2 ? even : uneven;
        u32x4 v;
#pragma unroll
        for (int y = 0; y < 4; ++y) v[y] = e & 1 ? fp8_pair_hi(col[y]) : fp8_pair_lo(col[y]);
        f32x4& o = O[x * 4 + e];
#pragma unroll
        for (int y = 0; y < 3; ++y)
          o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, part[y]),
                                                      __builtin_bit_cast(bf16x8, v), o, 0, 0, 0);
      }
    }
    if (more) {
      load_v(at, (n + 2) & 63);
      ok = (uint32_t)(at.ok >> ((n + 2) & 63)) & 3;
    }
  }
  if (__any(odd)) {
#pragma unroll 1
    for (int t = max(first_new, t_lo); t < t_hi; ++t) {
      if ((((t - t_lo) / kTurn) & 3) != w) continue;
      const int b = t / a.block_size, pg = table[b];
      if (!in_cache(pg)) continue;
      const uint8_t* vp = (const uint8_t*)a.vc8.p + kvh * a.vc8.head_s + pg * a.vc8.block_s +
                          (int64_t)(t - b * a.block_size) * a.vc8.token_s + l16 * VPL;
      bool sees[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sees[i] = __shfl(limit, lg * 4 + i) >= t;
      const CodeRun<VPL> run = *(const CodeRun<VPL>*)vp;
#pragma unroll
      for (int e = 0; e < VPL; ++e) {
        const bool add = (byte_of(run[e / 4], e & 3) & 0x7Fu) == 0x7Fu;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          O[e][i] += add && sees[i] ? __uint_as_float(0x7FC00000u) : 0.f;
      }
    }
  }
  if constexpr (AFTER == After::kWhole)
    take_prefix<HD, VPL, 1>(a, r, kvh, rg * kRows, w,
                       start > 0 ? (start + a.prefix_split_len - 1) / a.prefix_split_len : 0, m, l, O);
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  // join the four waves: wave 0 takes in the others' parts. O[d] of a lane is
  // value l16 VPL + d of rows 4 lg + i.
  if (w > 0) {
    if (lg == 0) {
      ml[w - 1][l16] = m;
      ll[w - 1][l16] = l;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < VC; ++u)
        *(f32x4*)&Ol[w - 1][(lg * 4 + i) * HD + l16 * VPL + u * 4] =
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
  const bool parts = AFTER == After::kParts || (AFTER == After::kNo && a.splits > 1);
  const float inv = parts ? 1.f : (lt > 0.f ? 1.f / lt : 0.f);
  const int64_t n_rows = (int64_t)a.batch * a.nq_tok * a.nq;
  const int row_parts = AFTER != After::kNo ? a.prefix_splits + a.splits : a.splits;
  const int my_part = AFTER != After::kNo ? a.prefix_splits + split : split;
  float* const wo = a.ws + values_at(n_rows * row_parts);
  const int64_t part = (q_row * a.nq + head) * row_parts + my_part;
  if (parts && row_ok && lg == 0) {
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
    for (int u = 0; u < VC; ++u) {
      const int col = l16 * VPL + u * 4, at = src * HD + col;
      const f32x4 a1 = *(const f32x4*)&Ol[0][at], a2 = *(const f32x4*)&Ol[1][at],
                  a3 = *(const f32x4*)&Ol[2][at];
      f32x4 y;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] = (O[u * 4 + e][i] * g0 + a1[e] * g1 + a2[e] * g2 + a3[e] * g3) * gi;
      if (rr < rows) {
        if (parts) {
          *(f32x4*)(wo + ((qr * a.nq + hh) * row_parts + my_part) * HD + col) = y;
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

int64_t plan_paged_attn_fp8(PagedAttnArgs* a) {
  const int64_t rows = (int64_t)(a->nq / a->nkv) * a->nq_tok;
  const int64_t base = (int64_t)a->batch * a->nkv * ((rows + kRows - 1) / kRows);
  const int64_t unit = 4 * kTurn;            // tokens of one turn of the four waves
  const int64_t units = std::max<int64_t>(1, (a->max_len + unit - 1) / unit);
  // Two workgroups a CU stream as fast as three (all that its registers hold), so the
  // split makes two, of 256 tokens or more. Where the requests alone give one a CU,
  // it only evens out unequal lengths, up to four a CU, if 2,048 tokens or more are left
  // to each. 16 query and 4 key/value heads x 128, us with 1, 2, 4, .. 64 splits:
  //   1 x 2,048              22 17 13 11 10 10 10
  //   1 x 8,192              78 43 26 18 14 13 13
  //   4 x 4,096              43 28 19 14 13 14 14
  //   4 of up to 32,768     262 140 75 43 28 26 31
  //   16 of up to 8,192      77 46 29 25 26 29 37
  //   16 x 32,768           368 200 126 120 125 125 132
  //   64 of up to 8,192     105 81 75 74 77 91 129
  //   64 x 2,000             33 35 36 39 46 46 46
  //   256 of up to 2,048     67 77 83 99 135 134 134
  const int64_t cus = device_cus();
  int64_t splits = base < cus ? std::min((2 * cus + base - 1) / base, units / 2)
                              : std::min(4 * cus / base, units / (2048 / unit));
  splits = std::clamp<int64_t>(splits, 1, kMaxSplits);
  const int64_t per = (units + splits - 1) / splits;
  splits = (units + per - 1) / per;
  a->splits = (int32_t)splits;
  a->split_len = (int32_t)(per * unit);
  // the longest first, as in plan_paged_attn, where some workgroups wait for a CU
  a->sorted = base * splits > 3 * cus && a->batch > 1 && a->batch <= kSortMax && a->max_len >= 512;
  if (splits == 1) return 0;
  const int64_t parts = (int64_t)a->batch * a->nq_tok * a->nq * splits;
  return (values_at(parts) + parts * a->hd) * (int64_t)sizeof(float);
}

namespace {
template <After AFTER>
hipError_t launch_split(const PagedAttnArgs& a, hipStream_t s) {
  const int64_t grid = own_attn_grid(a);
  if (grid > 0x7FFFFFFFLL) return hipErrorNotSupported;
  const dim3 g((unsigned)grid), b(kBlock);
  if (a.hd == 64) hipLaunchKernelGGL((attn_split_fp8<64, AFTER>), g, b, 0, s, a);
  else if (a.hd == 128) hipLaunchKernelGGL((attn_split_fp8<128, AFTER>), g, b, 0, s, a);
  else hipLaunchKernelGGL((attn_split_fp8<256, AFTER>), g, b, 0, s, a);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_paged_attn_fp8(const PagedAttnArgs& a, hipStream_t s) {
  const hipError_t e = launch_split<After::kNo>(a, s);
  return e != hipSuccess || a.splits == 1 ? e : launch_attn_join(a, s);
}

hipError_t launch_paged_attn_after_fp8(const PagedAttnArgs& a, hipStream_t s) {
  return a.whole ? launch_split<After::kWhole>(a, s) : launch_split<After::kParts>(a, s);
}

}  // namespace sc
