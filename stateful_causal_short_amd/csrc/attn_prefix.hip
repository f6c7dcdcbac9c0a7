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
// values in LDS, double buffered; bf16 tiles are copied there directly, quantised ones
// pass through registers and are widened. Scores are taken transposed, keys as the
// left operand of 32x32x16 bf16 products: a lane then has 16 scores of one row per 32
// tokens, its maximum and sum need one exchange with the other half-wave, and rescaling
// the output is a product by a lane's own factor. The same registers, as two bf16
// parts, are the right operands of the second product, values transposed x weights, whose
// inner index counts the tokens in the order in which they lie there; the transposing
// LDS read brings the values' columns in that order.
//
// Matrix instructions and exponentials take about the same time: scores run a tile
// ahead, and the products' instructions are issued with the exponentials, LDS reads,
// sums and the next tiles' copies between them. 2,048 rows x 4 key/value heads x 128 on
// 32,768 tokens: 194 us, 208 GFLOP with both parts of the weights, 1,070 TFLOP/s (a large
// bf16 library product reaches 1,158 here). Of weights in one part, 139 GFLOP, it took
// 146 us so; with the compiler's order 187, with this order and tiles through registers
// 174, with copies that stop the counters of LDS reads 153, with no LDS reads, copies or
// barriers at all 116. 7 us are the parts' way to the workspace. Matrix units are busy 52%
// of the cycles, and the clock falls (2.2 to 2.0 GHz) as they get busier.
//
// Weights enter the second product in two bf16 parts, the fp32 weight cut to its first
// eight bits and the rest rounded: 2^-15 of each at most. One rounded part would halve that
// product (512 requests on 32,768 tokens 223 us for 271) and cost 2^-8 of each, an error as
// large as the output's own rounding. The second part is never zero or negative, so that an
// infinite value stays one. Scores, maxima, sums and outputs are fp32.
#include "attn_device.hpp"
#include "fp8_device.hpp"

#include <algorithm>
#include <utility>

namespace sc {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// The kernel's parts are lambdas over its registers: none may become a call.
#define SC_INLINE __attribute__((always_inline))

namespace {

constexpr int kWaveRows = 32;
constexpr int kMaxPrefixSplits = 96;
constexpr int kMaxOwnSplits = 32;
constexpr int kMostTakenIn = 16;   // prefix parts that workgroups of single requests take in
// Weights refer to a power of two that is 2^kSlack above their row's maximum when it is set,
// so that the maximum may grow as much before the outputs are rescaled, and no weight is
// ever above one: sums and outputs stay as far from fp32's limits as with the maximum itself.
constexpr float kSlack = 8.f;
// A weight's second part is kMore times the weight less its first part, never zero.
constexpr float kMore = 1.f + 0x1p-20f;

// Tokens of a tile.
constexpr int tile_tokens(int hd, int waves) { return hd == 64 || (hd == 128 && waves >= 4) ? 64 : 32; }

// Where 16-byte chunk c of a tile's row lies in it. Sixteen rows' same chunk, as the lanes
// of a key read take them together, lie in different banks; so do four rows' same four
// chunks, which 32 lanes of a transposing read take.
template <int HD>
__device__ __forceinline__ int key_chunk(int row, int c) {
  return c ^ (HD == 64 ? row >> 1 & 7 : row & 15);
}
template <int HD>
__device__ __forceinline__ int value_chunk(int row, int c) {
  return c ^ (HD == 64 ? (row >> 1 & 1) * 4 : (row & 3) * 4);
}

// f(0), f(1), ... f(N - 1) with the numbers as types: what depends on one is settled when
// it is compiled, so that a sequence of steps stays one block of instructions.
template <class F, int... I>
__device__ __forceinline__ void steps_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void steps(F f) {
  steps_of(f, std::make_integer_sequence<int, N>{});
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  f32x2 p = {x, y};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}

// Reads from `bytes` behind `from` (uniform), as buffer accesses: a lane's offset has 32
// bits, nothing is read where `there` is false, and the counters of LDS reads go on
// beside one that ends in LDS, which a global access stops.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* from, bool there) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(from), (short)0, there ? 0x7FFFFFFF : 0, 0x00020000);
}
// 16 bytes a lane to LDS, lane after lane.
__device__ __forceinline__ void copy_to_lds(const uint16_t* from, int bytes, bool there, uint16_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_at(from, there),
                                           (__attribute__((address_space(3))) void*)to, 16, bytes, 0, 0, 0);
}
__device__ __forceinline__ uint2 read_codes(const uint8_t* from, int bytes, bool there) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(buffer_at(from, there), bytes, 0, 0));
}
__device__ __forceinline__ uint32_t read_scale(const uint8_t* from, int bytes, bool there) {
  return (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(buffer_at(from, there), bytes, 0, 0);
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
__global__ __launch_bounds__(WAVES * 64, HD == 256 ? 1 : 2) void attn_prefix(PagedAttnArgs a) {
  constexpr int TN = tile_tokens(HD, WAVES);
  constexpr int NT = WAVES * 64;
  constexpr int M = WAVES * kWaveRows;
  constexpr int RC = HD / 8;                  // 16-byte chunks of a row
  constexpr int CH = TN * RC / NT;            // ... of a tile, per thread
  constexpr int KS = HD / 16, DB = HD / 32, TB = TN / 32;
  static_assert(TN * RC % NT == 0 && 64 % RC == 0, "a thread's chunks, a wave's rows");
  // four arrays: loads into one and reads of another have no order between them
  __shared__ __align__(16) uint16_t K0[TN * HD], K1[TN * HD], V0[TN * HD], V1[TN * HD];

  // A key/value head's split of the prefix is read by all its row tiles: neighbours in
  // this order, which is dealt to the XCDs in eight pieces.
  const unsigned total = (unsigned)a.row_tiles * (unsigned)a.nkv * (unsigned)a.prefix_splits;
  const unsigned per_xcd = (total + kXcds - 1) / kXcds;
  const unsigned id = (blockIdx.x % kXcds) * per_xcd + blockIdx.x / kXcds;
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
  // The places of 64 pieces at a time are kept in the lanes of a register, so that a
  // piece costs a wave two lane reads and its page's division is one in 64.
  constexpr int RP = NT / RC;                        // rows of a pass of all threads
  constexpr int TP = TN / kTile;                     // pieces of a tile
  const int c0 = (int)threadIdx.x % RC;
  const int my_row = (int)threadIdx.x / RC;          // of the first pass
  const int lane_row = my_row & (kTile - 1);
  const int w_piece = w * (64 / RC) / kTile;         // of the wave's rows in a pass
  struct Places {
    int64_t at, scale_at;                            // of this lane's piece
    uint64_t ok;                                     // the pieces that are in the cache
  };
  auto page_of = [&](int t) SC_INLINE {                        // of this lane's piece of 64 from t on
    const int tp = t + lane * kTile;
    return tp < t_hi ? table[tp / a.block_size] : -1;
  };
  auto places = [&](int t, int page, const PagedCache& c, const PagedCacheFp8& c8) SC_INLINE {
    Places x;
    const int in = (t + lane * kTile) % a.block_size;
    const bool ok = page >= 0 && page < a.num_blocks;
    const int64_t b = ok ? page : 0;
    x.at = FP8 ? kvh * c8.head_s + b * c8.block_s + in * c8.token_s
               : kvh * c.head_s + b * c.block_s + in * c.token_s;
    x.scale_at = FP8 ? kvh * c8.scale_head_s + b * c8.scale_block_s + in : 0;
    x.ok = __ballot(ok);
    return x;
  };
  // Chunk i of a thread: the piece it is in, and its row's first in the piece.
  auto piece = [&](int n, int i) SC_INLINE { return n + (RP >= kTile ? i * (RP / kTile) + w_piece : i * RP / kTile); };
  constexpr auto row_in = [](int i) { return RP >= kTile ? 0 : (i * RP) & (kTile - 1); };
  // Chunk i of a tile of a bf16 cache goes to LDS past the registers, a wave's 64 chunks to
  // 1 KB in their order: the lane that fills a place takes the chunk that belongs there.
  auto copy_chunk = [&](const PagedCache& c, const Places& x, int n, int i, bool there, bool keys,
                        uint16_t* to) SC_INLINE {
    const int row = row_in(i) + lane_row;
    const int ch = keys ? key_chunk<HD>(row, c0) : value_chunk<HD>(row, c0);
    // from the piece's start, so that a lane's offset has 32 bits (token strides are checked)
    copy_to_lds((uint16_t*)c.p + lane_of(x.at, piece(n, i)), (row * (int)c.token_s + ch * 8) * 2,
                there, to + (i * NT + w * 64) * 8);
  };
  // Codes of a quantised one pass through registers and are widened there.
  constexpr int CR = FP8 ? CH : 1;
  uint2 kr[CR], vr[CR];
  uint32_t ks[CR], vs[CR];
  auto load_codes = [&](const PagedCacheFp8& c, const Places& x, int n, int i, bool there, uint2& to,
                        uint32_t& scale) SC_INLINE {
    const int row = row_in(i) + lane_row;
    to = read_codes((uint8_t*)c.p + lane_of(x.at, piece(n, i)), row * (int)c.token_s + c0 * 8, there);
    scale = read_scale(c.scale + lane_of(x.scale_at, piece(n, i)), row, there);
  };
  auto store_codes = [&](uint16_t* to, int i, bool keys, uint2 from, uint32_t scale) SC_INLINE {
    const int row = i * RP + my_row;
    const int ch = keys ? key_chunk<HD>(row, c0) : value_chunk<HD>(row, c0);
    st16(to + row * HD + ch * 8, fp8_to_bf16(from.x, from.y, scale_float(scale)));
  };
  // Values of tokens that no row sees count as zeros: a weight of 0 would not undo an
  // infinity or a NaN. `seen`: the tile's pieces that are in the cache.
  constexpr uint32_t kWhole = (1u << TP) - 1;
  auto clear_v = [&](uint16_t* V, int t, uint32_t seen) SC_INLINE {
    if (t + TN <= t_hi && seen == kWhole) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int row = i * RP + my_row;
      if (t + row >= t_hi || !(seen >> (row / kTile) & 1)) st16(V + row * HD + c0 * 8, u32x4{0, 0, 0, 0});
    }
  };

  float m = kNone, l = 0.f;
  f32x16 O[DB], S0[TB], S1[TB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) O[d][i] = 0.f;

  // where this lane reads: keys by row, values four tokens by sixteen columns
  // (step s's chunk of a key row, 2 s + half dealt, is that of step 0 with 2 s flipped)
  const int k_at = l32 * HD + key_chunk<HD>(l32, half) * 8;
  int v_at[DB];
  const int v_row = half * 4 + (lane >> 2 & 3);
#pragma unroll
  for (int d = 0; d < DB; ++d)
    v_at[d] = v_row * HD + value_chunk<HD>(v_row, d * 4 + (lane >> 4 & 1) * 2 + (lane >> 1 & 1)) * 8 + (lane & 1) * 4;

  auto scores = [&](const uint16_t* K, f32x16* s) SC_INLINE {
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
    for (int x = 0; x < KS; ++x)
#pragma unroll
      for (int b = 0; b < TB; ++b)
        s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, ld16(K + (k_at ^ x * 16) + b * 32 * HD)),
            __builtin_bit_cast(bf16x8, qf[x]), s[b], 0, 0, 0);
  };
  // scores of tokens behind the split's end or in pages outside the cache
  auto mask = [&](int t, uint32_t seen, f32x16* s) SC_INLINE {
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int at = b * 32 + (i >> 2) * 8 + half * 4 + (i & 3);
        if (t + at >= t_hi || !(seen >> (at / kTile) & 1)) s[b][i] = -INFINITY;
      }
  };
  auto largest = [&](const f32x16* s) SC_INLINE {
    float top = kNone;
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    return top;
  };
  // the running maximum takes in a tile's scores
  auto take_max = [&](float top) SC_INLINE {
    const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * c;
    if (__any(top > m)) {
      const float mn = top > m ? top + kSlack : m;
      const float f = exp2_(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) O[d][i] *= f;
    }
  };
  constexpr int NW = TB * 8;                          // words of a part of a tile's weights, two in each
  struct Two { float x, y; };
  auto exponents = [&](const f32x16* s, int x) SC_INLINE {
    return Two{fmaf(s[x / 8][x % 8 * 2], c, -m), fmaf(s[x / 8][x % 8 * 2 + 1], c, -m)};
  };
  struct Columns { s16x4 a, b; };
  auto read_v = [&](const uint16_t* V, int n) SC_INLINE {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const uint16_t* at = V + v_at[n % DB] + n / DB * 16 * HD;
    return Columns{__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)at),
                   __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(at + 8 * HD))};
  };
  auto value_step = [&](const Columns& v, const uint32_t* p, int n) SC_INLINE {
    const u32x4 pf = {p[n / DB * 4], p[n / DB * 4 + 1], p[n / DB * 4 + 2], p[n / DB * 4 + 3]};
    O[n % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v),
                                                       __builtin_bit_cast(bf16x8, pf), O[n % DB], 0, 0, 0);
  };
  // The products of a turn, the scores of the next tile (keys Kn) and the values of this one
  // (V) under each part of its weights, step by step in the order in which they are to be issued: a
  // matrix instruction, the LDS read that a later one needs, and of the weights the
  // exponent of one pair, the power of the pair before and the sum of the one before that,
  // so that no instruction waits for its neighbour. `chore(i)`, of `chores`, is what else a
  // turn has to do, the next tiles' way to LDS. The maximum of the next scores is returned.
  auto products = [&](const uint16_t* Kn, const uint16_t* V, const f32x16* cur, f32x16* next, auto chores,
                      auto chore) SC_INLINE {
    // values' steps: one with each part of the weights
    constexpr int NQ = KS * TB, NV = TB * 2 * DB * 2, AHEAD = 3;
    // steps that take weights; a pair is done two slots after its own, and in time
    constexpr int NS = NW + 2, ES = NQ + NV * 3 / 8;
    static_assert((NW + 1) * ES / NS < NQ + (NW / 4 - 1) * DB * 2 && 5 * ES / NS < NQ, "weights before their product");
    u32x4 kf[AHEAD];
    Columns vf[AHEAD];
    uint32_t p[2][NW];
    Two e[2];
    float top[2] = {kNone, kNone};
    int k_lane = k_at;
    asm volatile("" : "+v"(k_lane));                  // its steps are made anew, not kept in registers
    auto read_k = [&](int n) SC_INLINE { return ld16(Kn + (k_lane ^ n / TB * 16) + n % TB * 32 * HD); };
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) kf[n] = read_k(n);
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) next[b][i] = 0.f;
    __builtin_amdgcn_sched_barrier(0);
    steps<NQ + NV>([&](auto step) SC_INLINE {
      constexpr int n = step, nv = n - NQ;
      if constexpr (n < NQ) {
        next[n % TB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_bit_cast(bf16x8, kf[n % AHEAD]), __builtin_bit_cast(bf16x8, qf[n / TB]), next[n % TB], 0, 0, 0);
        if constexpr (n + AHEAD < NQ) kf[n % AHEAD] = read_k(n + AHEAD);
        else vf[n + AHEAD - NQ] = read_v(V, n + AHEAD - NQ);
      } else {
        value_step(vf[nv / 2 % AHEAD], p[nv % 2], nv / 2);
        if constexpr (nv % 2 == 1 && nv / 2 + AHEAD < NV / 2) vf[nv / 2 % AHEAD] = read_v(V, nv / 2 + AHEAD);
      }
      steps<NS>([&](auto slot) SC_INLINE {
        constexpr int x = slot;
        if constexpr (x * ES / NS == n) {
          if constexpr (x >= 2) {
            const Two y = e[x % 2];
            const uint32_t ux = __float_as_uint(y.x), uy = __float_as_uint(y.y);
            p[0][x - 2] = __builtin_amdgcn_perm(uy, ux, 0x07060302u);
            p[1][x - 2] = pack_bf16(fmaf(y.x, kMore, -__uint_as_float(ux & 0xFFFF0000u)),
                                    fmaf(y.y, kMore, -__uint_as_float(uy & 0xFFFF0000u)));
            l += y.x + y.y;
          }
          if constexpr (x >= 1 && x <= NW) e[(x - 1) % 2] = Two{exp2_(e[(x - 1) % 2].x), exp2_(e[(x - 1) % 2].y)};
          if constexpr (x < NW) e[x % 2] = exponents(cur, x);
        }
      });
      if constexpr (nv >= NV / 2) {
        constexpr int per = TB * 16 * 2 / NV, from = (nv - NV / 2) * per;
        steps<per>([&](auto i) SC_INLINE {
          constexpr int x = from + i;
          top[x / 2 % 2] = fmaxf(top[x / 2 % 2], next[x / 16][x % 16]);
        });
      }
      steps<decltype(chores)::value>([&](auto i) SC_INLINE {
        if constexpr (1 + i * (NQ + NV / 2) / decltype(chores)::value == n) chore(i);
      });
      // sums and maxima stay in their step
      if constexpr (nv < NV / 2) asm volatile("" : "+v"(l));
      else asm volatile("" : "+v"(l), "+v"(top[0]), "+v"(top[1]));
      __builtin_amdgcn_sched_barrier(0);
    });
    return fmaxf(top[0], top[1]);
  };

  // Scores run a tile ahead of their weights, so that the first product of the next tile
  // and the exponentials of this one have no order between them. In the turn of tile x,
  // keys of tile x + 2 and values of x + 1 go to LDS; codes were requested a turn before.
  constexpr int kSpan = 64 * kTile;                   // tokens that have their places in lanes
  int next_page = page_of(t_lo);
  Places pk = places(t_lo, next_page, a.kc, a.kc8), pv = places(t_lo, next_page, a.vc, a.vc8);
  next_page = page_of(t_lo + kSpan);
  auto piece_at = [&](int t) SC_INLINE { return (t - t_lo) / kTile & 63; };
  auto seen_at = [&](const Places& x, int t) SC_INLINE { return (uint32_t)(x.ok >> piece_at(t)) & kWhole; };
  // the places of 64 pieces begin with a tile's; the values follow the keys by a tile
  auto go_on = [&](int t) SC_INLINE {
    if (piece_at(t) == 0) pk = places(t, next_page, a.kc, a.kc8);
    if (piece_at(t - TN) == 0) {
      pv = places(t - TN, next_page, a.vc, a.vc8);
      next_page = page_of(t - TN + kSpan);
    }
  };
  auto fetch_k = [&](int t, int i, uint16_t* to) SC_INLINE {
    if constexpr (FP8) load_codes(a.kc8, pk, piece_at(t), i, t < t_hi, kr[i], ks[i]);
    else copy_chunk(a.kc, pk, piece_at(t), i, t < t_hi, true, to);
  };
  auto fetch_v = [&](int t, int i, uint16_t* to) SC_INLINE {
    if constexpr (FP8) load_codes(a.vc8, pv, piece_at(t), i, t < t_hi, vr[i], vs[i]);
    else copy_chunk(a.vc, pv, piece_at(t), i, t < t_hi, false, to);
  };
  // pieces there are: of the next keys, of those after them, of the next values
  uint32_t k_seen1 = seen_at(pk, t_lo + TN), k_seen2 = seen_at(pk, t_lo + 2 * TN), v_seen1 = k_seen1;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    fetch_k(t_lo, i, K0);
    fetch_v(t_lo, i, V0);
    if constexpr (FP8) {
      store_codes(K0, i, true, kr[i], ks[i]);
      store_codes(V0, i, false, vr[i], vs[i]);
    }
  }
  if (t_lo + TN < t_hi) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      fetch_k(t_lo + TN, i, K1);
      if constexpr (FP8) {
        store_codes(K1, i, true, kr[i], ks[i]);
        fetch_k(t_lo + 2 * TN, i, nullptr);
        fetch_v(t_lo + TN, i, nullptr);
      }
    }
  }
  if constexpr (!FP8) __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
  clear_v(V0, t_lo, seen_at(pk, t_lo));
  __syncthreads();
  if (busy) {
    scores(K0, S0);
    if (t_lo + TN > t_hi || seen_at(pk, t_lo) != kWhole) mask(t_lo, seen_at(pk, t_lo), S0);
    take_max(largest(S0));
  }
  __syncthreads();                                    // the first tile's keys have been read

  // Tile t: its scores are in `cur`, its values in V; the next one's keys in Kn. What
  // belongs to tiles behind the last one is done all the same, so that a turn has no
  // branches, but for their reads.
  // A wave without rows takes its share in the fetching alone.
  auto turn = [&](auto idle, int t, uint16_t* K, uint16_t* Kn, uint16_t* V, uint16_t* Vn, f32x16* cur,
                  f32x16* next) SC_INLINE {
    constexpr std::integral_constant<int, (FP8 ? 4 : 2) * CH> chores{};
    auto chore = [&](auto which) SC_INLINE {
      constexpr int i = which, j = i % CH;
      if constexpr (FP8 && i < CH) store_codes(Vn, j, false, vr[j], vs[j]);
      else if constexpr (FP8 && i < 2 * CH) store_codes(K, j, true, kr[j], ks[j]);
      else if constexpr (FP8 && i < 3 * CH) fetch_v(t + 2 * TN, j, nullptr);
      else if constexpr (FP8) fetch_k(t + 3 * TN, j, nullptr);
      else if constexpr (i < CH) fetch_v(t + TN, j, Vn);
      else fetch_k(t + 2 * TN, j, K);
    };
    const uint32_t v_seen2 = FP8 ? seen_at(pv, t + 2 * TN) : seen_at(pv, t + TN);
    const uint32_t k_seen3 = FP8 ? seen_at(pk, t + 3 * TN) : seen_at(pk, t + 2 * TN);
    if (!FP8) k_seen2 = k_seen3, v_seen1 = v_seen2;
    if constexpr (!idle) {
      float top = products(Kn, V, cur, next, chores, chore);
      if (t + TN < t_hi) {
        if (t + 2 * TN > t_hi || k_seen1 != kWhole) {
          mask(t + TN, k_seen1, next);
          top = largest(next);
        }
        take_max(top);
      }
    } else {
      steps<chores>(chore);
    }
    go_on(t + (FP8 ? 4 : 3) * TN);
    if constexpr (!FP8) __builtin_amdgcn_s_waitcnt(0x0f70);
    if (t + TN < t_hi) clear_v(Vn, t + TN, v_seen1);
    k_seen1 = k_seen2;
    k_seen2 = k_seen3;
    v_seen1 = v_seen2;
    __syncthreads();
  };
  auto turns = [&](auto idle) SC_INLINE {
    for (int t = t_lo;;) {
      turn(idle, t, K0, K1, V0, V1, S0, S1);
      if ((t += TN) >= t_hi) break;
      turn(idle, t, K1, K0, V1, V0, S1, S0);
      if ((t += TN) >= t_hi) break;
    }
  };
  if (!busy) {
    turns(std::true_type{});
    return;
  }
  turns(std::false_type{});

  l = (l + __shfl_xor(l, 32)) * kMore;
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

// Adds a query row's parts, those of the prefix and of its own tokens, where the latter
// are more than one or the former many. WPR waves of a workgroup per row take parts in
// turn, hd/64 values a lane, eight loads at a time that do not wait for the weights.
template <int HD, int WPR>
__global__ __launch_bounds__(kBlock) void attn_prefix_join(PagedAttnArgs a, int unit) {
  constexpr int N = HD / 64, PER = 4 / WPR, AT_ONCE = 8;
  constexpr int NP = (kMaxPrefixSplits + kMaxOwnSplits) / 64;
  typedef float row_t __attribute__((ext_vector_type(N)));
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
    // the i-th part there is
    auto number = [&](int i) { return i < n1 ? i : a.prefix_splits + i - n1; };
    row_t x[AT_ONCE];
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const int i = i0 + u * WPR;
        if (i < n1 + n2) x[u] = *(const row_t*)(part + (int64_t)number(i) * HD);
      }
    };
    load(w % WPR);
    float mi[NP], f[NP], mt = kNone;
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      const int i = u * 64 + lane;
      const bool in = i < n1 + n2;
      mi[u] = in ? ml[number(i) * 2] : kNone;
      f[u] = in ? ml[number(i) * 2 + 1] : 0.f;
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
    for (int i0 = w % WPR; i0 < n1 + n2; i0 += AT_ONCE * WPR) {
      if (i0 >= WPR) load(i0);
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const int i = i0 + u * WPR;
        if (i >= n1 + n2) break;
        float fi = __shfl(f[0], i & 63);
#pragma unroll
        for (int v = 1; v < NP; ++v) {
          const float z = __shfl(f[v], i & 63);
          fi = i >= v * 64 ? z : fi;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] = fmaf(x[u][e], fi, y[e]);
      }
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

namespace {

// About how long attn_prefix and the way of its parts take (us) with `splits` of the
// prefix and `waves` in a workgroup. Measured, 64 tokens x 128: a tile takes 0.9 us (0.6
// with 32 tokens, but of 256-wide heads) and 0.24 for each busy wave on its CU, widening
// codes 0.17 for each workgroup of fewer than eight waves there; a call 7 us to begin and
// end, a part 1 us for each 2 MB there and back, a join launch 4; the prefix comes at 5.5
// TB/s. What is taken (waves / splits) and others, us for the call with 16 own tokens or
// fewer; rows of each of 4 heads:
//   256 rows x 128 on 16,384      4 / 32  37   (8 / 32  44, 4 / 16  43, 4 / 64  39, 2 / 64  41)
//   1,024 on 4,096                4 / 8   37   (8 / 16  39, 4 / 16  39, 2 / 16  39)
//   2,048 on 32,768               8 / 8  203   (8 / 16 219, 4 / 8  209, 4 / 4  227)
//   1,024 on 16,384, quantised    8 / 16  73   (8 / 8  100, 4 / 16  77, 4 / 8   83)
//   32 on 1,024                   8 / 16  16   (8 / 8   15, 4 / 8   16, 2 / 8   16)
//   201 x 8 x 64 in ten groups    2 / 8   47   (4 / 16  56, 8 / 5   56, 2 / 16  52)
//   512 x 64 on 8,192             4 / 16  26   (8 / 16  31, 4 / 32  33, 2 / 16  31)
//   4,096 x 64 on 8,192           8 / 4   77   (8 / 8   84, 4 / 4   78, 4 / 8   81)
//   256 x 256 on 8,192            2 / 16  47   (4 / 16  51, 4 / 32  45, 2 / 32  46)
//   2,048 x 256 on 8,192          4 / 4  147   (4 / 8  166, 2 / 4  153, 2 / 8  168)
//   32 x 256 on 16,384            4 / 64  33   (4 / 32  43, 4 / 96  44, 2 / 96  34)
//   1,024 x 256, quantised        4 / 8   91   (4 / 16 111, 2 / 8  106, 4 / 4  148)
struct PrefixTime {
  PrefixTime(const PagedAttnArgs& a, int waves, int64_t rows, int64_t groups, bool fp8) {
    cus = device_cus();
    tn = tile_tokens(a.hd, waves);
    units = (a.max_prefix + tn - 1) / tn;
    const int64_t tiles = (rows - groups) / (waves * kWaveRows) + groups;
    each = tiles * a.nkv;
    slots = (a.hd == 256 ? 4 : 8) / waves * cus;
    base_us = tn == 64 || a.hd == 256 ? 0.9 : 0.6;
    // a workgroup's, of its busy waves
    more_us = 0.24 * tn * a.hd / 8192 * ((double)rows / kWaveRows + groups * 0.5) / tiles +
              (fp8 && waves < 8 ? 0.17 : 0);
    read_us = (double)groups * a.max_prefix * a.nkv * a.hd * (fp8 ? 2 : 4) / 5.5e6;
    part_us = (double)rows * a.nkv * a.hd * 4 / 2.2e6;
    uneven = groups > 1;
  }
  double of(int64_t splits) const {
    const int64_t total = each * splits;
    const int64_t at_once = std::min((total + cus - 1) / cus, slots / cus);
    // groups have prefixes of several lengths, so that rounds of their workgroups run together
    const double rounds = uneven ? std::max(1.0, (double)total / slots) : (double)((total + slots - 1) / slots);
    const int64_t turns = (units + splits - 1) / splits;
    return std::max(rounds * turns * (base_us + more_us * at_once), read_us) + splits * part_us + 7 +
           (splits > kMostTakenIn ? 4 : 0);
  }
  double base_us, more_us, read_us, part_us;
  int64_t cus, each, slots, tn, units;     // each: workgroups of a split
  bool uneven;
};

}  // namespace

int64_t plan_paged_attn_prefix(PagedAttnArgs* a, bool fp8) {
  const int64_t rows_each = (int64_t)(a->nq / a->nkv) * a->nq_tok;
  const int64_t rows = a->batch * rows_each;
  const int64_t groups = std::max<int64_t>(1, std::min(a->groups, a->batch));
  const int64_t cus = device_cus();
  // 256-wide heads leave registers for four waves
  int64_t best = 1;
  double best_us = -1;
  for (int waves = a->hd == 256 ? 4 : 8; waves >= 2; waves /= 2) {
    const PrefixTime time(*a, waves, rows, groups, fp8);
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(time.units, kMaxPrefixSplits));
    auto look = [&](int64_t n) {
      n = std::clamp<int64_t>(n, 1, most);
      const double us = time.of(n);
      if (best_us < 0 || us < best_us) a->waves = waves, best = n, best_us = us;
    };
    for (int64_t n : {1, 2, 4, 8, 16, 32, 64, 96}) look(n);
    look(time.cus / time.each);                         // as fill the chip once
    look(time.slots / time.each);
  }
  const int64_t m = (int64_t)a->waves * kWaveRows, tn = tile_tokens(a->hd, a->waves);
  const int64_t tiles = (rows - groups) / m + groups;   // the groups' last tiles may be part
  const int64_t units = (a->max_prefix + tn - 1) / tn;
  const int64_t per = std::max<int64_t>(1, (units + best - 1) / best);
  a->prefix_splits = (int32_t)((units + per - 1) / per);
  a->prefix_split_len = (int32_t)(per * tn);
  a->row_tiles = (int32_t)std::min<int64_t>(tiles, 0x7FFFFFFF);
  // Splits of the requests' own tokens: as in plan_paged_attn, for the length that is
  // left behind the longest prefix. A longer rest is cut into as many, longer, parts. Where
  // few rows leave so many parts of the prefix that a launch of its own joins them, a longer
  // rest would keep its workgroups alone on the card: there the split is for whole caches
  // of own tokens, up to four workgroups a CU, and those behind a short rest end at once. 8
  // requests on 32,768 tokens, 16 query and 4 key/value heads x 128, and 4 of 32,000 of no
  // group: 732 us without, 82 with (quantised 319 and 59; by sc_paged_attn_decode 110); the
  // 8 alone 31 us either way. With more rows the split would cost each batch a join, 64 x 4
  // drafts on 16,384 tokens 82 us for 86 and ten groups 58 for 63, long rest or not.
  // Quantised own tokens take the same rule: 4 requests of up to 8,192 behind 1,024, 8 splits
  // 25 us (16: 21), 16 of up to 4,096, 4 splits 29 us (8: 27), 64 of up to 2,000, 2 splits 42
  // (1: 44, 4: 43), 256 of them, 2 splits 91 (1: 88, 4: 92).
  const int64_t base = (int64_t)a->batch * a->nkv * ((rows_each + kRows - 1) / kRows);
  const bool every = a->prefix_splits > kMostTakenIn;
  const int64_t left = every ? a->max_len : a->max_len - a->max_prefix + kTile;
  const int64_t want = every ? 4 * cus : base >= 4 * cus ? 8 * cus : 16 * cus;
  a->splits = (int32_t)std::max<int64_t>(
      1, std::min<int64_t>({(want + base - 1) / base, (left + 1023) / 1024, kMaxOwnSplits}));
  // One split of them takes the prefix's parts in by itself, a wave a fourth of them.
  a->whole = a->splits == 1 && a->prefix_splits <= kMostTakenIn;
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
    else if constexpr (HD != 256) launch_prefix<HD, 8, FP8>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const hipError_t e = FP8 ? launch_paged_attn_after_fp8(a, s) : launch_paged_attn_after(a, s);
  if (e != hipSuccess || a.whole) return e;
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
