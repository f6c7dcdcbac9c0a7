// Gated delta rule, chunked form, for varlen prefill.
//
// Over a chunk of 64 tokens with G the running sum of the log decays, the
// recurrence S <- e^g S + u k^T, u = beta (v - e^g S k), o = scale S q becomes
//
//   (I + A) U = diag(beta) (V - diag(e^G) K S0^T)     A_ts = beta_t e^{G_t-G_s} k_t.k_s, s < t
//   O  = diag(scale e^G) Q S0^T + P U                 P_ts = scale e^{G_t-G_s} q_t.k_s, s <= t
//   S' = e^{G_C} S0 + U^T diag(e^{G_C-G}) K
//
// Only S0 ties a request's chunks together. gdn_chunk computes T = (I + A)^-1
// diag(beta) and P of every chunk at once; gdn_scan walks each request's chunks with the
// state, split over the value columns, which never mix.
//
// Precision: the state and every sum are fp32. Products run on bf16 MFMA with
// each fp32 factor cut into 16-bit parts (x = hi + mid + lo to 2^-24) and
// the small cross terms left out; q, k and v enter as they are, which is
// exact: the unit lengths of q and k are row factors applied in fp32. P, the
// copy of U it multiplies and the state as Q multiplies it carry two parts (they
// leave 2^-16): those products only reach the bf16 output, whose own rounding is
// 2^-8 of a value. The gates are fp32, their running sum in a chunk fp64.
#include "conv_device.hpp"
#include "gdn_device.hpp"

#include <climits>

namespace sc {

namespace {

constexpr int CH = kGdnChunk;

// Fragment index of (row tile w, k step ks) among the six at or below the
// diagonal of a 64 x 64 matrix: tiles of 16 rows, k steps of 32 columns.
__device__ __forceinline__ constexpr int frag_of(int w, int ks) {
  return w < 2 ? w : 2 + (w - 2) * 2 + ks;
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  f32x2 p = {x, y};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// N 16-bit parts of eight values as one operand: each part is the bf16 nearest
// to what the parts before it leave, which is exact in fp32. Plain subtractions:
// the two-term bf16 dot product would do with fewer instructions, but it does
// not run beside the matrix unit (a product and two dot products took 38 cycles
// here, a product and two fused multiply-adds 20, a product alone 17).
template <int N>
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, u32x4* part) {
  float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint32_t h[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) part[n][p] = h[p] = pack2(v[2 * p], v[2 * p + 1]);
    if (n + 1 < N) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        v[2 * p] -= lo_f(h[p]);
        v[2 * p + 1] -= hi_f(h[p]);
      }
    }
  }
}

// Range-checked buffer over the n rows (<= 64, of stride rs elements) from p:
// rows behind them read zeros and drop stores. The base is uniform, so a
// lane's offsets within a chunk stay the same from chunk to chunk. The check
// covers the lane's own (vector) offset; the scalar offset of the builtins is
// outside it by their contract, so a row's distance always goes into the former.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ rsrc_t row_rsrc(const uint16_t* p, int64_t rs, int n) {
  return make_rsrc(p, n * (int)rs * 2);
}

// Token rows of chunk `id`: request r, first row, rows (0: none).
struct Chunk {
  int r, row0, n;
};
__device__ __forceinline__ Chunk chunk_of(const GdnArgs& a, int id) {
  int s0 = 0, s1 = 0;
  Chunk c{0, 0, 0};
  c.r = find_request_bounds(a.qsl, a.batch, id, CH, s0, s1);
  if (c.r >= a.batch) return c;
  const int base = s0 / CH + c.r;
  const int first = s0 + (id - base) * CH;
  const int T = (int)a.num_tokens;
  c.row0 = min(max(first, 0), T);
  c.n = id < base ? 0 : min(max(min(s1, T) - c.row0, 0), CH);
  return c;
}

}  // namespace

// ---------------------------------------------------------------------------
// gdn_chunk: T and P of one (chunk, value head), four waves; bound by the
// latency of its steps, so that they are few and short, and four workgroups
// share a CU. Four chunks of 32 heads x 128: 10 us; 512: 0.20 ms (0.65 GB
// written to the workspace; 0.37 with row-wise products and LDS between all
// steps, 0.25 with two workgroups a CU).
//
// Wave w owns rows 16w..16w+15. The products are taken transposed, K_j K_w^T
// and K_j Q_w^T (16x16x32 bf16): a lane then holds one row t and four adjacent
// columns s, which is how the scan's operands are laid out, so P goes to the
// workspace from registers, and A to LDS in 16-byte rows. The unit lower
// triangular inverse goes by blocks: the four 16 x 16 diagonal blocks by forward
// substitution, a lane per column of each, with the row's elements broadcast
// over 16 lanes; then T_ij = -T_ii (A_ij T_jj) at 16 and at 32 on fp32 MFMA, the
// inner product staying in registers (an accumulator tile is a right operand of
// 16x16x4 products whose step i sums over rows 4 g + i).
// The first value head of a key head also writes the keys transposed, as the
// scan's state update multiplies by them.
// ---------------------------------------------------------------------------

// Lane n of each 16, in all of them.
template <int N>
__device__ __forceinline__ float row16_bcast(float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + N, 0xF, 0xF, true));
}
// x_i = (i == column) + sum_{j<i} row_i[j] x_j, for rows held across 16 lanes.
template <int I, int J>
__device__ __forceinline__ float substitute(const float (&row)[16], const float (&x)[16], float s) {
  if constexpr (J < I) return substitute<I, J + 1>(row, x, fmaf(row16_bcast<J>(row[I]), x[J], s));
  else return s;
}
template <int I>
__device__ __forceinline__ void substitute_rows(const float (&row)[16], float (&x)[16], int col) {
  if constexpr (I < 16) {
    x[I] = substitute<I, 0>(row, x, I == col ? 1.f : 0.f);
    substitute_rows<I + 1>(row, x, col);
  }
}

// x plus what another lane holds (DPP control), in the rows of the mask.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_lane(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return x + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sum of this lane's value and all before it.
__device__ __forceinline__ double wave_running_sum(double x) {
  x = add_lane<0x111, 0xF>(x);      // 1, 2, 4 and 8 lanes before, within 16
  x = add_lane<0x112, 0xF>(x);
  x = add_lane<0x114, 0xF>(x);
  x = add_lane<0x118, 0xF>(x);
  x = add_lane<0x142, 0xA>(x);      // lane 15 of the 16 before
  return add_lane<0x143, 0xC>(x);   // lane 31
}

// Requests by falling length into the workspace, by a workgroup: a scan takes as
// long as its chunks, so where workgroups wait for a CU the longest go first
// (100 requests of 60 tokens with one of 6,000 behind them, 32 heads x 128: 0.62
// ms as they come, 0.45 so; 8 ragged ones 5 to 13% faster). It runs beside the
// chunks' workgroups, in a few microseconds for 1,024 requests; of more, one
// request is a small part of the whole.
constexpr int kSortMax = 1024;
__device__ __forceinline__ void order_requests(const GdnArgs& a, int* n) {
  const int tid = (int)threadIdx.x;
  const int padded = (a.batch + 3) & ~3;
  for (int r = tid; r < padded; r += kBlock)
    n[r] = r < a.batch ? a.qsl[r + 1] - a.qsl[r] : INT_MIN;
  __syncthreads();
  int* const order = (int*)(a.ws + GdnWorkspace::order(a.n_chunks, a.hk, a.hv, a.dk));
  for (int r = tid; r < a.batch; r += kBlock) {
    const int mine = n[r];
    int rank = 0;
    for (int m = 0; m < padded; m += 4) {
      const int4 o = *(const int4*)(n + m);
      rank += (o.x > mine || (o.x == mine && m < r)) + (o.y > mine || (o.y == mine && m + 1 < r)) +
              (o.z > mine || (o.z == mine && m + 2 < r)) + (o.w > mine || (o.w == mine && m + 3 < r));
    }
    order[rank] = r;
  }
}

template <int DK>
__global__ __launch_bounds__(kBlock, 4) void gdn_chunk(GdnArgs a) {
  constexpr int KS = DK / 32;
  constexpr int LD = 68;                      // fp32 row stride of the LDS matrices
  constexpr int LK = DK + 8;                  // row stride of the keys
  // the keys are read before T is written
  constexpr int kKeyBytes = CH * LK * 2, kMatBytes = CH * LD * 4;
  __shared__ __align__(16) char kt_mem[kKeyBytes > kMatBytes ? kKeyBytes : kMatBytes];
  __shared__ __align__(16) float Am[CH * LD];
  __shared__ __align__(16) double Gs[CH];
  __shared__ __align__(16) float beta_s[CH], rk_s[CH], rq_s[CH];
  uint16_t* const Kl = (uint16_t*)kt_mem;
  float* const Tm = (float*)kt_mem;

  unsigned block = blockIdx.x;
  if (a.sorted && block-- == 0) {
    static_assert(sizeof(Am) >= kSortMax * sizeof(int));
    order_requests(a, (int*)Am);
    return;
  }
  const int h = (int)(block % (unsigned)a.hv);
  const int id = (int)(block / (unsigned)a.hv);
  const Chunk c = chunk_of(a, id);
  if (c.n == 0) return;
  const int rep = a.hv / a.hk, hk = h / rep;
  const int lane = (int)(threadIdx.x & 63);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l16 = lane & 15, lg = lane >> 4;
  const bool put_kt = h == hk * rep;

  // rows as MFMA operands: lane holds row l16 of a tile, 8 values from 8 lg
  u32x4 kw[KS], qw[KS];
  const int my_row = w * 16 + l16;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    kw[ks] = qw[ks] = u32x4{0, 0, 0, 0};
    if (my_row < c.n) {
      const int64_t row = c.row0 + my_row;
      kw[ks] = ld16((const uint16_t*)a.k + row * a.k_rs + hk * DK + ks * 32 + lg * 8);
      qw[ks] = ld16((const uint16_t*)a.q + row * a.q_rs + hk * DK + ks * 32 + lg * 8);
    }
  }
  // gates: wave 0, a lane per token; the running sum in fp64 (of base 2
  // exponents), so that the difference of two of a chunk's sums keeps fp32
  // accuracy whatever came before. A decay below e^-110 is zero in fp32 already.
  if (w == 0) {
    float g = 0.f, be = 0.f;
    if (lane < c.n) {
      g = gdn_log_decay(a, c.row0 + lane, h);
      g = g < -110.f ? -110.f : g;
      be = gdn_beta(a, c.row0 + lane, h);
    }
    Gs[lane] = wave_running_sum((double)g * 1.4426950408889634);
    beta_s[lane] = be;
  }
  // unit lengths; keys to LDS
  {
    float kk = 0.f, qq = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      *(u32x4*)(Kl + my_row * LK + ks * 32 + lg * 8) = kw[ks];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kk = fmaf(lo_f(kw[ks][e]), lo_f(kw[ks][e]), kk);
        kk = fmaf(hi_f(kw[ks][e]), hi_f(kw[ks][e]), kk);
        qq = fmaf(lo_f(qw[ks][e]), lo_f(qw[ks][e]), qq);
        qq = fmaf(hi_f(qw[ks][e]), hi_f(qw[ks][e]), qq);
      }
    }
    kk += __shfl_xor(kk, 16);
    kk += __shfl_xor(kk, 32);
    qq += __shfl_xor(qq, 16);
    qq += __shfl_xor(qq, 32);
    if (lg == 0) {
      rk_s[my_row] = a.l2norm ? rsqrtf(kk + kL2Eps) : 1.f;
      rq_s[my_row] = a.scale * (a.l2norm ? rsqrtf(qq + kL2Eps) : 1.f);
    }
  }
  __syncthreads();

  char* const ws = a.ws + ((int64_t)id * a.hv + h) * GdnWorkspace::kHead;
  // raw products and their factors, column tiles j <= w
  f32x4 P[4];
  {
    const double gt = Gs[my_row];
    const float rq = rq_s[my_row], bk = beta_s[my_row] * rk_s[my_row];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      P[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (j > w) continue;
      f32x4 kk = P[j], qk = P[j];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const u32x4 kj = *(const u32x4*)(Kl + (j * 16 + l16) * LK + ks * 32 + lg * 8);
        kk = mfma_bf16(kj, kw[ks], kk);
        qk = mfma_bf16(kj, qw[ks], qk);
      }
      const f32x4 rk = *(const f32x4*)(rk_s + j * 16 + lg * 4);
      f32x4 A;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = j * 16 + lg * 4 + i;
        const float d = __builtin_amdgcn_exp2f((float)(gt - Gs[s])) * rk[i];
        A[i] = s < my_row ? bk * d * kk[i] : 0.f;
        P[j][i] = s <= my_row ? rq * d * qk[i] : 0.f;
      }
      *(f32x4*)(Am + my_row * LD + j * 16 + lg * 4) = A;
    }
  }
  // row factors of the scan
  if (w == 0) {
    float* vec = (float*)(ws + GdnWorkspace::kT + GdnWorkspace::kP);
    const float eg = __builtin_amdgcn_exp2f((float)Gs[lane]), rk = rk_s[lane];
    vec[lane] = eg * rk;                                                             // of S k
    vec[CH + lane] = rk * __builtin_amdgcn_exp2f((float)(Gs[CH - 1] - Gs[lane]));    // of U in the update
    vec[2 * CH + lane] = rq_s[lane] * eg;                                            // of S q
    if (lane == 0) vec[3 * CH] = __builtin_amdgcn_exp2f((float)Gs[CH - 1]);          // of S
  }
  if (put_kt) {
    // keys transposed, in the scan's orders of key dims (row l16 of state tile
    // m) and of tokens
    char* kt = a.ws + (int64_t)a.n_chunks * a.hv * GdnWorkspace::kHead +
               ((int64_t)id * a.hk + hk) * (DK * CH * 2);
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) {
      const int f = w * (DK / 32) + i;        // fragment (tile m, k step ks)
      const int m = f >> 1, ks = f & 1;
      const int dim = (m >> 1) * 32 + (l16 >> 2) * 8 + (m & 1) * 4 + (l16 & 3);
      const uint16_t* p = Kl + (ks * 32 + lg * 4) * LK + dim;
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint16_t* t = p + ((e >> 1) * 16 + (e & 1) * 2) * LK;
        v[e] = (uint32_t)t[0] | ((uint32_t)t[LK] << 16);
      }
      *(u32x4*)(kt + f * GdnWorkspace::kFrag + lane * 16) = v;
    }
  }
  __syncthreads();                            // A is there, and the keys are done with
  // diagonal blocks of T by substitution (wave 0; lane: column l16 of block
  // lg); the others write P meanwhile
  if (w == 0) {
    float row[16], x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) row[i] = -Am[(lg * 16 + i) * LD + lg * 16 + l16];
    substitute_rows<0>(row, x, l16);
#pragma unroll
    for (int i = 0; i < 16; ++i) Tm[(lg * 16 + i) * LD + lg * 16 + l16] = x[i];
  }
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    if (ks == 1 && w < 2) continue;
    u32x4 part[2];
    split8<2>(P[2 * ks], P[2 * ks + 1], part);
#pragma unroll
    for (int n = 0; n < 2; ++n)
      *(u32x4*)(ws + GdnWorkspace::kT + (frag_of(w, ks) * 2 + n) * GdnWorkspace::kFrag + lane * 16) =
          part[n];
  }
  // blocks (0, 1) and (2, 3) of T, which the operands of 32 columns take in
  if (w == 1 || w == 2) {
    const int r0 = (w - 1) * 32 + l16, c0 = (w - 1) * 32 + 16 + lg * 4;
    *(f32x4*)(Tm + r0 * LD + c0) = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();
  // X(rx, cx) Y + acc for a block X in LDS and an accumulator tile Y
  auto mul_reg = [&](const float* X, int rx, int cx, f32x4 y, f32x4 acc) {
    const f32x4 x = *(const f32x4*)(X + (rx * 16 + l16) * LD + cx * 16 + lg * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = mfma_f32(x[i], y[i], acc);
    return acc;
  };
  auto get16 = [&](const float* X, int r, int col) {
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = X[(r * 16 + lg * 4 + i) * LD + col * 16 + l16];
    return y;
  };
  auto put_neg16 = [&](float* X, int r, int col, f32x4 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) X[(r * 16 + lg * 4 + i) * LD + col * 16 + l16] = -v[i];
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  // blocks (1,0) and (3,2)
  if (w < 2) {
    const int b = 2 * w;
    const f32x4 y = mul_reg(Am, b + 1, b, get16(Tm, b, b), zero);
    put_neg16(Tm, b + 1, b, mul_reg(Tm, b + 1, b + 1, y, zero));
  }
  __syncthreads();
  // the 32 x 32 block below: a wave per 16 x 16 tile (i, j)
  {
    const int i = 2 + (w >> 1), j = w & 1;
    const f32x4 t1 = get16(Tm, 1, j);
    f32x4 t0 = zero;                           // block (0, 1) is zero
    if (j == 0) t0 = get16(Tm, 0, 0);
    f32x4 y2 = mul_reg(Am, 2, 1, t1, zero);
    if (j == 0) y2 = mul_reg(Am, 2, 0, t0, y2);
    f32x4 z = mul_reg(Tm, i, 2, y2, zero);
    if (i == 3) {
      f32x4 y3 = mul_reg(Am, 3, 1, t1, zero);
      if (j == 0) y3 = mul_reg(Am, 3, 0, t0, y3);
      z = mul_reg(Tm, 3, 3, y3, z);
    }
    put_neg16(Tm, i, j, z);
  }
  __syncthreads();
  // T diag(beta) as operand fragments, in the scan's order of tokens: three
  // parts of 4 adjacent values from column 32 ks + 4 lg and 4 from 16 further on
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    if (ks == 1 && w < 2) continue;
    const int c0 = ks * 32 + lg * 4;
    f32x4 x = *(const f32x4*)(Tm + my_row * LD + c0), y = *(const f32x4*)(Tm + my_row * LD + c0 + 16);
    const f32x4 bx = *(const f32x4*)(beta_s + c0), by = *(const f32x4*)(beta_s + c0 + 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] *= bx[e];
      y[e] *= by[e];
    }
    u32x4 part[3];
    split8<3>(x, y, part);
#pragma unroll
    for (int n = 0; n < 3; ++n)
      *(u32x4*)(ws + (frag_of(w, ks) * 3 + n) * GdnWorkspace::kFrag + lane * 16) = part[n];
  }
}

// ---------------------------------------------------------------------------
// gdn_scan: one request's chunks in turn for one value head; each wave has 16
// value columns of the state and never needs another wave's.
//
// The state of a wave is held as S^T (DK x 16) in MFMA accumulators. An
// accumulator tile has column lane % 16 and rows 4 (lane / 16) + i in register
// i; the right operand of a 16x16x32 product has column lane % 16 and eight
// values of its inner index per lane. So two accumulator tiles, cut into bf16
// parts, are a right operand as they stand, if the inner index is counted in
// the order in which they hold it; the left operands are laid out in that
// order (gdn_chunk does it for T, P and the transposed keys; for rows of q
// and k it is a choice of which key dim is which state row). State, right-hand
// sides and U go from product to product in registers, without LDS or a
// barrier between.
//
// LDS holds the left operands of a chunk, which the waves share, and its
// values. NL more waves do nothing but load them, straight into LDS: the
// address unit takes about 32 bytes a clock, so that a wave that computed and
// loaded stood still for most of the time. K, Q, T and the values, used first,
// are loaded a chunk ahead into the other of two buffers; P and the transposed
// keys while the first half of their own chunk is computed. Two barriers a
// chunk. The outputs are taken with the operands exchanged, which gives a lane
// four adjacent values of a row to store. A chunk takes about 3 us, products
// and the cutting of their operands, so that a call takes as long as its
// longest request: eight requests of 8,196 tokens in all, 32 heads x 128, 0.16
// to 0.20 ms by the spread of their lengths.
// ---------------------------------------------------------------------------
template <int DK, int NW>
struct ScanBuf {
  static constexpr int kF = GdnWorkspace::kFrag;
  static constexpr int kKey = DK * CH * 2;
  // first half of a chunk
  static constexpr int kT = 0, kVec = GdnWorkspace::kT;      // as in the workspace
  static constexpr int kK = kVec + GdnWorkspace::kVec, kQ = kK + kKey, kV = kQ + kKey;
  static constexpr int kFirst = kV + CH * NW * 32;
  // second half
  static constexpr int kP = 0, kKt = GdnWorkspace::kP, kSecond = kKt + kKey;
};

typedef const __attribute__((address_space(1))) void* gptr;
typedef __attribute__((address_space(3))) void* lptr;

// What a workgroup of a scan does: value head h of request r, slice `slice` of
// its columns. Workgroups are dealt to the XCDs in turn, so those of one key
// head, which read the same rows at about the same time, are placed eight
// apart: one L2 then fetches them once.
struct ScanWork {
  int r, h, slice, row_lo, rows, base, nch;
};
__device__ __forceinline__ ScanWork scan_work(const GdnArgs& a, int slices) {
  ScanWork k{};
  const int rep = a.hv / a.hk;
  const unsigned per_group = (unsigned)(rep * slices);
  const unsigned yb = blockIdx.x / kXcds;
  const unsigned group = yb / per_group * kXcds + blockIdx.x % kXcds;   // (request, key head)
  if (group >= (unsigned)a.batch * (unsigned)a.hk) return k;
  const unsigned in_group = yb % per_group;
  k.slice = (int)(in_group % (unsigned)slices);
  k.h = (int)(group % (unsigned)a.hk) * rep + (int)(in_group / (unsigned)slices);
  k.r = (int)(group / (unsigned)a.hk);
  if (a.sorted)
    k.r = __builtin_amdgcn_readfirstlane(
        ((const int*)(a.ws + GdnWorkspace::order(a.n_chunks, a.hk, a.hv, a.dk)))[k.r]);
  const int T = (int)a.num_tokens;
  const int s0 = __builtin_amdgcn_readfirstlane(a.qsl[k.r]);
  const int s1 = __builtin_amdgcn_readfirstlane(a.qsl[k.r + 1]);
  k.row_lo = min(max(s0, 0), T);
  k.rows = min(max(s1, k.row_lo), T) - k.row_lo;
  k.base = max(s0, 0) / CH + k.r;
  k.nch = min((k.rows + CH - 1) / CH, a.n_chunks - k.base);
  return k;
}

// slices = ceil(dv / (16 NW)) workgroups of NW + NL waves per (request, value
// head).
template <int DK, int NW, int NL>
__global__ __launch_bounds__(64 * (NW + NL)) void gdn_scan(GdnArgs a, int slices) {
  using B = ScanBuf<DK, NW>;
  constexpr int KS = DK / 32;
  __shared__ __align__(16) char first[2][B::kFirst];
  __shared__ __align__(16) char second[B::kSecond];
  const ScanWork wk = scan_work(a, slices);
  const int r = wk.r, h = wk.h, slice = wk.slice, row_lo = wk.row_lo, rows = wk.rows;
  const int base = wk.base, nch = wk.nch, hk = h / (a.hv / a.hk);
  if (nch <= 0) return;                       // no tokens: the slot stays as it is
  const int lane = (int)(threadIdx.x & 63), l16 = lane & 15, lg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const char* const wsb = a.ws + ((int64_t)base * a.hv + h) * GdnWorkspace::kHead;
  const char* const ktb = a.ws + (int64_t)a.n_chunks * a.hv * GdnWorkspace::kHead +
                          ((int64_t)base * a.hk + hk) * B::kKey;

  if (w >= NW) {
    const int ld = w - NW;                 // this loader's share: every NL-th fragment
    // Rows behind the request's end are read as its last one: the matrices
    // have zeros for them, and what they give is not stored.
    auto put = [&](const void* src, char* dst) {
      __builtin_amdgcn_global_load_lds((gptr)src, (lptr)dst, 16, 0, 0);
    };
    auto put_run = [&](const char* src, char* dst, int bytes) {
#pragma unroll
      for (int f = 0; f < bytes; f += NL * B::kF)
        if (f + NL * B::kF <= bytes || f + ld * B::kF < bytes)
          put(src + f + ld * B::kF + lane * 16, dst + f + ld * B::kF);
    };
    const uint16_t* const kb = (const uint16_t*)a.k + row_lo * a.k_rs + hk * DK + lg * 8;
    const uint16_t* const qb = (const uint16_t*)a.q + row_lo * a.q_rs + hk * DK + lg * 8;
    // values: 2 NW runs of 8 columns a row; the runs of a row are turned by 2
    // for each 4 rows, so that the 4 rows x 32 bytes of a read are in different
    // banks
    constexpr int VR = 2 * NW;
    const int vt = lane / VR, vrun = lane % VR;
    const uint16_t* const vb = (const uint16_t*)a.v + row_lo * a.v_rs + h * a.dv;
    auto load_rows = [&](int c) {
      char* const dst = first[c & 1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t row = min(c * CH + j * 16 + l16, rows - 1);
#pragma unroll
        for (int k0 = 0; k0 < KS; k0 += NL) {
          const int ks = k0 + ld;
          if (KS % NL != 0 && ks >= KS) continue;
          put(kb + row * a.k_rs + ks * 32, dst + B::kK + (j * KS + ks) * B::kF);
          put(qb + row * a.q_rs + ks * 32, dst + B::kQ + (j * KS + ks) * B::kF);
        }
      }
    };
    auto load_rest = [&](int c) {
      char* const dst = first[c & 1];
      const char* const ws = wsb + (int64_t)c * a.hv * GdnWorkspace::kHead;
      put_run(ws + GdnWorkspace::kT + GdnWorkspace::kP, dst + B::kVec, GdnWorkspace::kVec);
#pragma unroll
      for (int tb = 0; tb < CH; tb += NL * (64 / VR)) {
        const int t0 = tb + ld * (64 / VR), t = t0 + vt;
        const int run = (vrun - 2 * ((t >> 2) & 3)) & (VR - 1);
        const int col = min((slice * NW) * 16 + run * 8, a.dv - 8);   // behind the last: unused
        put(vb + (int64_t)min(c * CH + t, rows - 1) * a.v_rs + col, dst + B::kV + t0 * NW * 32);
      }
      put_run(ws, dst + B::kT, GdnWorkspace::kT);
    };
    load_rows(0);
    load_rest(0);
    for (int c = 0; c < nch; ++c) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();                     // first half of c is there; the second buffer is free
      const char* const ws = wsb + (int64_t)c * a.hv * GdnWorkspace::kHead;
      put_run(ktb + (int64_t)c * a.hk * B::kKey, second + B::kKt, B::kKey);
      put_run(ws + GdnWorkspace::kT, second + B::kP, GdnWorkspace::kP);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();                     // second half of c is there
      if (c + 1 < nch) {
        load_rows(c + 1);
        load_rest(c + 1);
      }
    }
    return;
  }

  const int col0 = (slice * NW + w) * 16;
  const bool work = col0 < a.dv;              // a wave behind the last column only waits
  const int32_t slot = a.slots[(int64_t)r * a.slot_stride];
  const bool in_pool = slot >= 0 && slot < a.num_slots;
  // state tile m, register i: key dim 32 (m / 2) + 8 lg + 4 (m % 2) + i
  float* const pool = a.pool + ((int64_t)slot * a.hv + h) * ((int64_t)a.dv * DK) +
                      (int64_t)(col0 + l16) * DK + lg * 8;
  f32x4 S[2 * KS];
  const bool cont = work && in_pool && a.has_init[r];
#pragma unroll
  for (int m = 0; m < 2 * KS; ++m) {
    S[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (cont) S[m] = *(const f32x4*)(pool + (m >> 1) * 32 + (m & 1) * 4);
  }
  // this lane's values: rows 4 lg + i, column l16 of the wave's
  const int v_at = B::kV + lg * 4 * (NW * 32) +
                   ((w * 2 + (l16 >> 3) + 2 * lg) & (2 * NW - 1)) * 16 + (l16 & 7) * 2;

  for (int c = 0; c < nch; ++c) {
    __syncthreads();
    if (!work) {
      __syncthreads();
      continue;
    }
    const char* const ops = first[c & 1];
    auto frag = [&](int off, int f) { return *(const u32x4*)(ops + off + f * B::kF + lane * 16); };
    auto frag2 = [&](int off, int f) { return *(const u32x4*)(second + off + f * B::kF + lane * 16); };
    const float* const vec = (const float*)(ops + B::kVec);
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // Left operands are read from LDS a step ahead of their products, and the
    // next step's right operand is cut between this one's products.
    // K S and (Q S)^T
    f32x4 Z[4], O[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) Z[j] = O[j] = zero;
    u32x4 kf[2][4], qf[2][4], s[2][3];
    auto read_kq = [&](int ks) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        kf[ks & 1][j] = frag(B::kK, j * KS + ks);
        qf[ks & 1][j] = frag(B::kQ, j * KS + ks);
      }
    };
    u32x4 t[6][3];
    f32x4 cr[4];
    uint16_t v[4][4];
    read_kq(0);
    split8<3>(S[0], S[1], s[0]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int b = ks & 1;
      if (ks + 1 < KS) {
        read_kq(ks + 1);
        split8<3>(S[2 * ks + 2], S[2 * ks + 3], s[b ^ 1]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cr[j] = *(const f32x4*)(vec + j * 16 + lg * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[j][i] = *(const uint16_t*)(ops + v_at + (j * 16 + i) * (NW * 32));
        }
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int e = 0; e < 3; ++e) t[f][e] = frag(B::kT, f * 3 + e);
      }
#pragma unroll
      for (int e = 2; e >= 0; --e)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          Z[j] = mfma_bf16(kf[b][j], s[b][e], Z[j]);
          if (e < 2) O[j] = mfma_bf16(s[b][e], qf[b][j], O[j]);
        }
      if (ks + 1 < KS) {
#pragma unroll
        for (int i = 0; i < 20; ++i) {
          if (i < 8) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // right-hand sides v - e^G S k, as operands of 32 tokens
    u32x4 R[2][3];
    auto rhs = [&](int g) {
      f32x4 x[2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[m][i] = fmaf(-cr[2 * g + m][i], Z[2 * g + m][i], lo_f(v[2 * g + m][i]));
      split8<3>(x[0], x[1], R[g]);
    };
    rhs(0);
    __builtin_amdgcn_sched_barrier(0);
    // U = T R. Row tiles 0 and 1 end with the first 32 tokens.
    f32x4 U[4];
    auto mul_t = [&](f32x4 u, const u32x4* tf, const u32x4* rr) {
      u = mfma_bf16(tf[2], rr[0], u);
      u = mfma_bf16(tf[0], rr[2], u);
      u = mfma_bf16(tf[1], rr[1], u);
      u = mfma_bf16(tf[1], rr[0], u);
      u = mfma_bf16(tf[0], rr[1], u);
      return mfma_bf16(tf[0], rr[0], u);
    };
#pragma unroll
    for (int f = 2; f < 6; ++f)
#pragma unroll
      for (int e = 0; e < 3; ++e) t[f][e] = frag(B::kT, f * 3 + e);
    f32x4 cu[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) cu[j] = *(const f32x4*)(vec + CH + j * 16 + lg * 4);
    U[0] = mul_t(zero, t[0], R[0]);
    U[1] = mul_t(zero, t[1], R[0]);
    rhs(1);
    U[2] = mul_t(zero, t[2], R[0]);
    U[3] = mul_t(zero, t[4], R[0]);
#pragma unroll
    for (int i = 0; i < 24; ++i) {
      if (i < 16) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    // U cut for P U (two parts) and, scaled, for the state (three)
    u32x4 Uf[2][2], X[2][3];
    auto cut_u = [&](int g) {
      f32x4 x[2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[m][i] = U[2 * g + m][i] * cu[2 * g + m][i];
      split8<3>(x[0], x[1], X[g]);
      split8<2>(U[2 * g], U[2 * g + 1], Uf[g]);
    };
    u32x4 kt[2 * KS][2], pf[6][2];
    __syncthreads();                       // P and the transposed keys are there
    const float decay = vec[GdnWorkspace::kDecay / 4];
    float co[4];
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m) kt[m][0] = frag2(B::kKt, m * 2);
    U[2] = mul_t(U[2], t[3], R[1]);
    U[3] = mul_t(U[3], t[5], R[1]);
    cut_u(0);
#pragma unroll
    for (int i = 0; i < 12; ++i) {
      if (i < 2 * KS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    // the state, by the first 32 tokens and then by the others
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m) kt[m][1] = frag2(B::kKt, m * 2 + 1);
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int e = 0; e < 2; ++e) pf[f][e] = frag2(B::kP, f * 2 + e);
#pragma unroll
    for (int j = 0; j < 4; ++j) co[j] = vec[2 * CH + j * 16 + l16];
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) S[m][i] *= decay;
#pragma unroll
      for (int e = 2; e >= 0; --e) S[m] = mfma_bf16(kt[m][0], X[0][e], S[m]);
    }
    cut_u(1);
#pragma unroll
    for (int i = 0; i < 6 * KS; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
      if (i < 2 * KS + 8) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 2; f < 6; ++f)
#pragma unroll
      for (int e = 0; e < 2; ++e) pf[f][e] = frag2(B::kP, f * 2 + e);
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
#pragma unroll
      for (int e = 2; e >= 0; --e) S[m] = mfma_bf16(kt[m][1], X[1][e], S[m]);
    // the outputs
    const rsrc_t orr = row_rsrc((uint16_t*)a.out + (row_lo + (int64_t)c * CH) * a.out_rs +
                                    h * a.dv + col0, a.out_rs, min(rows - c * CH, CH));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) O[j][i] *= co[j];
#pragma unroll
      for (int ks = 0; ks < (j < 2 ? 1 : 2); ++ks) {
        const u32x4* p = pf[frag_of(j, ks)];
        O[j] = mfma_bf16(Uf[ks][0], p[1], O[j]);
        O[j] = mfma_bf16(Uf[ks][1], p[0], O[j]);
        O[j] = mfma_bf16(Uf[ks][0], p[0], O[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_raw_buffer_store_b64(
          u32x2{pack2(O[j][0], O[j][1]), pack2(O[j][2], O[j][3])}, orr,
          (j * 16 + l16) * (uint32_t)a.out_rs * 2 + lg * 8, 0, 0);
  }
  if (in_pool && work) {
#pragma unroll
    for (int m = 0; m < 2 * KS; ++m)
      *(f32x4*)(pool + (m >> 1) * 32 + (m & 1) * 4) = S[m];
  }
}

// ---------------------------------------------------------------------------
// gdn_scan_few: the same scan for few (request, head, 16 columns), which would
// leave most of the chip idle: four waves share 16 value columns, so that the
// chain of a chunk (state -> K S -> right-hand sides -> U -> state), which is
// all that matters then, is a quarter as long.
//
// Each wave holds DK/4 key dims of the state, multiplies all 64 rows by them,
// and the four partial products meet in LDS in fp32; then each wave has 16 rows
// of the right-hand sides and of U. Three barriers a chunk: partial products
// written, right-hand sides written, U written. Left operands are used by one
// wave each and go straight to registers, a chunk ahead into the other of two
// sets, in three groups and the first of them between products: all at once
// they fill the address queue, and the wave stands still behind it (one
// request of 32,768 tokens: 1.95 ms all at once, 1.19 in groups, 1.10 so). It
// is still bound by that queue (78 KB a chunk and CU at about 32 bytes a clock)
// and by the chain; without its loads it takes 0.73 ms.
// ---------------------------------------------------------------------------
template <int DK>
struct KeyFrag;            // DK/4 key dims of a row: a lane's part of a left operand
template <>
struct KeyFrag<128> {
  u32x4 x;
  __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
    x = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
  }
};
template <>
struct KeyFrag<64> {
  u32x2 x;
  __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
    x = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
  }
};
__device__ __forceinline__ f32x4 mfma_key(const KeyFrag<128>& a, const KeyFrag<128>& b, f32x4 c) {
  return mfma_bf16(a.x, b.x, c);
}
__device__ __forceinline__ f32x4 mfma_key(const KeyFrag<64>& a, const KeyFrag<64>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a.x),
                                                   __builtin_bit_cast(s16x4, b.x), c, 0, 0, 0);
}

struct FewLds {
  static constexpr int LT = CH + 8;                // row stride (elements): banks differ by row
  f32x4 Z[4][4][64];                               // partial K S: of wave, row tile
  f32x4 O[4][4][64];                               // partial Q S
  __align__(16) uint16_t R[3][16 * LT];            // right-hand sides
  __align__(16) uint16_t U[2][16 * LT];            // U, as P multiplies it
  __align__(16) uint16_t X[3][16 * LT];            // U scaled for the state update
};

// The chunks of one request, for a wave whose rows of T and P reach NK k steps
// (waves 0 and 1: 1, waves 2 and 3: 2).
template <int DK, int NK>
struct FewOps {
  KeyFrag<DK> k[4], q[4];      // the wave's key dims of every row tile
  u32x4 t[NK][3], p[NK][2];    // T and P of row tile w
  u32x4 kt[DK / 64][2];        // transposed keys of the wave's state tiles
  uint16_t v[4];
  f32x4 c_rhs, c_upd;
  float c_out, decay;
};

template <int DK, int NK>
__device__ __forceinline__ void scan_few(const GdnArgs& a, FewLds& lds, int r, int h, int col0,
                                         int row_lo, int rows, int base, int nch, int w, int lane) {
  constexpr int MT = DK / 64, LT = FewLds::LT, kKey = DK * CH * 2, kF = GdnWorkspace::kFrag;
  constexpr int kVec = GdnWorkspace::kT + GdnWorkspace::kP;
  const int l16 = lane & 15, lg = lane >> 4;
  const int hk = h / (a.hv / a.hk);
  const int32_t slot = a.slots[(int64_t)r * a.slot_stride];
  const bool in_pool = slot >= 0 && slot < a.num_slots;
  const bool cont = in_pool && a.has_init[r];
  // register i of state tile m: key dim kd0 + 4 m + i
  const int kd0 = DK == 128 ? w * 32 + lg * 8 : (w >> 1) * 32 + lg * 8 + (w & 1) * 4;
  float* const pool = a.pool + ((int64_t)slot * a.hv + h) * ((int64_t)a.dv * DK) +
                      (int64_t)(col0 + l16) * DK + kd0;
  f32x4 S[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    S[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (cont) S[m] = *(const f32x4*)(pool + m * 4);
  }

  using Ops = FewOps<DK, NK>;
  const uint16_t* const qb = (const uint16_t*)a.q + row_lo * a.q_rs + hk * DK;
  const uint16_t* const kb = (const uint16_t*)a.k + row_lo * a.k_rs + hk * DK;
  const uint16_t* const vb = (const uint16_t*)a.v + row_lo * a.v_rs + h * a.dv + col0;
  uint16_t* const ob = (uint16_t*)a.out + row_lo * a.out_rs + h * a.dv + col0;
  const char* const wsb = a.ws + ((int64_t)base * a.hv + h) * GdnWorkspace::kHead;
  const char* const ktb = a.ws + (int64_t)a.n_chunks * a.hv * GdnWorkspace::kHead +
                          ((int64_t)base * a.hk + hk) * kKey;
  const uint32_t qrs = (uint32_t)a.q_rs * 2, krs = (uint32_t)a.k_rs * 2, vrs = (uint32_t)a.v_rs * 2;
  const uint32_t q_off = l16 * qrs + kd0 * 2, k_off = l16 * krs + kd0 * 2;
  const uint32_t v_off = (w * 16 + lg * 4) * vrs + l16 * 2;
  const uint32_t o_off = (w * 16 + l16) * (uint32_t)a.out_rs * 2 + lg * 8;
  const uint32_t f_off = lane * 16;
  auto matrices = [&](int c) {
    return make_rsrc(wsb + (int64_t)c * a.hv * GdnWorkspace::kHead, GdnWorkspace::kHead);
  };
  auto ld_frag = [&](rsrc_t b, int at) {
    return (u32x4)__builtin_amdgcn_raw_buffer_load_b128(b, f_off, at, 0);
  };
  auto ld_f32 = [&](rsrc_t b, uint32_t off, int at) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, off, at, 0));
  };
  auto ld_factor = [&](rsrc_t b, int i) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                         b, (w * 16 + lg * 4) * 4, kVec + i * CH * 4, 0));
  };
  auto load_qk = [&](Ops& o, int c) {
    const int n = min(rows - c * CH, CH);
    const rsrc_t kr = row_rsrc(kb + (int64_t)c * CH * a.k_rs, a.k_rs, n);
    const rsrc_t qr = row_rsrc(qb + (int64_t)c * CH * a.q_rs, a.q_rs, n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o.k[j].load(kr, k_off + j * 16 * krs);
      o.q[j].load(qr, q_off + j * 16 * qrs);
    }
  };
  auto load_t = [&](Ops& o, int c) {
    const rsrc_t vr = row_rsrc(vb + (int64_t)c * CH * a.v_rs, a.v_rs, min(rows - c * CH, CH));
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __builtin_amdgcn_raw_buffer_load_b16(vr, v_off + i * vrs, 0, 0);
    const rsrc_t m = matrices(c);
    o.c_rhs = ld_factor(m, 0);
    o.c_upd = ld_factor(m, 1);
    o.c_out = ld_f32(m, (w * 16 + l16) * 4, kVec + 2 * CH * 4);
    o.decay = ld_f32(m, 0, kVec + GdnWorkspace::kDecay);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int e = 0; e < 3; ++e) o.t[ks][e] = ld_frag(m, ((frag_of(w, 0) + ks) * 3 + e) * kF);
  };
  auto load_p = [&](Ops& o, int c) {
    const rsrc_t m = matrices(c), kr = make_rsrc(ktb + (int64_t)c * a.hk * kKey, kKey);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) o.kt[t][ks] = ld_frag(kr, ((w * MT + t) * 2 + ks) * kF);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        o.p[ks][e] = ld_frag(m, GdnWorkspace::kT + ((frag_of(w, 0) + ks) * 2 + e) * kF);
  };

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  // where rows 4 lg + i of row tile w are, in the order of tokens of T, P and
  // the transposed keys
  const int lt_at = l16 * LT + (w >> 1) * 32 + lg * 8 + (w & 1) * 4;
  auto lt_frag = [&](const uint16_t* m, int ks) {
    return *(const u32x4*)(m + l16 * LT + ks * 32 + lg * 8);
  };
  auto step = [&](const Ops& cur, Ops& nxt, int c) {
    const int cn = min(c + 1, nch - 1);
    // 1: partial K S and (Q S)^T of the wave's key dims
    u32x4 sp[3];
    split8<3>(S[0], MT == 2 ? S[MT - 1] : zero, sp);
    KeyFrag<DK> s[3];
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
      for (int i = 0; i < 2 * MT; ++i) s[e].x[i] = sp[e][i];
    f32x4 Z[4], Q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) Z[j] = Q[j] = zero;
#pragma unroll
    for (int e = 2; e >= 0; --e)
#pragma unroll
      for (int j = 0; j < 4; ++j) Z[j] = mfma_key(cur.k[j], s[e], Z[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) lds.Z[w][j][lane] = Z[j];
#pragma unroll
    for (int e = 1; e >= 0; --e)
#pragma unroll
      for (int j = 0; j < 4; ++j) Q[j] = mfma_key(s[e], cur.q[j], Q[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) lds.O[w][j][lane] = Q[j];
    load_qk(nxt, cn);
#pragma unroll
    for (int i = 0; i < 20; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i >= 4 && (i & 1)) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __syncthreads();
    // 2: right-hand sides v - e^G S k of row tile w
    {
      f32x4 z[4], x;
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = lds.Z[j][w][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = fmaf(-cur.c_rhs[i], (z[0][i] + z[1][i]) + (z[2][i] + z[3][i]), lo_f(cur.v[i]));
      u32x4 p[3];
      split8<3>(x, zero, p);
#pragma unroll
      for (int e = 0; e < 3; ++e) *(u32x2*)(lds.R[e] + lt_at) = u32x2{p[e][0], p[e][1]};
    }
    __syncthreads();
    // 3: U = T R of row tile w
    u32x4 x[NK][3];
    f32x4 z[4], O;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int e = 0; e < 3; ++e) x[ks][e] = lt_frag(lds.R[e], ks);
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = lds.O[j][w][lane];
    load_t(nxt, cn);
    __builtin_amdgcn_sched_barrier(0);   // all reads in flight before the first product
    f32x4 U = zero;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      U = mfma_bf16(cur.t[ks][2], x[ks][0], U);
      U = mfma_bf16(cur.t[ks][0], x[ks][2], U);
      U = mfma_bf16(cur.t[ks][1], x[ks][1], U);
      U = mfma_bf16(cur.t[ks][1], x[ks][0], U);
      U = mfma_bf16(cur.t[ks][0], x[ks][1], U);
      U = mfma_bf16(cur.t[ks][0], x[ks][0], U);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) O[i] = cur.c_out * ((z[0][i] + z[1][i]) + (z[2][i] + z[3][i]));
    {
      f32x4 y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = U[i] * cur.c_upd[i];
      u32x4 xp[3], up[2];
      split8<3>(y, zero, xp);
      split8<2>(U, zero, up);
#pragma unroll
      for (int e = 0; e < 3; ++e) *(u32x2*)(lds.X[e] + lt_at) = u32x2{xp[e][0], xp[e][1]};
#pragma unroll
      for (int e = 0; e < 2; ++e) *(u32x2*)(lds.U[e] + lt_at) = u32x2{up[e][0], up[e][1]};
    }
    __syncthreads();
    // 4: the state, and the outputs of row tile w
    u32x4 xs[2][3], u[NK][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int e = 0; e < 3; ++e) xs[ks][e] = lt_frag(lds.X[e], ks);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) u[ks][e] = lt_frag(lds.U[e], ks);
    load_p(nxt, cn);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[m][i] *= cur.decay;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int e = 2; e >= 0; --e)
#pragma unroll
        for (int m = 0; m < MT; ++m) S[m] = mfma_bf16(cur.kt[m][ks], xs[ks][e], S[m]);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      O = mfma_bf16(u[ks][0], cur.p[ks][1], O);
      O = mfma_bf16(u[ks][1], cur.p[ks][0], O);
      O = mfma_bf16(u[ks][0], cur.p[ks][0], O);
    }
    const rsrc_t orr = row_rsrc(ob + (int64_t)c * CH * a.out_rs, a.out_rs, min(rows - c * CH, CH));
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2(O[0], O[1]), pack2(O[2], O[3])}, orr, o_off,
                                          0, 0);
  };

  Ops x, y;
  load_qk(x, 0);
  load_t(x, 0);
  load_p(x, 0);
  for (int c = 0; c < nch; c += 2) {
    step(x, y, c);
    if (c + 1 < nch) step(y, x, c + 1);
  }
  if (in_pool) {
#pragma unroll
    for (int m = 0; m < MT; ++m) *(f32x4*)(pool + m * 4) = S[m];
  }
}

template <int DK>
__global__ __launch_bounds__(kBlock) void gdn_scan_few(GdnArgs a) {
  __shared__ FewLds lds;
  const ScanWork k = scan_work(a, a.dv / 16);
  if (k.nch <= 0) return;                     // no tokens: the slot stays as it is
  const int lane = (int)(threadIdx.x & 63);
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (w < 2)
    scan_few<DK, 1>(a, lds, k.r, k.h, k.slice * 16, k.row_lo, k.rows, k.base, k.nch, w, lane);
  else
    scan_few<DK, 2>(a, lds, k.r, k.h, k.slice * 16, k.row_lo, k.rows, k.base, k.nch, w, lane);
}

namespace {
constexpr int kScanWaves = 4;      // compute waves of gdn_scan, and as many loaders

// Workgroups of a scan that takes `width` value columns in each.
int64_t scan_grid(int64_t batch, int64_t hk, int64_t hv, int64_t dv, int width) {
  const int64_t groups = (batch * hk + kXcds - 1) / kXcds * kXcds;
  return groups * (hv / hk) * ((dv + width - 1) / width);
}

template <int DK>
hipError_t launch_scan(const GdnArgs& a, hipStream_t s) {
  constexpr int NW = kScanWaves, NL = kScanWaves;
  const int64_t grid = scan_grid(a.batch, a.hk, a.hv, a.dv, 16 * NW);
  hipLaunchKernelGGL((gdn_scan<DK, NW, NL>), dim3((unsigned)grid), dim3(64 * (NW + NL)), 0, s, a,
                     (a.dv + 16 * NW - 1) / (16 * NW));
  return hipGetLastError();
}

template <int DK>
hipError_t launch_few(const GdnArgs& a, hipStream_t s) {
  const int64_t grid = scan_grid(a.batch, a.hk, a.hv, a.dv, 16);
  hipLaunchKernelGGL((gdn_scan_few<DK>), dim3((unsigned)grid), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_dk(GdnArgs a, hipStream_t s) {
  const int64_t tiles = (int64_t)a.batch * a.hv * (a.dv / 16);
  const bool few = tiles <= device_cus();
  a.sorted = !few && a.batch > 1 && a.batch <= kSortMax;
  const int64_t grid = (int64_t)a.n_chunks * a.hv + a.sorted;
  hipLaunchKernelGGL((gdn_chunk<DK>), dim3((unsigned)grid), dim3(kBlock), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Few (request, head, 16 columns), at most one to a CU: four waves to each.
  // One request of 32,768 tokens, 32 heads x 128: 1.10 ms, and 1.70 by the
  // other kernel; eight such requests of 8,196 tokens in all: 0.34 ms, and 0.16
  // to 0.20 by the other.
  if (few) return launch_few<DK>(a, s);
  return launch_scan<DK>(a, s);
}
}  // namespace

// Of the scans' grids only that of many columns can be too large: the other is
// for at most one workgroup a CU.
bool gdn_prefill_fits(int64_t n_chunks, int64_t batch, int64_t hk, int64_t hv, int64_t dv) {
  return n_chunks <= (0x7FFFFFFFLL - 1) / hv &&
         scan_grid(batch, hk, hv, dv, 16 * kScanWaves) <= 0x7FFFFFFFLL;
}

hipError_t launch_gdn_prefill(const GdnArgs& a, hipStream_t s) {
  if (a.dk == 128) return launch_dk<128>(a, s);
  if (a.dk == 64) return launch_dk<64>(a, s);
  return hipErrorNotSupported;
}

}  // namespace sc
