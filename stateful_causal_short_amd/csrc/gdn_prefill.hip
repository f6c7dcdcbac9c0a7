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
// and P of every chunk at once; gdn_scan walks each request's chunks with the
// state, split over the value columns, which never mix.
//
// Precision: the state and every sum are fp32. Products run on bf16 MFMA with
// each fp32 factor cut into 16-bit parts (x = hi + mid + lo to 2^-24) and
// the small cross terms left out; q, k and v enter as they are, which is
// exact: the unit lengths of q and k are row factors applied in fp32. P and
// the copy of U it multiplies carry two parts (2^-16): their product only
// reaches the bf16 output.
#include "conv_device.hpp"
#include "gdn_device.hpp"

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
__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  f32x2 p = {x, y};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// N 16-bit parts of two values, packed: each part is the bf16 nearest to what
// the parts before it leave.
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t* part) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    part[n] = pack2(x, y);
    if (n + 1 < N) {
      x -= lo_f(part[n]);
      y -= hi_f(part[n]);
    }
  }
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
// gdn_chunk: T and P of one (chunk, value head), four waves.
//
// Wave w owns rows 16w..16w+15. K K^T and Q K^T are 16x16x32 bf16 products of
// raw rows read from global memory as MFMA operands (both operands of K K^T
// have the same lane layout). The unit lower triangular inverse goes by
// blocks: the four 16 x 16 diagonal blocks by forward substitution, a lane per
// column, then T_ij = -T_ii (A_ij T_jj) at 16 and at 32 on fp32 MFMA.
// The first value head of a key head also writes the keys transposed, as the
// scan's state update multiplies by them.
// ---------------------------------------------------------------------------
template <int DK>
__global__ __launch_bounds__(kBlock) void gdn_chunk(GdnArgs a) {
  constexpr int KS = DK / 32;
  constexpr int LD = 68;                      // fp32 row stride of the LDS matrices
  __shared__ __align__(16) float Am[CH * LD];
  __shared__ __align__(16) float Tm[CH * LD];
  __shared__ double Gs[CH];
  __shared__ float beta_s[CH], rk_s[CH], rq_s[CH];
  __shared__ __align__(16) uint16_t Kl[CH * (DK + 8)];

  const int h = (int)(blockIdx.x % (unsigned)a.hv);
  const int id = (int)(blockIdx.x / (unsigned)a.hv);
  const Chunk c = chunk_of(a, id);
  if (c.n == 0) return;
  const int rep = a.hv / a.hk, hk = h / rep;
  const int lane = (int)(threadIdx.x & 63), w = (int)(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const bool put_kt = h == hk * rep;

  // rows as MFMA operands: lane holds row l16 of a tile, 8 values from 8 lg
  auto row_frag = [&](const void* p, int64_t rs, int t, int ks) {
    u32x4 v = {0, 0, 0, 0};
    if (t < c.n)
      v = ld16((const uint16_t*)p + (int64_t)(c.row0 + t) * rs + hk * DK + ks * 32 + lg * 8);
    return v;
  };
  u32x4 kw[KS], qw[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    kw[ks] = row_frag(a.k, a.k_rs, w * 16 + l16, ks);
    qw[ks] = row_frag(a.q, a.q_rs, w * 16 + l16, ks);
  }

  // gates: wave 0, a lane per token; the running sum in fp64, so that the
  // difference of two of a chunk's sums keeps fp32 accuracy whatever came
  // before. A decay below e^-110 is zero in fp32 already.
  if (w == 0) {
    float g = 0.f, be = 0.f;
    if (lane < c.n) {
      g = gdn_log_decay(a, c.row0 + lane, h);
      g = g < -110.f ? -110.f : g;
      be = gdn_beta(a, c.row0 + lane, h);
    }
    double s = g;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(s, d);
      if (lane >= d) s += o;
    }
    Gs[lane] = s;
    beta_s[lane] = be;
  }
  // unit lengths
  {
    float kk = 0.f, qq = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        kk = fmaf(lo_f(kw[ks][e]), lo_f(kw[ks][e]), kk);
        kk = fmaf(hi_f(kw[ks][e]), hi_f(kw[ks][e]), kk);
        qq = fmaf(lo_f(qw[ks][e]), lo_f(qw[ks][e]), qq);
        qq = fmaf(hi_f(qw[ks][e]), hi_f(qw[ks][e]), qq);
      }
    kk += __shfl_xor(kk, 16);
    kk += __shfl_xor(kk, 32);
    qq += __shfl_xor(qq, 16);
    qq += __shfl_xor(qq, 32);
    if (lg == 0) {
      rk_s[w * 16 + l16] = a.l2norm ? rsqrtf(kk + kL2Eps) : 1.f;
      rq_s[w * 16 + l16] = a.scale * (a.l2norm ? rsqrtf(qq + kL2Eps) : 1.f);
    }
  }
  if (put_kt) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      *(u32x4*)(Kl + (w * 16 + l16) * (DK + 8) + ks * 32 + lg * 8) = kw[ks];
  }
  // raw products: tiles (w, j), j <= w
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (j <= w) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const u32x4 bj = row_frag(a.k, a.k_rs, j * 16 + l16, ks);
        kk[j] = mfma_bf16(kw[ks], bj, kk[j]);
        qk[j] = mfma_bf16(qw[ks], bj, qk[j]);
      }
    }
  }
  __syncthreads();

  char* const ws = a.ws + ((int64_t)id * a.hv + h) * GdnWorkspace::kHead;
  // row factors of the scan
  if (w == 0) {
    float* vec = (float*)(ws + GdnWorkspace::kT + GdnWorkspace::kP);
    const float eg = expf((float)Gs[lane]), rk = rk_s[lane], be = beta_s[lane];
    vec[lane] = be;
    vec[CH + lane] = be * eg * rk;
    vec[2 * CH + lane] = rk * expf((float)(Gs[CH - 1] - Gs[lane]));
    vec[3 * CH + lane] = rq_s[lane] * eg;
    vec[4 * CH + lane] = expf((float)Gs[CH - 1]);
  }
  // A into LDS, P into LDS (Tm, until T overwrites it)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = w * 16 + lg * 4 + i, s = j * 16 + l16;
      float av = 0.f, pv = 0.f;
      if (s <= t) {
        const float d = expf((float)(Gs[t] - Gs[s])) * rk_s[s];
        if (s < t) av = beta_s[t] * rk_s[t] * d * kk[j][i];
        pv = rq_s[t] * d * qk[j][i];
      }
      Am[t * LD + s] = av;
      Tm[t * LD + s] = pv;
    }
  }
  __syncthreads();
  // matrix rows as operand fragments: N parts of 8 adjacent values
  auto put_frags = [&](auto parts, const float* m, char* dst) {
    constexpr int N = decltype(parts)::value;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (w < 2 && ks == 1) continue;
      const float* p = m + (w * 16 + l16) * LD + ks * 32 + lg * 8;
      const f32x4 x = *(const f32x4*)p, y = *(const f32x4*)(p + 4);
      uint32_t part[4][N];
      split2<N>(x[0], x[1], part[0]);
      split2<N>(x[2], x[3], part[1]);
      split2<N>(y[0], y[1], part[2]);
      split2<N>(y[2], y[3], part[3]);
#pragma unroll
      for (int n = 0; n < N; ++n)
        *(u32x4*)(dst + (frag_of(w, ks) * N + n) * GdnWorkspace::kFrag + lane * 16) =
            u32x4{part[0][n], part[1][n], part[2][n], part[3][n]};
    }
  };
  put_frags(std::integral_constant<int, 2>{}, Tm, ws + GdnWorkspace::kT);
  if (put_kt) {
    // keys transposed: lane holds key dim l16 of tile m, 8 tokens from 8 lg
    char* kt = a.ws + (int64_t)a.n_chunks * a.hv * GdnWorkspace::kHead +
               ((int64_t)id * a.hk + hk) * (DK * CH * 2);
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) {
      const int f = w * (DK / 32) + i;        // fragment (tile m, k step ks)
      const int m = f >> 1, ks = f & 1;
      const uint16_t* p = Kl + (ks * 32 + lg * 8) * (DK + 8) + m * 16 + l16;
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = (uint32_t)p[(2 * e) * (DK + 8)] | ((uint32_t)p[(2 * e + 1) * (DK + 8)] << 16);
      *(u32x4*)(kt + f * GdnWorkspace::kFrag + lane * 16) = v;
    }
  }
  __syncthreads();
  // T: zero above the diagonal blocks; diagonal blocks by substitution
  for (int i = (int)threadIdx.x; i < CH * LD / 4; i += kBlock)
    *(f32x4*)(Tm + i * 4) = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  if (w == 0) {
    const float* ab = Am + lg * 16 * LD + lg * 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == l16 ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(-ab[i * LD + j], x[j], s);
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) Tm[(lg * 16 + i) * LD + lg * 16 + l16] = x[i];
  }
  __syncthreads();
  // 16 x 16 product of LDS blocks at (rx, cx) of X and (ry, cy) of Y
  auto mul16 = [&](const float* X, int rx, int cx, const float* Y, int ry, int cy, f32x4 acc) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      acc = mfma_f32(X[(rx * 16 + l16) * LD + cx * 16 + k * 4 + lg],
                     Y[(ry * 16 + k * 4 + lg) * LD + cy * 16 + l16], acc);
    return acc;
  };
  auto put16 = [&](float* X, int r, int col, f32x4 v, float sign) {
#pragma unroll
    for (int i = 0; i < 4; ++i) X[(r * 16 + lg * 4 + i) * LD + col * 16 + l16] = sign * v[i];
  };
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  // blocks (1,0) and (3,2): the inner product goes where A's block was
  if (w < 2) {
    const int b = 2 * w;
    put16(Am, b + 1, b, mul16(Am, b + 1, b, Tm, b, b, zero), 1.f);
  }
  __syncthreads();
  if (w < 2) {
    const int b = 2 * w;
    put16(Tm, b + 1, b, mul16(Tm, b + 1, b + 1, Am, b + 1, b, zero), -1.f);
  }
  __syncthreads();
  // the 32 x 32 block below: a wave per 16 x 16 tile
  {
    const int i = 2 + (w >> 1), j = w & 1;
    f32x4 y = mul16(Am, i, 1, Tm, 1, j, zero);     // Tm(0, 1) is zero
    if (j == 0) y = mul16(Am, i, 0, Tm, 0, 0, y);
    __syncthreads();
    put16(Am, i, j, y, 1.f);
    __syncthreads();
    f32x4 z = mul16(Tm, i, 2, Am, 2, j, zero);
    if (i == 3) z = mul16(Tm, 3, 3, Am, 3, j, z);
    put16(Tm, i, j, z, -1.f);
  }
  __syncthreads();
  put_frags(std::integral_constant<int, 3>{}, Tm, ws);
}

// ---------------------------------------------------------------------------
// gdn_scan: one request's chunks in turn for one value head and 16 NV of its
// value columns, four waves.
//
// The state is held as S^T (DK x 16 NV) in MFMA accumulators, DK/64 tiles of
// 16 key dims a wave, and once a chunk also as three bf16 parts in LDS, where
// every wave reads it as the right operand of its 16 rows of K S and Q S
// (q and k rows come from global memory as left operands). Three barriers a
// chunk: state parts written, right-hand sides written, U written. Operands of
// the next chunk are loaded while this one is computed.
// ---------------------------------------------------------------------------
template <int DK, int NV>
struct ScanOperands {
  static constexpr int KS = DK / 32;
  static constexpr int MT = DK / 64;
  u32x4 k[KS], q[KS];          // row tile w
  u32x4 t[2][3], p[2][2];      // T and P of row tile w
  u32x4 kt[MT][2];             // transposed keys, tiles w MT + m
  uint16_t v[NV][4];
  f32x4 c1, c2, c3, c4;
  float decay;
};

template <int DK, int NV>
__global__ __launch_bounds__(kBlock) void gdn_scan(GdnArgs a) {
  constexpr int KS = DK / 32, MT = DK / 64, W = 16 * NV;
  constexpr int LS = DK + 8, LT = CH + 8;     // LDS row strides (elements): banks differ by row
  __shared__ __align__(16) uint16_t Sl[3][W * LS];
  __shared__ __align__(16) uint16_t Rl[3][W * LT];
  __shared__ __align__(16) uint16_t Ul[2][W * LT];
  __shared__ __align__(16) uint16_t Wl[3][W * LT];

  const int slices = (a.dv + W - 1) / W;
  const int slice = (int)(blockIdx.x % (unsigned)slices);
  const unsigned rest = blockIdx.x / (unsigned)slices;
  const int h = (int)(rest % (unsigned)a.hv);
  const int r = (int)(rest / (unsigned)a.hv);
  const int hk = h / (a.hv / a.hk);
  const int T = (int)a.num_tokens;
  const int s0 = a.qsl[r], row_lo = min(max(s0, 0), T);
  const int row_hi = min(max(a.qsl[r + 1], row_lo), T);
  const int base = max(s0, 0) / CH + r;
  const int nch = min((row_hi - row_lo + CH - 1) / CH, a.n_chunks - base);
  if (nch <= 0) return;                       // no tokens: the slot stays as it is

  const int lane = (int)(threadIdx.x & 63), w = (int)(threadIdx.x >> 6);
  const int l16 = lane & 15, lg = lane >> 4;
  const int col0 = slice * W;
  const int32_t slot = a.slots[(int64_t)r * a.slot_stride];
  const bool in_pool = slot >= 0 && slot < a.num_slots;
  const bool cont = in_pool && a.has_init[r];
  float* const pool = a.pool + ((int64_t)slot * a.hv + h) * ((int64_t)a.dv * DK);

  f32x4 S[MT][NV];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      S[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int col = col0 + n * 16 + l16;
      if (cont && col < a.dv)
        S[m][n] = *(const f32x4*)(pool + (int64_t)col * DK + (w * MT + m) * 16 + lg * 4);
    }
  auto put_state = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        uint32_t x[3], y[3];
        split2<3>(S[m][n][0], S[m][n][1], x);
        split2<3>(S[m][n][2], S[m][n][3], y);
#pragma unroll
        for (int e = 0; e < 3; ++e)
          *(uint2*)(Sl[e] + (n * 16 + l16) * LS + (w * MT + m) * 16 + lg * 4) = uint2{x[e], y[e]};
      }
  };

  const char* const kt_base = a.ws + (int64_t)a.n_chunks * a.hv * GdnWorkspace::kHead;
  using Ops = ScanOperands<DK, NV>;
  auto load = [&](Ops& o, int c) {
    const int row0 = row_lo + c * CH, n = min(row_hi - row0, CH);
    const char* ws = a.ws + ((int64_t)(base + c) * a.hv + h) * GdnWorkspace::kHead;
    const char* kt = kt_base + ((int64_t)(base + c) * a.hk + hk) * (DK * CH * 2);
    const int t = w * 16 + l16;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      o.k[ks] = o.q[ks] = u32x4{0, 0, 0, 0};
      if (t < n) {
        o.k[ks] = ld16((const uint16_t*)a.k + (int64_t)(row0 + t) * a.k_rs + hk * DK + ks * 32 + lg * 8);
        o.q[ks] = ld16((const uint16_t*)a.q + (int64_t)(row0 + t) * a.q_rs + hk * DK + ks * 32 + lg * 8);
      }
    }
#pragma unroll
    for (int nn = 0; nn < NV; ++nn) {
      const int col = col0 + nn * 16 + l16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tt = w * 16 + lg * 4 + i;
        o.v[nn][i] = 0;
        if (tt < n && col < a.dv)
          o.v[nn][i] = ((const uint16_t*)a.v)[(int64_t)(row0 + tt) * a.v_rs + (int64_t)h * a.dv + col];
      }
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 1 && w < 2) continue;
#pragma unroll
      for (int e = 0; e < 3; ++e)
        o.t[ks][e] = ld16(ws + (frag_of(w, ks) * 3 + e) * GdnWorkspace::kFrag + lane * 16);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        o.p[ks][e] = ld16(ws + GdnWorkspace::kT + (frag_of(w, ks) * 2 + e) * GdnWorkspace::kFrag + lane * 16);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        o.kt[m][ks] = ld16(kt + ((w * MT + m) * 2 + ks) * GdnWorkspace::kFrag + lane * 16);
    const float* vec = (const float*)(ws + GdnWorkspace::kT + GdnWorkspace::kP) + w * 16 + lg * 4;
    o.c1 = *(const f32x4*)vec;
    o.c2 = *(const f32x4*)(vec + CH);
    o.c3 = *(const f32x4*)(vec + 2 * CH);
    o.c4 = *(const f32x4*)(vec + 3 * CH);
    o.decay = ((const float*)(ws + GdnWorkspace::kT + GdnWorkspace::kP))[4 * CH];
  };

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  Ops cur, nxt;
  load(cur, 0);
  put_state();
  for (int c = 0; c < nch; ++c) {
    if (c + 1 < nch) load(nxt, c + 1);
    __syncthreads();
    f32x4 Z[NV], O[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) Z[n] = O[n] = zero;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int e = 2; e >= 0; --e)
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const u32x4 s = *(const u32x4*)(Sl[e] + (n * 16 + l16) * LS + ks * 32 + lg * 8);
          Z[n] = mfma_bf16(cur.k[ks], s, Z[n]);
          O[n] = mfma_bf16(cur.q[ks], s, O[n]);
        }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = cur.c1[i] * lo_f(cur.v[n][i]) - cur.c2[i] * Z[n][i];
        O[n][i] *= cur.c4[i];
      }
      uint32_t p0[3], p1[3];
      split2<3>(x[0], x[1], p0);
      split2<3>(x[2], x[3], p1);
#pragma unroll
      for (int e = 0; e < 3; ++e)
        *(uint2*)(Rl[e] + (n * 16 + l16) * LT + w * 16 + lg * 4) = uint2{p0[e], p1[e]};
    }
    __syncthreads();
    f32x4 U[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) U[n] = zero;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 1 && w < 2) continue;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        u32x4 x[3];
#pragma unroll
        for (int e = 0; e < 3; ++e)
          x[e] = *(const u32x4*)(Rl[e] + (n * 16 + l16) * LT + ks * 32 + lg * 8);
        U[n] = mfma_bf16(cur.t[ks][2], x[0], U[n]);
        U[n] = mfma_bf16(cur.t[ks][0], x[2], U[n]);
        U[n] = mfma_bf16(cur.t[ks][1], x[1], U[n]);
        U[n] = mfma_bf16(cur.t[ks][1], x[0], U[n]);
        U[n] = mfma_bf16(cur.t[ks][0], x[1], U[n]);
        U[n] = mfma_bf16(cur.t[ks][0], x[0], U[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      uint32_t u0[2], u1[2], s0p[3], s1p[3];
      split2<2>(U[n][0], U[n][1], u0);
      split2<2>(U[n][2], U[n][3], u1);
      split2<3>(U[n][0] * cur.c3[0], U[n][1] * cur.c3[1], s0p);
      split2<3>(U[n][2] * cur.c3[2], U[n][3] * cur.c3[3], s1p);
      const int at = (n * 16 + l16) * LT + w * 16 + lg * 4;
#pragma unroll
      for (int e = 0; e < 2; ++e) *(uint2*)(Ul[e] + at) = uint2{u0[e], u1[e]};
#pragma unroll
      for (int e = 0; e < 3; ++e) *(uint2*)(Wl[e] + at) = uint2{s0p[e], s1p[e]};
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NV; ++n) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[m][n][i] *= cur.decay;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int e = 2; e >= 0; --e) {
          const u32x4 x = *(const u32x4*)(Wl[e] + (n * 16 + l16) * LT + ks * 32 + lg * 8);
#pragma unroll
          for (int m = 0; m < MT; ++m) S[m][n] = mfma_bf16(cur.kt[m][ks], x, S[m][n]);
        }
    }
    if (c + 1 < nch) put_state();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (ks == 1 && w < 2) continue;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        u32x4 x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[e] = *(const u32x4*)(Ul[e] + (n * 16 + l16) * LT + ks * 32 + lg * 8);
        O[n] = mfma_bf16(cur.p[ks][1], x[0], O[n]);
        O[n] = mfma_bf16(cur.p[ks][0], x[1], O[n]);
        O[n] = mfma_bf16(cur.p[ks][0], x[0], O[n]);
      }
    }
    const int row0 = row_lo + c * CH;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int col = col0 + n * 16 + l16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + w * 16 + lg * 4 + i;
        if (row < row_hi && col < a.dv)
          ((uint16_t*)a.out)[(int64_t)row * a.out_rs + (int64_t)h * a.dv + col] = to_bf16(O[n][i]);
      }
    }
    cur = nxt;
  }
  if (in_pool) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int col = col0 + n * 16 + l16;
        if (col < a.dv)
          *(f32x4*)(pool + (int64_t)col * DK + (w * MT + m) * 16 + lg * 4) = S[m][n];
      }
  }
}

namespace {
template <int DK, int NV>
hipError_t launch_scan(const GdnArgs& a, hipStream_t s) {
  const int slices = (a.dv + 16 * NV - 1) / (16 * NV);
  const int64_t grid = (int64_t)a.batch * a.hv * slices;
  if (grid > 0x7FFFFFFFLL) return hipErrorNotSupported;
  hipLaunchKernelGGL((gdn_scan<DK, NV>), dim3((unsigned)grid), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_dk(const GdnArgs& a, hipStream_t s) {
  const int64_t grid = (int64_t)a.n_chunks * a.hv;
  if (grid > 0x7FFFFFFFLL) return hipErrorNotSupported;
  hipLaunchKernelGGL((gdn_chunk<DK>), dim3((unsigned)grid), dim3(kBlock), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_scan<DK, 1>(a, s);
}
}  // namespace

hipError_t launch_gdn_prefill(const GdnArgs& a, hipStream_t s) {
  if (a.dk == 128) return launch_dk<128>(a, s);
  if (a.dk == 64) return launch_dk<64>(a, s);
  return hipErrorNotSupported;
}

}  // namespace sc
