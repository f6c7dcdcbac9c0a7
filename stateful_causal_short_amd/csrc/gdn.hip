// Gated delta rule, recurrent form: one to a few tokens per request against a
// state in the slot pool.
//
//   S <- e^g S,  u = beta (v - S k),  S <- S + u k^T,  o = scale S q
//
// with S (DV x DK, fp32) of one value head, g = -exp(A_log) softplus(a +
// dt_bias), beta = sigmoid(b), and q, k scaled to unit length. Rows of S are
// independent given k and q, so a row is held by 16 lanes from its load to its
// store: the state is read once and written once however many tokens there
// are, and the products with k and q are sums over 16 lanes.
#include "gdn_device.hpp"

namespace sc {

// R rows of S per 16 lanes; a workgroup covers 16 R rows of one (request,
// head). The state (DK/64 x R 16-byte vectors a lane) is requested before
// anything else: the kernel is bound by its bytes (64 KB in and out per head at
// DK = DV = 128). SPEC: request r starts from the slot of its last accepted
// draft and leaves the state after each token in that token's slot.
// STREAM: state loads that keep nothing in the caches; the stores of R = 8
// never do (a state is not read again before the next step of the model).
template <int DK, int R, bool SPEC, bool STREAM>
__global__ __launch_bounds__(kBlock) void gdn_update(GdnArgs a, int row_blocks) {
  constexpr int NJ = DK / 64;
  const int rb = (int)(blockIdx.x % (unsigned)row_blocks);
  const unsigned rest = blockIdx.x / (unsigned)row_blocks;
  const int h = (int)(rest % (unsigned)a.hv);
  const int64_t r = rest / (unsigned)a.hv;
  const int l16 = (int)(threadIdx.x & 15);
  const int row0 = (rb * 16 + (int)(threadIdx.x >> 4)) * R;
  const int nq = a.nq;

  int32_t slot;
  if constexpr (SPEC) {
    const int acc = min(max(a.num_acc[r], 1), nq);
    slot = a.slots[r * a.slot_stride + acc - 1];
  } else {
    slot = a.slots[r * a.slot_stride];
  }
  const bool in_pool = slot >= 0 && slot < a.num_slots;
  const bool cont = in_pool && (!a.has_init || a.has_init[r]);
  const int64_t head_elems = (int64_t)a.dv * DK;
  const int64_t slot_elems = head_elems * a.hv;
  const int64_t off = h * head_elems + (int64_t)row0 * DK + l16 * 4;
  f32x4 S[R][NJ];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      S[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (cont && row0 + i < a.dv) {
        const f32x4* p = (const f32x4*)(a.pool + slot * slot_elems + off + i * DK + j * 64);
        S[i][j] = STREAM ? __builtin_nontemporal_load(p) : *p;
      }
    }

  const int hk = h / (a.hv / a.hk);
  for (int t = 0; t < nq; ++t) {
    const int64_t row = r * nq + t;
    const uint16_t* qp = (const uint16_t*)a.q + row * a.q_rs + hk * DK + l16 * 4;
    const uint16_t* kp = (const uint16_t*)a.k + row * a.k_rs + hk * DK + l16 * 4;
    float q[NJ][4], k[NJ][4], v[R];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const uint2 qw = *(const uint2*)(qp + j * 64), kw = *(const uint2*)(kp + j * 64);
      q[j][0] = __uint_as_float(qw.x << 16);
      q[j][1] = __uint_as_float(qw.x & 0xFFFF0000u);
      q[j][2] = __uint_as_float(qw.y << 16);
      q[j][3] = __uint_as_float(qw.y & 0xFFFF0000u);
      k[j][0] = __uint_as_float(kw.x << 16);
      k[j][1] = __uint_as_float(kw.x & 0xFFFF0000u);
      k[j][2] = __uint_as_float(kw.y << 16);
      k[j][3] = __uint_as_float(kw.y & 0xFFFF0000u);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      v[i] = row0 + i < a.dv ? bf16_at(a.v, row * a.v_rs + (int64_t)h * a.dv + row0 + i) : 0.f;
    const float eg = expf(gdn_log_decay(a, row, h));
    const float beta = gdn_beta(a, row, h);
    float qn = a.scale;
    if (a.l2norm) {
      float qq = 0.f, kk = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qq = fmaf(q[j][e], q[j][e], qq);
          kk = fmaf(k[j][e], k[j][e], kk);
        }
      qn *= rsqrtf(row16_sum(qq) + kL2Eps);
      const float kn = rsqrtf(row16_sum(kk) + kL2Eps);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) k[j][e] *= kn;
    }
    float o[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[i][j][e] *= eg;
          z = fmaf(S[i][j][e], k[j][e], z);
        }
      const float u = beta * (v[i] - row16_sum(z));
      float y = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[i][j][e] = fmaf(u, k[j][e], S[i][j][e]);
          y = fmaf(S[i][j][e], q[j][e], y);
        }
      o[i] = row16_sum(y) * qn;
    }
    // lane i of the 16 stores row i: one store of 16 R adjacent values
    float mine = o[0];
#pragma unroll
    for (int i = 1; i < R; ++i) mine = l16 == i ? o[i] : mine;
    if (l16 < R && row0 + l16 < a.dv)
      ((uint16_t*)a.out)[row * a.out_rs + (int64_t)h * a.dv + row0 + l16] = to_bf16(mine);
    if (SPEC || t == nq - 1) {
      const int32_t to = SPEC ? a.slots[r * a.slot_stride + t] : slot;
      if (to >= 0 && to < a.num_slots) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            if (row0 + i < a.dv) {
              f32x4* p = (f32x4*)(a.pool + to * slot_elems + off + i * DK + j * 64);
              if constexpr (R == 8) __builtin_nontemporal_store(S[i][j], p);
              else *p = S[i][j];
            }
      }
    }
  }
}

namespace {
template <int DK, int R, bool STREAM>
hipError_t launch_r(const GdnArgs& a, hipStream_t s) {
  const int row_blocks = (a.dv + 16 * R - 1) / (16 * R);
  const int64_t grid = (int64_t)a.batch * a.hv * row_blocks;
  if (grid > 0x7FFFFFFFLL) return hipErrorNotSupported;
  if (a.num_acc)
    hipLaunchKernelGGL((gdn_update<DK, R, true, false>), dim3((unsigned)grid), dim3(kBlock), 0, s,
                       a, row_blocks);
  else
    hipLaunchKernelGGL((gdn_update<DK, R, false, STREAM>), dim3((unsigned)grid), dim3(kBlock), 0,
                       s, a, row_blocks);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_dk(const GdnArgs& a, hipStream_t s) {
  // few (request, head) pairs: fewer rows per workgroup, until every CU has one
  const int64_t pairs = (int64_t)a.batch * a.hv;
  const int cus = device_cus();
  if (pairs * ((a.dv + 63) / 64) < cus) return launch_r<DK, 1, false>(a, s);
  if (pairs * ((a.dv + 127) / 128) < 2 * cus) return launch_r<DK, 4, false>(a, s);
  // Streaming loads where the states are 128 MB or more, which the 256 MB last
  // level would not keep over a model's layers. One-token updates of 32 heads
  // x 128 x 128, plain / streaming: 16 requests 15.3 / 17.3 us, 64 48.5 / 49.9,
  // 128 104.8 / 98.2, 512 389 / 369 (5.9 TB/s). Speculative updates write a
  // state for each draft and read one: 128 x 4 took 235 us, 255 streaming.
  // Streaming stores for R = 8, which starts at 16 requests of 32 heads; streaming
  // / plain, over 1 GB of states in all, as a model's layers have: 16 requests
  // 18.8 / 19.5 us, 24 20.9 / 26.6, 32 25.3 / 33.6, 64 49.2 / 51.8, 128 97.5 /
  // 107.7, 512 389 / 412; 16 x 4 drafts 31.1 / 42.6, 128 x 4 230 / 272. Over two
  // sets of states, which the last level keeps, 24 to 64 requests lose 2 to 8%.
  if (pairs * a.dv * DK * 4 >= (int64_t)128 << 20) return launch_r<DK, 8, true>(a, s);
  return launch_r<DK, 8, false>(a, s);
}
}  // namespace

hipError_t launch_gdn_update(const GdnArgs& a, hipStream_t s) {
  if (a.dk == 128) return launch_dk<128>(a, s);
  if (a.dk == 64) return launch_dk<64>(a, s);
  return hipErrorNotSupported;
}

}  // namespace sc
