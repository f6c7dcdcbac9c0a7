// Norms of the query and key heads, the position rotation, and the write of
// keys and values into the paged cache, in one pass.
//
//   x^ = w o x / sqrt(mean(x^2) + eps);  pairs (x1, x2) of the first `rot`
//   values of a head turn: (x1 cos - x2 sin, x2 cos + x1 sin)
//
// A head is held by hd/8 lanes, 8 values a lane, as two runs of four: for the
// half-split rotation a lane owns values 4l.. and rot/2 + 4l.., so both members
// of a pair are in one lane and nothing is exchanged after the norm's sum. The
// same lanes take several heads of a token in turn, with the token's cos and
// sin in registers. All arithmetic is fp32 with one rounding at the store. The
// kernel moves bytes: each row is read once and written once (keys twice with
// k_out and a cache). 32,768 tokens of 16 + 2 + 2 heads x 128, 355 MB: 84 us
// (4.2 TB/s; a row copy reaches 5.8). Loading the next heads while these are
// stored took 90 us, two heads at a time 87, ten 84. 17 tokens: 3.5 us, the
// latency of three dependent loads.
#include "attn.hpp"
#include "common.hpp"

#include <algorithm>

namespace sc {

namespace {

__device__ __forceinline__ void unpack4(uint2 w, float* f) {
  f[0] = __uint_as_float(w.x << 16);
  f[1] = __uint_as_float(w.x & 0xFFFF0000u);
  f[2] = __uint_as_float(w.y << 16);
  f[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ uint2 pack4(const float* f) {
  f32x2 a = {f[0], f[1]}, b = {f[2], f[3]};
  return uint2{__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2)),
               __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf16x2))};
}

// Sum over the L lanes of a head (8, 16 or 32, aligned).
template <int L>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

}  // namespace

// Token blockIdx.x * PER + ..., heads [per blockIdx.y, per (blockIdx.y + 1)) of
// its query, key and (copied to the cache) value heads.
template <int HD, int N>
__global__ __launch_bounds__(kBlock) void qk_norm_rope(QkNormArgs a, int per) {
  constexpr int L = HD / 8, PER = kBlock / L;
  const int heads = a.nq + a.nkv + (a.vc.p ? a.nkv : 0);
  const int64_t t = (int64_t)blockIdx.x * PER + threadIdx.x / L;
  const int l = (int)(threadIdx.x % L);
  if (t >= a.num_tokens) return;               // whole heads leave: sums stay within a head
  const int h_lo = (int)blockIdx.y * per, h_hi = min(h_lo + per, heads);

  // the lane's two runs of four values in a query or key head
  const int half = a.rot / 2;
  const bool turns = l * 8 < a.rot;
  const int d0 = turns && !a.interleaved ? l * 4 : l * 8;
  const int d1 = turns && !a.interleaved ? half + l * 4 : l * 8 + 4;
  int64_t block = -1, in_block = 0;            // cache row, block -1: none
  if (a.slots && h_hi > a.nq) {
    const int64_t slot = a.slots[t];
    if (slot >= 0 && slot < (int64_t)a.num_blocks * a.block_size) {
      block = slot / a.block_size;
      in_block = slot - block * a.block_size;
    }
  }
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (turns && h_lo < a.nq + a.nkv) {
    int64_t pos = a.positions[t];
    pos = pos < 0 ? 0 : (pos >= a.max_pos ? a.max_pos - 1 : pos);
    if (a.table_f32) {
      const float* p = (const float*)a.table + pos * a.table_rs + l * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[e] = p[e];
        sn[e] = p[half + e];
      }
    } else {
      const uint16_t* p = (const uint16_t*)a.table + pos * a.table_rs + l * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[e] = __uint_as_float((uint32_t)p[e] << 16);
        sn[e] = __uint_as_float((uint32_t)p[half + e] << 16);
      }
    }
  }
  const uint16_t* const q = (const uint16_t*)a.q + t * a.q_rs;
  const uint16_t* const k = (const uint16_t*)a.k + t * a.k_rs;
  const uint16_t* const v = (const uint16_t*)a.v + t * a.v_rs;
  uint16_t* const qo = (uint16_t*)a.q_out + t * a.qo_rs;
  uint16_t* const ko = (uint16_t*)a.k_out + t * a.ko_rs;
  uint16_t* const kc = (uint16_t*)a.kc.p + block * a.kc.block_s + in_block * a.kc.token_s;
  uint16_t* const vc = (uint16_t*)a.vc.p + block * a.vc.block_s + in_block * a.vc.token_s;

  for (int h0 = h_lo; h0 < h_hi; h0 += N) {    // N heads' loads in flight together
    uint2 x0[N], x1[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int h = min(h0 + n, h_hi - 1);
      const bool is_v = h >= a.nq + a.nkv;
      const uint16_t* src = h < a.nq ? q + (int64_t)h * HD
                            : is_v   ? v + (int64_t)(h - a.nq - a.nkv) * HD
                                     : k + (int64_t)(h - a.nq) * HD;
      x0[n] = *(const uint2*)(src + (is_v ? l * 8 : d0));
      x1[n] = *(const uint2*)(src + (is_v ? l * 8 + 4 : d1));
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int h = h0 + n;
      if (h >= h_hi) break;
      if (h >= a.nq + a.nkv) {                 // a value head: copied
        if (block >= 0) {
          uint16_t* d = vc + (int64_t)(h - a.nq - a.nkv) * a.vc.head_s + l * 8;
          *(uint2*)d = x0[n];
          *(uint2*)(d + 4) = x1[n];
        }
        continue;
      }
      const bool is_q = h < a.nq;
      float x[8];
      unpack4(x0[n], x);
      unpack4(x1[n], x + 4);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      const float inv = rsqrtf(head_sum<L>(ss) * (1.f / HD) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv;
      if (const uint16_t* wp = (const uint16_t*)(is_q ? a.q_w : a.k_w)) {
        float wv[8];
        unpack4(*(const uint2*)(wp + d0), wv);
        unpack4(*(const uint2*)(wp + d1), wv + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= wv[e];
      }
      if (turns) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y1 = x[2 * e], y2 = x[2 * e + 1];
            x[2 * e] = y1 * cs[e] - y2 * sn[e];
            x[2 * e + 1] = y2 * cs[e] + y1 * sn[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y1 = x[e], y2 = x[4 + e];
            x[e] = y1 * cs[e] - y2 * sn[e];
            x[4 + e] = y2 * cs[e] + y1 * sn[e];
          }
        }
      }
      const uint2 y0 = pack4(x), y1 = pack4(x + 4);
      if (is_q || a.k_out) {
        uint16_t* d = is_q ? qo + (int64_t)h * HD : ko + (int64_t)(h - a.nq) * HD;
        *(uint2*)(d + d0) = y0;
        *(uint2*)(d + d1) = y1;
      }
      if (!is_q && block >= 0) {
        uint16_t* d = kc + (int64_t)(h - a.nq) * a.kc.head_s;
        *(uint2*)(d + d0) = y0;
        *(uint2*)(d + d1) = y1;
      }
    }
  }
}

namespace {
template <int HD>
hipError_t launch_hd(const QkNormArgs& a, hipStream_t s) {
  const int64_t heads = a.nq + a.nkv + (a.vc.p ? a.nkv : 0);
  constexpr int PER = kBlock / (HD / 8);
  const int64_t blocks = (a.num_tokens + PER - 1) / PER;
  // one head to a workgroup's lanes, and more as the tokens alone fill the chip
  // (eight workgroups a CU); four heads' loads together from four heads a lane
  const int64_t want = (int64_t)device_cus() * 8;
  const int64_t parts = std::min<int64_t>(heads, std::max<int64_t>(1, want / blocks));
  const int64_t per = (heads + parts - 1) / parts, ny = (heads + per - 1) / per;
  if (blocks > 0x7FFFFFFFLL || ny > 65535) return hipErrorNotSupported;
  const dim3 grid((unsigned)blocks, (unsigned)ny);
  if (per >= 4)
    hipLaunchKernelGGL((qk_norm_rope<HD, 4>), grid, dim3(kBlock), 0, s, a, (int)per);
  else
    hipLaunchKernelGGL((qk_norm_rope<HD, 1>), grid, dim3(kBlock), 0, s, a, (int)per);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t s) {
  switch (a.hd) {
    case 64: return launch_hd<64>(a, s);
    case 128: return launch_hd<128>(a, s);
    case 256: return launch_hd<256>(a, s);
  }
  return hipErrorNotSupported;
}

}  // namespace sc
