// Norms of the query and key heads, the position rotation, and the write of
// keys and values into the paged cache, in one pass.
//
//   x^ = w o x / sqrt(mean(x^2) + eps);  pairs (x1, x2) of the first `rot`
//   values of a head turn: (x1 cos - x2 sin, x2 cos + x1 sin)
//
// A head is held by hd/8 lanes, 8 values a lane, as two runs of four: for the
// half-split rotation a lane owns values 4l.. and rot/2 + 4l.., so both members
// of a pair are in one lane and nothing is exchanged after the norm's sum. All
// arithmetic is fp32 with one rounding at the store. The kernel moves bytes:
// each row is read once and written once (keys twice with k_out and a cache).
#include "attn.hpp"
#include "common.hpp"

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

// Row index of a workgroup's heads: head rows are numbered token by token,
// query heads first, then key heads, then value heads (copied to the cache).
template <int HD>
__global__ __launch_bounds__(kBlock) void qk_norm_rope(QkNormArgs a) {
  constexpr int L = HD / 8, PER = kBlock / L;
  const int heads = a.nq + a.nkv + (a.vc.p ? a.nkv : 0);
  const int64_t unit = (int64_t)blockIdx.x * PER + threadIdx.x / L;
  const int l = (int)(threadIdx.x % L);
  const bool live = unit < a.num_tokens * heads;
  const int64_t t = live ? unit / heads : 0;
  const int h = live ? (int)(unit - t * heads) : 0;

  int64_t slot = -1;
  if (a.slots && h >= a.nq) {
    slot = a.slots[t];
    if (slot >= (int64_t)a.num_blocks * a.block_size) slot = -1;
  }
  const int64_t block = slot < 0 ? 0 : slot / a.block_size;
  const int64_t in_block = slot < 0 ? 0 : slot - block * a.block_size;

  if (h >= a.nq + a.nkv) {                       // a value head: copied
    if (live && slot >= 0) {
      const int hv = h - a.nq - a.nkv;
      const uint16_t* p = (const uint16_t*)a.v + t * a.v_rs + (int64_t)hv * HD + l * 8;
      uint16_t* d = (uint16_t*)a.vc.p + block * a.vc.block_s + in_block * a.vc.token_s +
                    (int64_t)hv * a.vc.head_s + l * 8;
      *(uint2*)d = *(const uint2*)p;
      *(uint2*)(d + 4) = *(const uint2*)(p + 4);
    }
    return;                                      // whole heads leave: sums stay within a head
  }
  const bool is_q = h < a.nq;
  const int hh = is_q ? h : h - a.nq;
  const uint16_t* src = is_q ? (const uint16_t*)a.q + t * a.q_rs + (int64_t)hh * HD
                             : (const uint16_t*)a.k + t * a.k_rs + (int64_t)hh * HD;
  // the lane's two runs of four values
  const int half = a.rot / 2;
  const bool turns = l * 8 < a.rot;
  const int d0 = turns && !a.interleaved ? l * 4 : l * 8;
  const int d1 = turns && !a.interleaved ? half + l * 4 : l * 8 + 4;
  float x[8];
  unpack4(*(const uint2*)(src + d0), x);
  unpack4(*(const uint2*)(src + d1), x + 4);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  const float inv = rsqrtf(head_sum<L>(ss) * (1.f / HD) + a.eps);
  const uint16_t* wp = (const uint16_t*)(is_q ? a.q_w : a.k_w);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= inv;
  if (wp) {
    float wv[8];
    unpack4(*(const uint2*)(wp + d0), wv);
    unpack4(*(const uint2*)(wp + d1), wv + 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= wv[e];
  }
  if (turns) {
    int64_t pos = a.positions[t];
    pos = pos < 0 ? 0 : (pos >= a.max_pos ? a.max_pos - 1 : pos);
    float cs[4], sn[4];
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
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x1 = x[2 * e], x2 = x[2 * e + 1];
        x[2 * e] = x1 * cs[e] - x2 * sn[e];
        x[2 * e + 1] = x2 * cs[e] + x1 * sn[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x1 = x[e], x2 = x[4 + e];
        x[e] = x1 * cs[e] - x2 * sn[e];
        x[4 + e] = x2 * cs[e] + x1 * sn[e];
      }
    }
  }
  if (!live) return;
  const uint2 y0 = pack4(x), y1 = pack4(x + 4);
  if (is_q || a.k_out) {
    uint16_t* d = is_q ? (uint16_t*)a.q_out + t * a.qo_rs + (int64_t)hh * HD
                       : (uint16_t*)a.k_out + t * a.ko_rs + (int64_t)hh * HD;
    *(uint2*)(d + d0) = y0;
    *(uint2*)(d + d1) = y1;
  }
  if (!is_q && slot >= 0 && a.kc.p) {
    uint16_t* d = (uint16_t*)a.kc.p + block * a.kc.block_s + in_block * a.kc.token_s +
                  (int64_t)hh * a.kc.head_s;
    *(uint2*)(d + d0) = y0;
    *(uint2*)(d + d1) = y1;
  }
}

namespace {
template <int HD>
hipError_t launch_hd(const QkNormArgs& a, hipStream_t s) {
  const int64_t heads = a.nq + a.nkv + (a.vc.p ? a.nkv : 0);
  constexpr int PER = kBlock / (HD / 8);
  const int64_t grid = (a.num_tokens * heads + PER - 1) / PER;
  if (grid > 0x7FFFFFFFLL) return hipErrorNotSupported;
  hipLaunchKernelGGL((qk_norm_rope<HD>), dim3((unsigned)grid), dim3(kBlock), 0, s, a);
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
