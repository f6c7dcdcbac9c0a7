// Device helpers of the gated delta rule kernels: the gates, sums over 16
// lanes, and bf16 parts of fp32 values.
#pragma once

#include "common.hpp"
#include "gdn.hpp"

namespace sc {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kL2Eps = 1e-6f;

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
  f32x2 p = {f, 0.f};
  return (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
}

__device__ __forceinline__ float gate_at(const void* p, int64_t i, int f32) {
  return f32 ? ((const float*)p)[i] : bf16_at(p, i);
}

// Log decay g = -exp(A_log) softplus(a + dt_bias) (<= 0).
__device__ __forceinline__ float gdn_log_decay(const GdnArgs& a, int64_t row, int h) {
  const float x = gate_at(a.a, row * a.a_rs + h, a.gate_f32) + a.dt_bias[h];
  const float sp = x > 20.f ? x : log1pf(expf(x));   // beyond 20 they agree to fp32
  return -expf(a.A_log[h]) * sp;
}

__device__ __forceinline__ float gdn_beta(const GdnArgs& a, int64_t row, int h) {
  return 1.f / (1.f + expf(-gate_at(a.b, row * a.b_rs + h, a.gate_f32)));
}

// Sum over the 16 lanes of a row (every lane gets it): four rotations.
__device__ __forceinline__ float row16_sum(float x) {
#define SC_ROR_ADD(n)                                                                     \
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + n, 0xF, \
                                                  0xF, true))
  SC_ROR_ADD(8);
  SC_ROR_ADD(4);
  SC_ROR_ADD(2);
  SC_ROR_ADD(1);
#undef SC_ROR_ADD
  return x;
}

}  // namespace sc
