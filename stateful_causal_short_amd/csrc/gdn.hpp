// Gated delta rule argument block and launchers, shared by gdn.hip,
// gdn_prefill.hip and abi.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sc {

constexpr int kGdnChunk = 64;   // tokens per chunk of the prefill

// Gated delta rule launch arguments (by value into the kernels).
struct GdnArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* a;
  const void* b;
  const float* A_log;
  const float* dt_bias;
  void* out;
  float* pool;
  const int32_t* qsl;        // prefill: request bounds
  const int32_t* slots;
  const uint8_t* has_init;   // nullable for updates (all continue their state)
  const int32_t* num_acc;    // speculative update: accepted counts, else nullptr
  char* ws;                  // prefill: chunk matrices (see GdnWorkspace)
  int64_t q_rs, k_rs, v_rs, a_rs, b_rs, out_rs, slot_stride;   // elements
  int64_t num_tokens;
  float scale;
  int32_t hk, hv, dk, dv, l2norm, gate_f32, num_slots, batch;
  int32_t nq;                // update: tokens per request
  int32_t n_chunks;          // prefill: chunk slots of the workspace
  int32_t sorted;            // prefill: the scan takes requests in the workspace's order
};

// Prefill workspace: for each (chunk, value head) the matrices T and P of the
// chunk as MFMA operands (16-bit parts, 3 of T and 2 of P), and its row
// factors; for each (chunk, key head) the keys transposed; last, the requests by
// falling length.
struct GdnWorkspace {
  static constexpr int64_t kFrag = 1024;             // 64 lanes x 16 bytes
  static constexpr int64_t kFrags = 6;               // (row tile, k step) pairs at or below the diagonal
  static constexpr int64_t kT = kFrags * 3 * kFrag;
  static constexpr int64_t kP = kFrags * 2 * kFrag;
  static constexpr int64_t kDecay = 3 * kGdnChunk * 4;
  static constexpr int64_t kVec = 4 * kGdnChunk * 4; // three row factors, the chunk's decay
  static constexpr int64_t kHead = kT + kP + kVec;
  __host__ __device__ static int64_t order(int64_t n_chunks, int64_t hk, int64_t hv, int64_t dk) {
    return n_chunks * (hv * kHead + hk * dk * kGdnChunk * 2);
  }
  static int64_t bytes(int64_t n_chunks, int64_t hk, int64_t hv, int64_t dk, int64_t batch) {
    return order(n_chunks, hk, hv, dk) + batch * 4;
  }
};

// Whether the grids of a prefill can be launched (and its workspace counted).
bool gdn_prefill_fits(int64_t n_chunks, int64_t batch, int64_t hk, int64_t hv, int64_t dv);

hipError_t launch_gdn_update(const GdnArgs& a, hipStream_t stream);
hipError_t launch_gdn_prefill(const GdnArgs& a, hipStream_t stream);

}  // namespace sc
