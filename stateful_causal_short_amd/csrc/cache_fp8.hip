// Reading a quantised cache back: tokens of requests, by their pages, as bf16 rows.
//
//   row starts[r] + t  =  code * 2^(byte - 127) of token first[r] + t of request r
//
// exact, as four significant bits and a power of two fit bf16. A thread takes 16
// codes of a key row and of the value row at once: one 16-byte load each, two
// stores. Bound by bytes: 1 + 1/head_dim read and 2 written per value.
#include "attn_device.hpp"
#include "fp8_device.hpp"

#include <algorithm>

namespace sc {

namespace {

// The last request that begins at or before `row` (starts[0] <= row), a wave looking
// at 64 evenly spaced entries, then at those between two of them, and so on.
__device__ __forceinline__ int request_of(const int32_t* starts, int batch, int64_t row) {
  const int lane = (int)(threadIdx.x & 63);
  int lo = 0, n = batch;              // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int at = lo + lane * step;
    const int in = __popcll(__ballot(lane * step < n && starts[at] <= row));
    lo += (max(in, 1) - 1) * step;
    n = min(step, batch - lo);
  }
  return lo;
}

}  // namespace

// Rows [blockIdx.x * per, ...) of the output; a thread per 16 values of a row, `per_row`
// of them, several rows at a time.
__global__ __launch_bounds__(kBlock) void cache_read_fp8(CacheReadArgs a, int per_row, int per) {
  const int64_t row_lo = (int64_t)blockIdx.x * per;
  const int64_t row_hi = min(row_lo + per, a.num_rows);
  if (row_hi <= a.starts[0]) return;
  // the request of the workgroup's first row; each thread goes on from there
  int r = request_of(a.starts, a.batch, max(row_lo, (int64_t)a.starts[0]));
  const int items = (int)(row_hi - row_lo) * per_row;
  for (int i = (int)threadIdx.x; i < items; i += kBlock) {
    const int in_row = i / per_row, c = i - in_row * per_row;
    const int64_t row = row_lo + in_row;
    while (r < a.batch && row >= a.starts[r + 1]) ++r;
    if (r >= a.batch) return;                  // behind the last request
    if (row < a.starts[r]) continue;
    const int head = c / (a.hd / 16), d = (c - head * (a.hd / 16)) * 16;
    const int64_t t = row - a.starts[r] + (a.first ? a.first[r] : 0);
    const int64_t b = t / a.block_size;
    int page = -1;
    if (t >= 0 && b < a.max_blocks) page = a.table[(int64_t)r * a.table_rs + b];
    u32x4 k = {0, 0, 0, 0}, v = k;             // a page outside the cache reads as zeros
    int kb = 0, vb = 0;
    if (page >= 0 && page < a.num_blocks) {
      const int64_t in = t - b * a.block_size;
      k = ld16((const uint8_t*)a.kc.p + page * a.kc.block_s + in * a.kc.token_s + head * a.kc.head_s + d);
      v = ld16((const uint8_t*)a.vc.p + page * a.vc.block_s + in * a.vc.token_s + head * a.vc.head_s + d);
      kb = a.kc.scale[page * a.kc.scale_block_s + head * a.kc.scale_head_s + in];
      vb = a.vc.scale[page * a.vc.scale_block_s + head * a.vc.scale_head_s + in];
    }
    uint16_t* ko = (uint16_t*)a.k_out + row * a.k_rs + (int64_t)c * 16;
    uint16_t* vo = (uint16_t*)a.v_out + row * a.v_rs + (int64_t)c * 16;
    u32x4 y[2];
    fp8_to_bf16_scaled(k, kb, y);
    st16(ko, y[0]);
    st16(ko + 8, y[1]);
    fp8_to_bf16_scaled(v, vb, y);
    st16(vo, y[0]);
    st16(vo + 8, y[1]);
  }
}

hipError_t launch_cache_read_fp8(const CacheReadArgs& a, hipStream_t s) {
  const int per_row = a.nkv * a.hd / 16;
  // a workgroup's rows: eight turns of its threads where there are that many
  // workgroups for every CU, else one
  const int64_t items = a.num_rows * per_row;
  const int64_t turns = std::clamp<int64_t>(items / kBlock / (8 * device_cus()), 1, 8);
  const int64_t per = std::max<int64_t>(1, turns * kBlock / per_row);
  const int64_t blocks = (a.num_rows + per - 1) / per;
  if (blocks > 0x7FFFFFFFLL) return hipErrorNotSupported;
  hipLaunchKernelGGL(cache_read_fp8, dim3((unsigned)blocks), dim3(kBlock), 0, s, a, per_row, (int)per);
  return hipGetLastError();
}

}  // namespace sc
