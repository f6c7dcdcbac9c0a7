// Reading a quantised cache back: tokens of requests, by their pages, as bf16 rows.
//
//   row starts[r] + t  =  code * 2^(byte - 127) of token first[r] + t of request r
//
// exact in bf16's range, as four significant bits and a power of two fit bf16. A thread takes 16
// codes of a key row and of the value row at once: one 16-byte load each, two
// stores. Bound by bytes: 1 + 1/head_dim read and 2 written per value. 8 requests of up
// to 262,143 tokens, 4 heads x 128, 806 MB: 151 us (5.3 TB/s; the loads alone 48, the
// stores alone 101). One turn of its threads to a workgroup: two took 171, four 177,
// eight 184, with or without several turns' loads together; then streaming loads and
// stores (164 without). 300 tokens: 3.4 us.
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
// of them.
__global__ __launch_bounds__(kBlock) void cache_read_fp8(CacheReadArgs a, int per_row, int per) {
  const int64_t row_lo = (int64_t)blockIdx.x * per;
  const int64_t row_hi = min(row_lo + per, a.num_rows);
  if (row_hi <= a.starts[0]) return;
  // the request of the workgroup's first row; each thread goes on from there
  int r = request_of(a.starts, a.batch, max(row_lo, (int64_t)a.starts[0]));
  const int items = (int)(row_hi - row_lo) * per_row;
  const int per_head = a.hd / 16;
  for (int i = (int)threadIdx.x; i < items; i += kBlock) {
    const int in_row = i / per_row, c = i - in_row * per_row;
    const int64_t row = row_lo + in_row;
    while (r < a.batch && row >= a.starts[r + 1]) ++r;
    if (r >= a.batch) return;                  // behind the last request
    if (row < a.starts[r]) continue;
    const int head = c / per_head, d = (c - head * per_head) * 16;
    const int64_t t = row - a.starts[r] + (a.first ? a.first[r] : 0);   // below 2^32
    const uint32_t b = (uint32_t)t / (uint32_t)a.block_size;
    int page = -1;
    if (t >= 0 && b < (uint32_t)a.max_blocks) page = a.table[(int64_t)r * a.table_rs + b];
    u32x4 k = {0, 0, 0, 0}, v = k;             // a page outside the cache reads as zeros
    int kb = 127, vb = 127;
    if (page >= 0 && page < a.num_blocks) {
      const uint32_t in = (uint32_t)t - b * (uint32_t)a.block_size;
      k = ld16_stream((const uint8_t*)a.kc.p + page * a.kc.block_s + in * a.kc.token_s + head * a.kc.head_s + d);
      v = ld16_stream((const uint8_t*)a.vc.p + page * a.vc.block_s + in * a.vc.token_s + head * a.vc.head_s + d);
      kb = a.kc.scale[page * a.kc.scale_block_s + head * a.kc.scale_head_s + in];
      vb = a.vc.scale[page * a.vc.scale_block_s + head * a.vc.scale_head_s + in];
    }
    uint16_t* ko = (uint16_t*)a.k_out + row * a.k_rs + (int64_t)c * 16;
    uint16_t* vo = (uint16_t*)a.v_out + row * a.v_rs + (int64_t)c * 16;
    u32x4 y[2];
    fp8_to_bf16_scaled(k, kb, y);
    st16_stream(ko, y[0]);
    st16_stream(ko + 8, y[1]);
    fp8_to_bf16_scaled(v, vb, y);
    st16_stream(vo, y[0]);
    st16_stream(vo + 8, y[1]);
  }
}

hipError_t launch_cache_read_fp8(const CacheReadArgs& a, hipStream_t s) {
  const int per_row = a.nkv * a.hd / 16;
  const int per = std::max(1, kBlock / per_row);     // rows of a workgroup
  const int64_t blocks = (a.num_rows + per - 1) / per;
  if (blocks > 0x7FFFFFFFLL) return hipErrorNotSupported;
  hipLaunchKernelGGL(cache_read_fp8, dim3((unsigned)blocks), dim3(kBlock), 0, s, a, per_row, per);
  return hipGetLastError();
}

}  // namespace sc
