// Shared by the kernels of the 8-bit key / value cache: requests and their rows,
// the scale rule, and the addresses of a (block, head).
#pragma once

#include "csa_device.cuh"

namespace csa {

constexpr float kKv8MinScale = 7.888609052210118e-31f;  // 2^-100

// Rows [r0, r1) of request b sit at positions cached .. cached + (r1 - r0) - 1.
struct Kv8Req {
  int32_t r0, r1, cached;
  __device__ __forceinline__ int32_t rows() const { return r1 - r0; }
  __device__ __forceinline__ int32_t len() const { return cached + (r1 - r0); }  // tokens in the cache
};

// Request b, or false (and the error word set) where its rows or tokens are out
// of bounds.
__device__ __forceinline__ bool kv8_request(const int32_t* row_start, const int32_t* cached, int b, int32_t n_rows,
                                            const csa_block_table& bt, int32_t rows_per_block, Kv8Req& r,
                                            int32_t* err) {
  r.r0 = row_start[b];
  r.r1 = row_start[b + 1];
  r.cached = cached[b];
  const bool ok = r.r0 >= 0 && r.r1 >= r.r0 && r.r1 <= n_rows && r.cached >= 0 &&
                  (int64_t)r.cached + (r.r1 - r.r0) <= min((int64_t)bt.stride * rows_per_block, (int64_t)INT32_MAX);
  if (!ok) record_error(err, CSA_ERR_DEVICE_BOUNDS);
  return ok;
}

// Physical block of logical block lb of request b (lb within the table), or -1.
__device__ __forceinline__ int32_t kv8_block(const csa_block_table& bt, int32_t num_blocks, int b, int32_t lb) {
  const int32_t id = bt.table[(int64_t)b * bt.stride + lb];
  return id >= 0 && id < num_blocks ? id : -1;
}

// The last b in [0, n) with key(b) <= x, for a non-decreasing key with key(0) <= x;
// all 32 lanes of a warp search together, 32 probes a round.
template <typename F>
__device__ __forceinline__ int warp_last_le(int n, int64_t x, F key) {
  int lo = 0;
  const int lane = threadIdx.x & 31;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && key(lo + at) <= x;  // a prefix of the lanes
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

}  // namespace csa
