// Insert into the 8-bit key / value cache: one scale for each block of tokens and head.
//
// A block's scale is the largest of what it was and amax / 448 over its new rows, so a
// (request, block, head, key or value) is one unit of work: one CTA reads the unit's rows
// twice (amax, then the codes; the second time from L1), rounds the block's older rows
// again in the rare case that the scale rose, and no two CTAs meet at a scale.
// HBM bounds it: 2 or 4 bytes in and 1 byte out a value.
//
// Units are found without a list.  With f(b) = row_start[b] / P + b, request b owns the
// grid's x in [f(b), f(b+1)): the grid is n_rows / P + num_seqs wide, whatever the
// lengths are, a request of n rows owns at least n / P + 1 of them and touches at most one
// block more, which the owner of its first block takes too.

#include "csa_kernels.h"
#include "kv8.cuh"

namespace csa {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load16(const T* p, bool vec, float* v) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + j);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[8 * j + 2 * i] = __uint_as_float(u[i] << 16);
          v[8 * j + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(p) + j);
        v[4 * j] = w.x, v[4 * j + 1] = w.y, v[4 * j + 2] = w.z, v[4 * j + 3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (sizeof(T) == 2) v[i] = bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
      else v[i] = p[i];
    }
  }
}

__device__ __forceinline__ uint4 pack16(const float* v, float mul) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)f32x2_to_e4m3x2(v[4 * i] * mul, v[4 * i + 1] * mul) |
           (uint32_t)f32x2_to_e4m3x2(v[4 * i + 2] * mul, v[4 * i + 3] * mul) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(const Kv8StoreArgs a) {
  __shared__ float red[32];
  __shared__ int owner;
  pdl_trigger();
  pdl_wait();
  const int B = a.bt.num_seqs, P = a.cache.rows_per_block, Hk = a.cache.kv_heads, D = a.cache.dim;
  const int tid = threadIdx.x, h = blockIdx.y;
  const int64_t x = blockIdx.x;
  auto first_x = [&](int b) { return (int64_t)a.row_start[b] / P + b; };
  if (tid < 32) {
    const int b = warp_last_le(B, x, first_x);
    if (tid == 0) owner = b;
  }
  __syncthreads();
  const int b = owner;
  Kv8Req r;
  if (!kv8_request(a.row_start, a.cached, b, a.n_rows, a.bt, P, r, a.err) || r.rows() == 0) return;
  const int64_t x0 = first_x(b), owned = (int64_t)r.r1 / P + b + 1 - x0;
  if (x < x0 || x >= x0 + owned) return;
  const bool val = blockIdx.z != 0;
  const T* src = reinterpret_cast<const T*>(a.x[val]) + (int64_t)h * D;
  const int64_t stride = a.stride[val];
  uint8_t* codes = reinterpret_cast<uint8_t*>(val ? a.cache.v : a.cache.k);
  float* scales = val ? a.cache.v_scale : a.cache.k_scale;
  const int units = D / 16;  // 16 values, one 16-byte store of codes
  const int last = (r.len() - 1) / P;
  for (int64_t lb = r.cached / P + (x - x0); lb <= last; lb += owned) {
    const int32_t blk = kv8_block(a.bt, a.cache.num_blocks, b, (int32_t)lb);
    if (blk < 0) {
      if (tid == 0) record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
      continue;
    }
    const int32_t p0 = max(r.cached, (int32_t)(lb * P)), p1 = (int32_t)min((int64_t)r.len(), (lb + 1) * P);
    const int old = p0 - (int32_t)(lb * P), m = p1 - p0;  // older rows, new rows
    const T* rows = src + (int64_t)(r.r0 + p0 - r.cached) * stride;
    const int64_t at = (int64_t)blk * Hk + h;
    uint8_t* dst = codes + at * P * D;
    const float was = old ? scales[at] : 0.f;
    float top = 0.f;
    bool bad = false;
#pragma unroll 4
    for (int u = tid; u < m * units; u += kThreads) {
      const int row = u / units;
      float v[16];
      load16(rows + row * stride + (u - row * units) * 16, a.vec, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float y = fabsf(v[i]);
        const bool fin = y <= 3.402823466e38f;  // false for NaN
        bad |= !fin;
        top = fmaxf(top, fin ? y : 0.f);
      }
    }
    top = block_max(top, red);
    if (bad) record_error(a.err, CSA_ERR_NONFINITE);
    const float scale = fmaxf(fmaxf(was, top * (1.0f / 448.0f)), kKv8MinScale);
    const float inv = 1.0f / scale;
    if (old && scale > was) {
      const float ratio = was * inv;
      for (int u = tid; u < old * units; u += kThreads) {
        uint4* c = reinterpret_cast<uint4*>(dst) + u;
        const uint4 w = *c;
        const uint32_t k[4] = {w.x, w.y, w.z, w.w};
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = e4m3x2_to_f32x2(k[i >> 1] >> (16 * (i & 1)) & 0xffffu);
          v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
        *c = pack16(v, ratio);
      }
    }
#pragma unroll 2
    for (int u = tid; u < m * units; u += kThreads) {
      const int row = u / units;
      float v[16];
      load16(rows + row * stride + (u - row * units) * 16, a.vec, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] == v[i] ? v[i] : 0.f;
      reinterpret_cast<uint4*>(dst)[(int64_t)old * units + u] = pack16(v, inv);
    }
    if (tid == 0) scales[at] = scale;  // every thread has read it: block_max synchronises
  }
}

}  // namespace

cudaError_t launch_kv8_store(const Kv8StoreArgs& a, cudaStream_t s) {
  const unsigned gx = (unsigned)(a.n_rows / a.cache.rows_per_block + a.bt.num_seqs);
  const dim3 grid(gx, a.cache.kv_heads, 2);
  if (a.in_dtype == CSA_F32) return launch_k(kv8_store_kernel<float>, grid, dim3(kThreads), 0, s, 0, a);
  return launch_k(kv8_store_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, 0, a);
}

}  // namespace csa
