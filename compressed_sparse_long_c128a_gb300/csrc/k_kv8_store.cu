// Insert into the 8-bit key / value cache: one scale for each block of tokens and head.
//
// A block's scale is the largest of what it was and amax / 448 over its new rows, so a
// (request, block, head, key or value) is one unit of work: one CTA reads the unit's rows
// once (copies in shared memory last from amax to the codes; what does not fit there is
// read again), rounds the block's older rows again in the rare case that the scale rose,
// and no two CTAs meet at a scale.
// HBM bounds it: 2 or 4 bytes in and 1 byte out a value.  16384 bf16 rows of 8 heads of 128
// take 24.5 us in a graph, 4.1 TB/s; what is left is that a unit's codes wait for its maximum.
// 64 single tokens take 4.4 us: the launch and a chain of four dependent reads.
//
// Units are found without a list.  With f(b) = row_start[b] / P + b, request b owns the
// units x in [f(b), f(b+1)): there are n_rows / P + num_seqs, whatever the lengths are.  A
// request of n rows owns at least n / P + 1 of them and touches at most one block more,
// which the owner of its first block takes too.

#include <algorithm>

#include "csa_kernels.h"
#include "kv8.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace {

// Threads of a unit and the most bytes of it that stay in shared memory, with the registers
// held to what six CTAs of 256 threads (five, fp32) can have; the rest is read again, from L2.
// 16384 rows, 8 heads of 128, in a graph, by this rule and otherwise:
//  * a few rows, or blocks of few: 64 threads, 4 KB (blocks of 16: 26.6 us; 31.8 with the
//    80 registers that the compiler takes by itself);
//  * up to 32 KB: 128 threads, 24 KB (bf16, blocks of 64: 24.4 us; 28.9 with 256 threads);
//  * more: 256 threads, 16 KB of bf16 (blocks of 256: 24.5 us; 28.1 with all 64 KB, as only
//    three CTAs fit an SM then) and 64 KB of fp32 (47.8 us; 52.3 with 16).
constexpr int kFewThreads = 64, kMidThreads = 128, kBigThreads = 256;
constexpr int kFewBytes = 4096, kMidBytes = 24576, kMostBytes = 65536, kMostBytesBf16 = 16384;

// 16 values as they are stored.
template <typename T>
struct Raw {
  uint32_t w[4 * sizeof(T)];
};

template <typename T>
__device__ __forceinline__ Raw<T> load16(const T* p, bool vec) {
  Raw<T> r;
  if (vec) {
#pragma unroll
    for (int j = 0; j < (int)sizeof(T); ++j) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p) + j);
      r.w[4 * j] = x.x, r.w[4 * j + 1] = x.y, r.w[4 * j + 2] = x.z, r.w[4 * j + 3] = x.w;
    }
  } else if constexpr (sizeof(T) == 2) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = (uint32_t)h[2 * j] | (uint32_t)h[2 * j + 1] << 16;
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) r.w[j] = reinterpret_cast<const uint32_t*>(p)[j];
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void values(const Raw<T>& r, float* v) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r.w[i]);
  }
}

// The largest magnitude of 16 values, as the bits of a float.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const Raw<T>& r) {
  uint32_t m = 0;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
    return max(m << 16, m & 0x7fff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, r.w[i] & 0x7fffffffu);
    return m;
  }
}

// Block-wide maximum; red: a word for each warp.
__device__ __forceinline__ uint32_t block_top(uint32_t v, uint32_t* red) {
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < nw ? red[lane] : 0u);
}

__device__ __forceinline__ uint4 pack16(const float* v, float mul) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (uint32_t)f32x2_to_e4m3x2(v[4 * i] * mul, v[4 * i + 1] * mul) |
           (uint32_t)f32x2_to_e4m3x2(v[4 * i + 2] * mul, v[4 * i + 3] * mul) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == kBigThreads ? (sizeof(T) == 2 ? 6 : 5) : 1280 / kThreads)
    kv8_store_kernel(const Kv8StoreArgs a, const int room) {
  extern __shared__ __align__(16) uint8_t buf[];
  __shared__ uint32_t red[32];
  __shared__ int owner;
  pdl_trigger();
  pdl_wait();
  const int B = a.bt.num_seqs, P = a.cache.rows_per_block, Hk = a.cache.kv_heads, D = a.cache.dim;
  // the heads' keys and values of one stretch of rows run together: they are neighbours in memory
  const int tid = threadIdx.x, hv = blockIdx.x % (2 * Hk), h = hv % Hk;
  const int64_t x = blockIdx.x / (2 * Hk);
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
  const bool val = hv >= Hk;
  const T* src = reinterpret_cast<const T*>(a.x[val]) + (int64_t)h * D;
  const int64_t stride = a.stride[val];
  uint8_t* codes = reinterpret_cast<uint8_t*>(val ? a.cache.v : a.cache.k);
  float* scales = val ? a.cache.v_scale : a.cache.k_scale;
  const int units = D / 16;  // 16 values, one 16-byte store of codes
  const int last = (r.len() - 1) / P;
  for (int64_t lb = r.cached / P + (x - x0); lb <= last; lb += owned) {
    const int32_t p0 = max(r.cached, (int32_t)(lb * P)), p1 = (int32_t)min((int64_t)r.len(), (lb + 1) * P);
    const int old = p0 - (int32_t)(lb * P), m = p1 - p0;  // older rows, new rows
    const T* rows = src + (int64_t)(r.r0 + p0 - r.cached) * stride;
    // the thread's pieces (16 values): as many as fit are copied to shared memory and stay there
    // between the two passes, 16 bytes of all pieces next to each other
    const int kept = a.vec ? min(m * units, room) : 0;
    auto source = [&](int u) {
      const int row = (unsigned)u / (unsigned)units;
      return rows + row * stride + (u - row * units) * 16;
    };
    for (int u = tid; u < kept; u += kThreads) {
      const T* src = source(u);
#pragma unroll
      for (int j = 0; j < (int)sizeof(T); ++j)
        tc::cp_async16(tc::smem_u32(buf) + (j * room + u) * 16, reinterpret_cast<const uint4*>(src) + j, 16);
    }
    tc::cp_async_commit();
    // (the block is looked up while the copies are on their way)
    const int32_t blk = kv8_block(a.bt, a.cache.num_blocks, b, (int32_t)lb);
    if (blk < 0) {
      if (tid == 0) record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
      tc::cp_async_wait<0>();
      continue;
    }
    const int64_t at = (int64_t)blk * Hk + h;
    uint8_t* dst = codes + at * P * D;
    const float was = old ? scales[at] : 0.f;
    auto piece = [&](int u) {
      if (u >= kept) return load16(source(u), a.vec);
      Raw<T> r;
#pragma unroll
      for (int j = 0; j < (int)sizeof(T); ++j) {
        const uint4 x = reinterpret_cast<const uint4*>(buf)[j * room + u];
        r.w[4 * j] = x.x, r.w[4 * j + 1] = x.y, r.w[4 * j + 2] = x.z, r.w[4 * j + 3] = x.w;
      }
      return r;
    };
    tc::cp_async_wait<0>();  // a thread reads its own copies alone
    // magnitudes order as their bits do; a NaN or an infinity lies at or above kInf
    constexpr uint32_t kInf = 0x7f800000u;
    uint32_t most = 0;
    for (int u = tid; u < m * units; u += kThreads) most = max(most, top_bits(piece(u)));
    most = block_top(most, red);
    const bool odd = most >= kInf;
    if (odd) {  // the largest finite one
      if (tid == 0) record_error(a.err, CSA_ERR_NONFINITE);
      most = 0;
      for (int u = tid; u < m * units; u += kThreads) {
        float v[16];
        values(piece(u), v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t y = __float_as_uint(v[i]) & 0x7fffffffu;
          most = y < kInf ? max(most, y) : most;
        }
      }
      most = block_top(most, red);
    }
    const float top = __uint_as_float(most);
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
    uint4* to = reinterpret_cast<uint4*>(dst) + (int64_t)old * units;
    if (!odd) {
      for (int u = tid; u < m * units; u += kThreads) {
        float v[16];
        values(piece(u), v);
        to[u] = pack16(v, inv);
      }
    } else {
      for (int u = tid; u < m * units; u += kThreads) {
        float v[16];
        values(piece(u), v);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] == v[i] ? v[i] : 0.f;
        to[u] = pack16(v, inv);
      }
    }
    if (tid == 0) scales[at] = scale;  // every thread has read it: block_top synchronises
  }
}

template <typename T>
int64_t unit_bytes(const Kv8StoreArgs& a) {
  return (int64_t)a.cache.rows_per_block * a.cache.dim * sizeof(T);
}

template <typename T, int kThreads>
cudaError_t launch(const Kv8StoreArgs& a, int32_t most_bytes, cudaStream_t s) {
  static PerDevice attr;
  const cudaError_t e = with_device_slot(attr, [](int, int64_t& v) {
    if (v) return cudaSuccess;
    const cudaError_t err = cudaFuncSetAttribute(kv8_store_kernel<T, kThreads>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMostBytes);
    if (err == cudaSuccess) v = 1;
    return err;
  });
  if (e != cudaSuccess) return e;
  const unsigned gx = (unsigned)(a.n_rows / a.cache.rows_per_block + a.bt.num_seqs);
  const int32_t bytes = (int32_t)std::min((int64_t)most_bytes, unit_bytes<T>(a));
  return launch_k(kv8_store_kernel<T, kThreads>, dim3(gx * 2 * a.cache.kv_heads), dim3(kThreads), bytes, s, 0, a,
                  bytes / (16 * (int)sizeof(T)));
}

template <typename T>
cudaError_t pick(const Kv8StoreArgs& a, cudaStream_t s) {
  // rows of a unit, by the average request: up to a block's, or a step's few
  if (std::min(a.n_rows / a.bt.num_seqs, a.cache.rows_per_block) <= 16) return launch<T, kFewThreads>(a, kFewBytes, s);
  if (unit_bytes<T>(a) <= 32768) return launch<T, kMidThreads>(a, kMidBytes, s);
  return launch<T, kBigThreads>(a, sizeof(T) == 2 ? kMostBytesBf16 : kMostBytes, s);
}

}  // namespace

cudaError_t launch_kv8_store(const Kv8StoreArgs& a, cudaStream_t s) {
  return a.in_dtype == CSA_F32 ? pick<float>(a, s) : pick<__nv_bfloat16>(a, s);
}

}  // namespace csa
