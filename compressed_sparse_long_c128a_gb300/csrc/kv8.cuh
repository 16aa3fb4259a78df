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

// Tiles of T tokens that some row of a request sees: those of the prefix, [tA, tA + nA),
// then those that causality and the window leave and that are not among them, [tB, tB + nB).
struct Kv8Tiles {
  int32_t tA, nA, tB, nB;
  __device__ __forceinline__ int32_t count() const { return nA + nB; }
  __device__ __forceinline__ int32_t at(int32_t i) const { return i < nA ? tA + i : tB + i - nA; }
};

// For keys t with first <= t and (t < pre or lo <= t <= hi), hi < n.
__device__ __forceinline__ Kv8Tiles kv8_tiles(int32_t T, int32_t first, int32_t pre, int32_t lo, int32_t hi) {
  Kv8Tiles x;
  x.tA = first / T;
  x.nA = first < pre ? (pre + T - 1) / T - x.tA : 0;
  x.tB = x.nA ? max(lo / T, x.tA + x.nA) : lo / T;
  x.nB = lo <= hi ? max(0, hi / T + 1 - x.tB) : 0;
  return x;
}

// Four e4m3 codes to two f16 pairs (of the low and the high 16 bits of w), exactly.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 w, x, y;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The power of two at or below x (x >= 0), kept where its reciprocal is a normal number too.
__device__ __forceinline__ float pow2_floor(float x) {
  const uint32_t e = min(max(__float_as_uint(x) >> 23, 1u), 253u);
  return __uint_as_float(e << 23);
}
__device__ __forceinline__ float pow2_recip(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) = 1 - 2 / (e^(2 x) + 1), of x 2 log2(e): about 2e-7 off, absolutely, for any x.
__device__ __forceinline__ float tanh_exp2(float x) { return fmaf(-2.0f, fast_rcp(fast_exp2(x) + 1.0f), 1.0f); }

// tanh of two numbers of at most 3/4 in magnitude: x P(x^2), P fitted to tanh(x) / x on [0, 3/4] by
// weighted least squares towards the smallest absolute error (1e-8; 7e-8 in fp32).  It needs
// the multipliers alone, which stand idle where exponentials are the limit.
constexpr float kTanhSmall = 0.75f;
__device__ __forceinline__ float2 tanh_small2(float2 x) {
  constexpr float c[6] = {0.9999998211860657f,   -0.33332470059394836f, 0.13320578634738922f,
                          -0.05314924940466881f, 0.01923721469938755f,  -0.00449344189837575f};
  const float2 s = mul2(x, x);
  float2 p = make_float2(c[5], c[5]);
#pragma unroll
  for (int i = 4; i >= 0; --i) p = fma2(p, s, make_float2(c[i], c[i]));
  return mul2(p, x);
}

}  // namespace csa
