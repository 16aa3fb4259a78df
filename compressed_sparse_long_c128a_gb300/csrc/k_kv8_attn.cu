// Attention over the 8-bit key / value cache on the CUDA cores, everything in fp32: for
// fp32 queries or results, whose products the tensor cores would round.
//
// One CTA holds one row's query heads of one key head (eight at a time), walks the
// keys the row sees in tiles of 32, and keeps one running maximum and sum a head:
// the codes of a tile become fp32 in shared memory, a lane scores a key, a thread
// accumulates a dim.  A head of D dims costs 2 D FMAs a key and the CUDA cores'
// FMA and shared-memory rates bound it; as it stands each tile is a chain of four barriers
// (ncu on a ragged fp32 batch: 44 % of the issue slots, fma pipe 17 %; 57 us in a graph).
// With few rows a row's tiles are split over up to 32 CTAs and joined by a second kernel.

#include <cfloat>

#include "csa_kernels.h"
#include "kv8.cuh"

namespace csa {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;   // keys
constexpr int kHeads = 8;   // query heads of a CTA
constexpr int kMaxDim = 256;
constexpr int kDimsPerThread = kMaxDim / kThreads;

__host__ __device__ constexpr int simt_smem_floats(int D) { return 2 * kTile * (D + 4) + kHeads * D + 2 * kHeads * kTile + 2 * kHeads; }

__global__ void __launch_bounds__(kThreads, 4) kv8_attn_simt_kernel(const Kv8AttnArgs a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int owner;
  pdl_trigger();
  pdl_wait();
  const int D = a.cache.dim, P = a.cache.rows_per_block, Hk = a.cache.kv_heads, G = a.group;
  const int LD = D + 4;
  float* sK = sm;                    // [32][D + 4]
  float* sV = sK + kTile * LD;       // [32][D + 4]
  float* sQ = sV + kTile * LD;       // [8][D], times the scale
  float* sP = sQ + kHeads * D;       // [8][32]
  float* sAlpha = sP + kHeads * kTile;  // [8]
  float* sL = sAlpha + kHeads;       // [8]
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int row = blockIdx.x, chunks = (G + kHeads - 1) / kHeads;
  const int kvh = blockIdx.y / chunks, g0 = (blockIdx.y % chunks) * kHeads, ng = min(kHeads, G - g0);
  const int h0 = kvh * G + g0, split = blockIdx.z, S = a.n_splits;
  if (tid < 32) {
    const int b = warp_last_le(a.bt.num_seqs, row, [&](int i) { return (int64_t)a.row_start[i]; });
    if (lane == 0) owner = b;
  }
  __syncthreads();
  const int b = owner;
  Kv8Req r;
  const bool ok = kv8_request(a.row_start, a.cached, b, a.n_rows, a.bt, P, r, a.err);
  if (!ok || row < r.r0 || row >= r.r1) return;  // padding, or a request that is out of bounds
  if (r.rows() > a.max_new) {
    if (tid == 0) record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
    return;
  }
  const int p = r.cached + (row - r.r0), n = r.len();
  const int first = a.mask.first ? max(0, a.mask.first[row]) : 0;
  const int pre = a.mask.prefix ? min(a.mask.prefix[b], n) : 0;
  const int lo = a.mask.window > 0 ? max(first, p - a.mask.window + 1) : first;
  // tiles of the prefix, then those of the window that are not among them
  const int tA = first / kTile, nA = first < pre ? (pre + kTile - 1) / kTile - tA : 0;
  const int tB = nA ? max(lo / kTile, tA + nA) : lo / kTile, nB = lo <= p ? max(0, p / kTile + 1 - tB) : 0;
  const int nt = nA + nB, t0 = (int)((int64_t)nt * split / S), t1 = (int)((int64_t)nt * (split + 1) / S);

  for (int u = tid; u < ng * D; u += kThreads)
    sQ[u] = load_elem(a.q, a.q_dtype, (int64_t)row * a.q_stride + (int64_t)(h0 + u / D) * D + u % D) * a.mask.scale;

  float o[kHeads][kDimsPerThread];
#pragma unroll
  for (int g = 0; g < kHeads; ++g)
#pragma unroll
    for (int j = 0; j < kDimsPerThread; ++j) o[g][j] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // of heads wid and wid + 4, the same in every lane
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.cache.k);
  const uint8_t* vc = reinterpret_cast<const uint8_t*>(a.cache.v);
  const int units = D / 16, shift = 31 - __clz(P);

  // a tile's codes and scales wait in registers while the tile before it is worked on
  constexpr int kMaxUnits = 2 * kTile * (kMaxDim / 16) / kThreads;
  uint4 code[kMaxUnits];
  float scl[kMaxUnits];
  auto tile_base = [&](int ti) { return (ti < nA ? tA + ti : tB + ti - nA) * kTile; };
  auto fetch = [&](int ti) {
    const int base = tile_base(ti);
#pragma unroll
    for (int i = 0; i < kMaxUnits; ++i) {
      const int u = tid + i * kThreads;
      if (u >= 2 * kTile * units) break;
      const bool val = u >= kTile * units;
      const int w = val ? u - kTile * units : u, j = (unsigned)w / (unsigned)units, t = base + j;
      code[i] = make_uint4(0, 0, 0, 0);
      scl[i] = 0.f;
      if (t < n) {
        const int32_t blk = kv8_block(a.bt, a.cache.num_blocks, b, t >> shift);
        if (blk >= 0) {
          const int64_t at = (int64_t)blk * Hk + kvh;
          code[i] = __ldg(reinterpret_cast<const uint4*>((val ? vc : kc) + (at * P + (t & (P - 1))) * D) + (w - j * units));
          scl[i] = (val ? a.cache.v_scale : a.cache.k_scale)[at];
        }
      }
    }
  };
  if (t0 < t1) fetch(t0);
  for (int ti = t0; ti < t1; ++ti) {
    const int base = tile_base(ti);
    __syncthreads();
    // codes to fp32, keys and values; tokens that are not there are zeros
#pragma unroll
    for (int i = 0; i < kMaxUnits; ++i) {
      const int u = tid + i * kThreads;
      if (u >= 2 * kTile * units) break;
      const bool val = u >= kTile * units;
      const int w = val ? u - kTile * units : u, j = (unsigned)w / (unsigned)units;
      const uint32_t k[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
      const float sc = scl[i];
      float* dst = (val ? sV : sK) + j * LD + (w - j * units) * 16;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 c0 = e4m3x2_to_f32x2(k[x] & 0xffffu), c1 = e4m3x2_to_f32x2(k[x] >> 16);
        *reinterpret_cast<float4*>(dst + 4 * x) = make_float4(c0.x * sc, c0.y * sc, c1.x * sc, c1.y * sc);
      }
    }
    if (ti + 1 < t1) fetch(ti + 1);
    __syncthreads();
    // scores and softmax: warp w takes heads w and w + 4, a lane a key
    const int t = base + lane;
    bool see = t < n && t >= first && (t < pre || (t <= p && t >= lo));
    if (see && kv8_block(a.bt, a.cache.num_blocks, b, t >> shift) < 0) {
      record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
      see = false;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = wid + 4 * j;
      if (g >= ng) break;
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
      const float4* kq = reinterpret_cast<const float4*>(sK + lane * LD);
      const float4* qq = reinterpret_cast<const float4*>(sQ + g * D);
      for (int d = 0; d < D / 4; ++d) {
        const float4 x = kq[d], y = qq[d];
        s0 = fmaf(x.x, y.x, s0), s1 = fmaf(x.y, y.y, s1), s2 = fmaf(x.z, y.z, s2), s3 = fmaf(x.w, y.w, s3);
      }
      float s = (s0 + s1) + (s2 + s3);
      if (a.mask.softcap > 0.f) s = a.mask.softcap * tanhf(s / a.mask.softcap);
      if (a.mask.slopes) s -= a.mask.slopes[h0 + g] * fabsf((float)(p - t));
      s = see ? s : -INFINITY;
      // a NaN score stays: it makes the row NaN, as its definition does
      const bool nan = __any_sync(0xffffffffu, s != s);
      const float mt = fmaxf(m[j], warp_max(s));
      const float ref = mt == -INFINITY ? 0.f : mt;
      const float e = expf(s - ref), alpha = expf(m[j] - ref);
      l[j] = l[j] * alpha + warp_sum(e);
      m[j] = nan ? NAN : mt;
      sP[g * kTile + lane] = e;
      if (lane == 0) sAlpha[g] = alpha;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kDimsPerThread; ++j) {
      const int d = tid + j * kThreads;
      if (d >= D) break;
#pragma unroll
      for (int g = 0; g < kHeads; ++g) o[g][j] *= g < ng ? sAlpha[g] : 0.f;
      for (int k = 0; k < kTile; k += 4) {
        const float v0 = sV[k * LD + d], v1 = sV[(k + 1) * LD + d], v2 = sV[(k + 2) * LD + d], v3 = sV[(k + 3) * LD + d];
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
          if (g >= ng) break;
          const float4 e = *reinterpret_cast<const float4*>(sP + g * kTile + k);
          o[g][j] = fmaf(e.x, v0, fmaf(e.y, v1, fmaf(e.z, v2, fmaf(e.w, v3, o[g][j]))));
        }
      }
    }
  }
  __syncthreads();
  // sAlpha: the maxima, sL: the sums
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (lane == 0 && wid + 4 * j < ng) sAlpha[wid + 4 * j] = m[j], sL[wid + 4 * j] = l[j];
  __syncthreads();
  const int64_t rh = (int64_t)row * a.heads + h0;
  if (S > 1) {
#pragma unroll
    for (int g = 0; g < kHeads; ++g) {
      if (g >= ng) break;
      const int64_t at = (rh + g) * S + split;
#pragma unroll
      for (int j = 0; j < kDimsPerThread; ++j)
        if (tid + j * kThreads < D) a.part_o[at * D + tid + j * kThreads] = o[g][j];
      if (tid == 0) a.part_ml[2 * at] = sAlpha[g], a.part_ml[2 * at + 1] = sL[g];
    }
    return;
  }
#pragma unroll
  for (int g = 0; g < kHeads; ++g) {
    if (g >= ng) break;
    const float inv = sL[g] == 0.f ? 0.f : 1.0f / sL[g];
#pragma unroll
    for (int j = 0; j < kDimsPerThread; ++j) {
      const int d = tid + j * kThreads;
      if (d >= D) break;
      const float y = o[g][j] * inv;
      if (a.out_dtype == CSA_F32) reinterpret_cast<float*>(a.out)[(rh + g) * D + d] = y;
      else reinterpret_cast<uint16_t*>(a.out)[(rh + g) * D + d] = f32_to_bf16(y);
    }
    if (a.lse && tid == 0) a.lse[rh + g] = sAlpha[g] + logf(sL[g]);  // -inf where nothing is seen
  }
}

// Joins the splits of a row and head; a row that no request owns stays as it is.
__global__ void __launch_bounds__(kThreads) kv8_simt_join_kernel(const Kv8AttnArgs a) {
  __shared__ int owner;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, h = blockIdx.y, S = a.n_splits, D = a.cache.dim;
  if (threadIdx.x < 32) {
    const int b = warp_last_le(a.bt.num_seqs, row, [&](int i) { return (int64_t)a.row_start[i]; });
    if (threadIdx.x == 0) owner = b;
  }
  __syncthreads();
  Kv8Req r;
  if (!kv8_request(a.row_start, a.cached, owner, a.n_rows, a.bt, a.cache.rows_per_block, r, a.err)) return;
  if (row < r.r0 || row >= r.r1 || r.rows() > a.max_new) return;
  const int64_t rh = (int64_t)row * a.heads + h;
  const float* ml = a.part_ml + 2 * rh * S;
  float m = -INFINITY;
  for (int s = 0; s < S; ++s) m = fmaxf(m, ml[2 * s]);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int s = 0; s < S; ++s) l += ml[2 * s + 1] * expf(ml[2 * s] - ref);  // NaN maxima: NaN
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float o = 0.f;
    for (int s = 0; s < S; ++s) o += a.part_o[(rh * S + s) * D + d] * expf(ml[2 * s] - ref);
    o *= inv;
    if (a.out_dtype == CSA_F32) reinterpret_cast<float*>(a.out)[rh * D + d] = o;
    else reinterpret_cast<uint16_t*>(a.out)[rh * D + d] = f32_to_bf16(o);
  }
  if (a.lse && threadIdx.x == 0) a.lse[rh] = ref + logf(l);
}

}  // namespace

int32_t kv8_simt_splits(int32_t n_rows, int32_t heads, int32_t kv_heads) {
  // A tile is a chain of latencies (codes, scores, softmax, sums) that four CTAs an SM only
  // half hide, so a row's keys are split until there are three times as many CTAs: 69 us
  // with one CTA a row, 57 us with four, on 111 rows of up to 740 keys.
  const int64_t ctas = (int64_t)n_rows * kv_heads * ((heads / kv_heads + kHeads - 1) / kHeads);
  const int64_t s = ctas > 0 ? 1824 / ctas : 1;
  return (int32_t)(s < 1 ? 1 : s > 32 ? 32 : s);
}

size_t kv8_simt_workspace(int32_t n_rows, int32_t heads, int32_t dim, int32_t n_splits) {
  return n_splits <= 1 ? 0 : (size_t)n_rows * heads * n_splits * (dim + 2) * sizeof(float);
}

cudaError_t launch_kv8_attn_simt(const Kv8AttnArgs& a, cudaStream_t s) {
  static PerDevice attr;
  const size_t smem = simt_smem_floats(a.cache.dim) * sizeof(float);
  const cudaError_t e = with_device_slot(attr, [](int, int64_t& v) {
    if (v) return cudaSuccess;
    const cudaError_t err = cudaFuncSetAttribute(kv8_attn_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 simt_smem_floats(kMaxDim) * sizeof(float));
    if (err == cudaSuccess) v = 1;
    return err;
  });
  if (e != cudaSuccess) return e;
  const int chunks = (a.group + kHeads - 1) / kHeads;
  const cudaError_t k = launch_k(kv8_attn_simt_kernel, dim3(a.n_rows, a.cache.kv_heads * chunks, a.n_splits),
                                 dim3(kThreads), smem, s, 0, a);
  if (k != cudaSuccess || a.n_splits <= 1) return k;
  return launch_k(kv8_simt_join_kernel, dim3(a.n_rows, a.heads), dim3(kThreads), 0, s, 0, a);
}

}  // namespace csa
