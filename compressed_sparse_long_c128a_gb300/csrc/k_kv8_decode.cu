// Attention of few rows a request over the 8-bit key / value cache: single tokens and
// short runs of them, bf16 queries and results.  D is the head size, rounded up to 64, 128
// or 256; the dims past it are zeros that are never read or written.
//
// Every key and value is read once and meets 8 to 32 query columns (rows x query heads
// of a key head), so HBM bounds it: 2 D bytes a token and key head.  What it takes is
// loads that never pause and work that is even.  32 sequences of 32k to 64k tokens,
// 8 key heads of 128 and 8 query heads each: 500 us, 6.6 TB/s (0.97 of the measured copy); one
// of 128k: 58 us, 40 of them its bytes.  With 24 to 32 columns the issue slots bound it instead.
//
//  * The deal.  The requests' tiles of 64 tokens, laid end to end (request, key head,
//    column chunk, tile), are cut into equal shares, one a CTA, three CTAs an SM: a long
//    sequence spreads over the GPU, short ones share a CTA.  Every CTA computes the deal
//    itself from the lengths.  A share's first and last pieces may be parts of a pair
//    (request, key head, chunk); their unnormalised results go to the workspace, and a
//    second small kernel joins them in tile order.  Where the table has room for 256 tokens
//    (four tiles) at most, whole pairs are dealt and nothing is left to join: one request of
//    60 tokens takes 6.0 us against 9.2, 64 of 250 17.1 against 18.1; at 500 tokens one
//    request would take 12.1 against 8.9.
//  * Inside a CTA four warps stream alone, each 16 of a tile's tokens, through a ring of
//    its own filled by 16-byte cp.async, and meet only at a pair's end.
//  * S^T [16 tokens x 8 columns] = K [16 x D] . Q^T and O^T [D x 8] += V^T . P^T, both as
//    mma.m16n8k16 with the cache as the A operand, whose codes become f16 in registers
//    (exactly).  The tensor pipe is far from full here, and a tcgen05 tile would have to
//    take the f16 keys through shared memory, three times the bytes of the codes.
//    The order of tokens and dims inside a product is free, so each lane reads whole
//    16-byte pieces: dims 16 (t + 4 j) .. + 15 of tokens r(g), r(g) + 8 for K, and dims
//    16 g .. + 15 of tokens t, t + 4, t + 8, t + 12 for V, g = lane / 4, t = lane % 4,
//    r(g) = 4 (g & 1) + g / 2.  P^T gets from the accumulator's layout to the operand's by
//    movmatrix.
//  * Softmax: the running maximum is raised only when a score passes it by 2^8, so that
//    most steps exchange nothing between lanes.  P is rounded to f16 as
//    2^(s - m + 7) <= 2^15, which keeps 11 bits down to 2^-21 of the maximum.  Queries
//    are scaled by a power of two to [1, 2) first, so f16 holds bf16 values exactly.
//    Block scales: a key's multiplies the score; a value's multiplies P relative to the
//    largest one so far.

#include <cfloat>

#include "csa_kernels.h"
#include "kv8.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;               // tokens of a warp's step
constexpr int kTile = kStep * kWarps;   // tokens of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleMargin = 8.0f;  // log2 units
constexpr float kPShift = 7.0f;

template <int D>
struct Cfg {
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 4 : 6;
  static constexpr int kCtasPerSm = D == 256 ? 2 : D == 128 ? 3 : 4;
  static constexpr int kStageBytes = 2 * kStep * D;
  static constexpr int kChunks = D / 16;   // 16-byte pieces of a row
  static constexpr int kMb = D / 16;       // 16-dim blocks of O^T
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
};

template <int D, int NB>
constexpr int ctas_per_sm() {
  return D == 64 && NB == 4 ? 3 : NB == 4 || (D == 256 && NB == 2) ? 2 : Cfg<D>::kCtasPerSm;
}

constexpr int kSms = 152;  // of a GB300; another count only changes how even the shares are
constexpr int kMaxParts = 4 * kSms;  // CTAs of a deal

// Byte offset of piece c of token r in a stage's key (or value) half; see the header
// comment for who reads what together.
template <int D, bool V>
__device__ __forceinline__ int piece_offset(int r, int c) {
  if constexpr (D == 64) return (r >> 1) * 128 + (((r ^ (r >> 2)) & 1) << 6) + (c << 4);
  const int x = V ? ((r & 3) << 1) | ((r >> 2) & 1) : r & 7;
  return r * D + ((c ^ x) << 4);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// A request's part in the deal.
struct Job {
  Kv8Req r;
  int32_t first, pre;  // bounds that hold for all of its rows
  Kv8Tiles tiles;
  int32_t pairs;       // key heads x column chunks; 0: not this kernel's
  bool whole;          // the deal is in pairs and not in tiles
  // Units of the deal.  A pair that sees nothing keeps a place of one tile, whose CTA writes the zeros.
  __device__ __forceinline__ int32_t per_pair() const { return whole ? 1 : max(1, tiles.count()); }
  __device__ __forceinline__ int64_t total() const { return (int64_t)pairs * per_pair(); }
};

template <int CC>
__device__ __forceinline__ Job load_job(const Kv8AttnArgs& a, int b) {
  Job j{};
  j.whole = a.whole_pairs;
  if (!kv8_request(a.row_start, a.cached, b, a.n_rows, a.bt, a.cache.rows_per_block, j.r, a.err)) return j;
  const int32_t n = j.r.rows();
  if (n == 0) return j;
  if (n > a.max_new) {
    record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
    return j;
  }
  if ((int64_t)n * a.group > a.few_cols) return j;
  if (a.mask.first && n <= 32) {
    j.first = INT32_MAX;
    for (int i = 0; i < n; ++i) j.first = min(j.first, a.mask.first[j.r.r0 + i]);
    j.first = max(j.first, 0);
  }
  j.pre = a.mask.prefix ? min(a.mask.prefix[b], j.r.len()) : 0;
  const int32_t lo = a.mask.window > 0 ? max(j.first, j.r.cached - a.mask.window + 1) : j.first;
  j.tiles = kv8_tiles(kTile, j.first, j.pre, lo, j.r.len() - 1);
  j.pairs = a.cache.kv_heads * ((n * a.group + CC - 1) / CC);
  return j;
}

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<D, NB>()) kv8_decode_kernel(const Kv8AttnArgs a) {
  using C = Cfg<D>;
  constexpr int CC = 8 * NB, ST = C::kStages, CH = C::kChunks;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int64_t seg_t[kThreads + 1];
  __shared__ int64_t warp_t[kWarps];
  __shared__ float s_scale[kWarps][ST][2];
  __shared__ float s_m[kWarps][CC], s_l[kWarps][CC];
  __shared__ int32_t c_p[CC], c_lo[CC], c_first[CC];  // of each column: position, window start, document start
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int B = a.bt.num_seqs, P = a.cache.rows_per_block, Hk = a.cache.kv_heads, G = a.group;
  const int shift = 31 - __clz(P), dim = a.cache.dim;

  // ---- the deal: exclusive prefix of the threads' segments of requests
  const int seg = (B + kThreads - 1) / kThreads;
  int64_t own = 0;
  for (int b = min(B, tid * seg); b < min(B, tid * seg + seg); ++b) own += load_job<CC>(a, b).total();
  int64_t inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_t[wid] = inc;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < wid; ++w) base += warp_t[w];
  seg_t[tid] = base + inc - own;
  if (tid == kThreads - 1) seg_t[kThreads] = base + inc;
  __syncthreads();
  const int64_t total = seg_t[kThreads];
  const int64_t share = (total + gridDim.x - 1) / gridDim.x;
  int64_t u = (int64_t)blockIdx.x * share;
  const int64_t u_end = min(total, u + share);
  int32_t* head = a.part_head + 8 * blockIdx.x;  // a pair that starts here and ends in a later CTA
  if (tid == 0) head[0] = 0;
  if (tid == 0 && blockIdx.x == 0) *a.part_next = 0;
  if (u >= u_end) return;

  int lo = 0, hi = kThreads;  // the last segment that starts at or before u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seg_t[mid] <= u) lo = mid; else hi = mid;
  }
  int b = lo * seg;
  int64_t b_start = seg_t[lo];
  Job job = load_job<CC>(a, b);

  const uint32_t my_ring = tc::smem_u32(ring) + wid * ST * C::kStageBytes;
  const uint8_t* my_ring_p = ring + wid * ST * C::kStageBytes;
  const uint32_t my_scale = tc::smem_u32(&s_scale[wid][0][0]);

  while (u < u_end) {
    while (u >= b_start + job.total()) {
      b_start += job.total();
      job = load_job<CC>(a, ++b);
    }
    const int per = job.per_pair(), nt = max(1, job.tiles.count());
    const int pair = (int)((u - b_start) / per), ti0 = (int)((u - b_start) % per);
    const int ti1 = job.whole ? nt : (int)min((int64_t)nt, ti0 + (u_end - u));
    const int steps = job.tiles.count() ? ti1 - ti0 : 0;
    const int n_rows = job.r.rows(), n = job.r.len();
    const int chunks = job.pairs / Hk, kvh = pair / chunks, col0 = (pair % chunks) * CC;
    const int n_cols = min(CC, n_rows * G - col0);
    // column blocks that hold something; the others are left out of the products (a request of one
    // row beside others of three)
    const int nbs = NB == 1 ? 1 : (n_cols + 7) / 8;

    // ---- stream: step s of this warp is 16 tokens of tile ti0 + s
    auto token0 = [&](int s) { return job.tiles.at(ti0 + s) * kTile + wid * kStep; };
    auto block_of = [&](int s) {
      if (s >= steps) return -1;
      const int t0 = token0(s);
      return t0 < n ? kv8_block(a.bt, a.cache.num_blocks, b, t0 >> shift) : -1;
    };
    auto issue = [&](int s, int blk) {
      if (s < steps) {
        const int st = s % ST, t0 = token0(s);
        const int left = blk >= 0 ? n - t0 : 0;  // tokens there are
        const int64_t at = (int64_t)max(blk, 0) * Hk + kvh;
        const int64_t off = (at * P + (t0 & (P - 1))) * dim;
        const uint8_t* ks = reinterpret_cast<const uint8_t*>(a.cache.k) + off;
        const uint8_t* vs = reinterpret_cast<const uint8_t*>(a.cache.v) + off;
        const uint32_t dst = my_ring + st * C::kStageBytes;
#pragma unroll
        for (int i = 0; i < CH / 2; ++i) {
          const int x = lane + 32 * i, r = x / CH, c = x % CH;
          const bool there = r < left && c * 16 < dim;  // else zeros are written and nothing is read
          const int from = r * dim + c * 16;
          tc::cp_async16(dst + piece_offset<D, false>(r, c),
                         there ? ks + from : reinterpret_cast<const uint8_t*>(a.cache.k), there ? 16u : 0u);
          tc::cp_async16(dst + kStep * D + piece_offset<D, true>(r, c),
                         there ? vs + from : reinterpret_cast<const uint8_t*>(a.cache.v), there ? 16u : 0u);
        }
        if (lane < 2) {
          if (blk >= 0) {
            cp_async4(my_scale + (st * 2 + lane) * 4, (lane ? a.cache.v_scale : a.cache.k_scale) + at);
          } else {
            s_scale[wid][st][lane] = -1.0f;
            if (t0 < n) record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
          }
        }
      }
      tc::cp_async_commit();
    };
    int32_t ids[ST];  // the first steps' blocks: looked up together, copied before all else
#pragma unroll
    for (int x = 0; x < ST; ++x) ids[x] = block_of(x);
    __syncthreads();  // the last pair's shared values are read
#pragma unroll
    for (int x = 0; x < ST - 1; ++x) issue(x, ids[x]);
    int32_t next_blk = ids[ST - 1];

    // ---- columns: bounds for the masks, and what they leave to all columns alike
    if (tid < CC) {
      const int i = min((col0 + tid) / G, n_rows - 1), p = job.r.cached + i;
      const int f = a.mask.first ? max(0, a.mask.first[job.r.r0 + i]) : 0;
      c_p[tid] = p;
      c_first[tid] = f;
      c_lo[tid] = a.mask.window > 0 ? max(f, p - a.mask.window + 1) : f;
    }
    __syncthreads();
    int all_lo = 0, all_first = 0, all_p = INT32_MAX;
    for (int c = 0; c < CC; ++c) {
      all_lo = max(all_lo, c_lo[c]);
      all_first = max(all_first, c_first[c]);
      all_p = min(all_p, c_p[c]);
    }

    // ---- queries: columns g of each block, as the B operand
    uint32_t qf[NB][CH][2];
    float fac[NB][2], slope[NB][2];  // of columns 2 t4, 2 t4 + 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int col = nb * 8 + g;
      const bool col_there = col < n_cols;
      const int cg = min(col0 + col, n_rows * G - 1);
      const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(job.r.r0 + cg / G) * a.q_stride +
                          (int64_t)(kvh * G + cg % G) * dim;
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < CH / 4; ++j) {
        uint32_t w[8];
        const bool real = col_there && (t4 + 4 * j) * 16 < dim;
        const uint16_t* src = q + (real ? (t4 + 4 * j) * 16 : 0);
        if (a.q_vec) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(src)), y = __ldg(reinterpret_cast<const uint4*>(src) + 1);
          w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = (uint32_t)src[2 * i] | (uint32_t)src[2 * i + 1] << 16;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          qf[nb][4 * j + i / 2][i & 1] = real ? w[i] : 0u;
          if (real) top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float p2 = pow2_floor(top), r2 = pow2_recip(p2);
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = qf[nb][k][i];
          qf[nb][k][i] = f32x2_to_f16x2(__uint_as_float(w << 16) * r2, __uint_as_float(w & 0xffff0000u) * r2);
        }
      const float f = p2 * a.mask.scale;
      const float s = a.mask.slopes ? a.mask.slopes[kvh * G + cg % G] * kLog2e : 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // from the lanes of columns 2 t4, 2 t4 + 1
        fac[nb][i] = __shfl_sync(0xffffffffu, f, (2 * t4 + i) * 4);
        slope[nb][i] = __shfl_sync(0xffffffffu, s, (2 * t4 + i) * 4);
      }
    }
    const bool cap = a.mask.softcap > 0.f, bias = a.mask.slopes != nullptr;
    const float pre_mul = cap ? 2.0f * kLog2e / a.mask.softcap : kLog2e, post_mul = a.mask.softcap * kLog2e;

    float o[NB][C::kMb][4], m[NB][2], l[NB][2], vref = kKv8MinScale, vinv = 1.0f / kKv8MinScale;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < C::kMb; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][k][i] = 0.f;
      m[nb][0] = m[nb][1] = -FLT_MAX;
      l[nb][0] = l[nb][1] = 0.f;
    }

    for (int s = 0; s < steps; ++s) {
      tc::cp_async_wait<ST - 2>();
      __syncwarp();
      issue(s + ST - 1, next_blk);
      next_blk = block_of(s + ST);
      const int st = s % ST, t0 = token0(s);
      const uint8_t* kb = my_ring_p + st * C::kStageBytes;
      const uint8_t* vb = kb + kStep * D;
      const float kscale = s_scale[wid][st][0], vscale = s_scale[wid][st][1];
      if (kscale < 0.f || t0 >= n) continue;  // no block, or no token

      float sc[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[nb][i] = 0.f;
      const int r0 = 4 * (g & 1) + (g >> 1);
#pragma unroll
      for (int j = 0; j < CH / 4; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(kb + piece_offset<D, false>(r0, t4 + 4 * j));
        const uint4 y = *reinterpret_cast<const uint4*>(kb + piece_offset<D, false>(r0 + 8, t4 + 4 * j));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2(xw[i], a0, a2);
          e4m3x4_to_f16x2(yw[i], a1, a3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            if (nb == 0 || nb < nbs) mma_f16(sc[nb], a0, a1, a2, a3, qf[nb][4 * j + i][0], qf[nb][4 * j + i][1]);
        }
      }

      // scores in log2 units: [0], [1] token t0 + r0 of columns 2 t4, 2 t4 + 1; [2], [3] token t0 + r0 + 8
      const float mul = kscale * pre_mul;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[nb][i] *= fac[nb][i & 1] * mul;
      if (cap) {
        bool small = true;  // for tanh_small2, whose error goes by the score and not by the cap
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) small &= fabsf(sc[nb][i]) <= kTanhSmall * 2.0f * kLog2e;
        small = __all_sync(0xffffffffu, small);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (nb >= nbs) break;
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float2 y = make_float2(sc[nb][i], sc[nb][i + 1]);
            const float2 z = small ? tanh_small2(mul2(y, make_float2(0.5f / kLog2e, 0.5f / kLog2e)))
                                   : make_float2(tanh_exp2(y.x), tanh_exp2(y.y));
            sc[nb][i] = post_mul * z.x;
            sc[nb][i + 1] = post_mul * z.y;
          }
        }
      }
      if (bias) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (nb >= nbs) break;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sc[nb][i] -= slope[nb][i & 1] * fabsf((float)(c_p[nb * 8 + 2 * t4 + (i & 1)] - (t0 + r0 + 4 * (i & 2))));
        }
      }
      const bool whole = t0 >= all_first && t0 + kStep <= n &&
                         ((t0 >= all_lo && t0 + kStep - 1 <= all_p) || t0 + kStep <= job.pre);
      if (!whole) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (nb >= nbs) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = nb * 8 + 2 * t4 + (i & 1), t = t0 + r0 + 4 * (i & 2);
            const bool see = t < n && t >= c_first[c] && (t < job.pre || (t <= c_p[c] && t >= c_lo[c]));
            if (!see) sc[nb][i] = -INFINITY;
          }
        }
      }
      bool raise = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) raise |= fmaxf(sc[nb][i], sc[nb][i + 2]) > m[nb][i] + kRescaleMargin;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = fmaxf(sc[nb][i], sc[nb][i + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            x = fmaxf(x, m[nb][i]);
            const float alpha = fast_exp2(m[nb][i] - x);
            m[nb][i] = x;
            l[nb][i] *= alpha;
#pragma unroll
            for (int k = 0; k < C::kMb; ++k) o[nb][k][i] *= alpha, o[nb][k][i + 2] *= alpha;
          }
      }
      if (vscale > vref) {
        const float alpha = __fdividef(vref, vscale);
        vref = vscale;
        vinv = 1.0f / vscale;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < C::kMb; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[nb][k][i] *= alpha;
      }
      const float vr = vscale * vinv;
      uint32_t pf[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (nb >= nbs) break;
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = fast_exp2(sc[nb][i] - (m[nb][i & 1] - kPShift));
          l[nb][i & 1] += e[i];
        }
        pf[nb][0] = transpose8x8(f32x2_to_f16x2(e[0] * vr, e[1] * vr));
        pf[nb][1] = transpose8x8(f32x2_to_f16x2(e[2] * vr, e[3] * vr));
      }
      // values: pieces of tokens t4, t4 + 4 (first half of the product's tokens), t4 + 8, t4 + 12
      if constexpr (D == 64) {
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = *reinterpret_cast<const uint2*>(vb + piece_offset<D, true>(t4 + 4 * i, g >> 1) + (g & 1) * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x[4] = {i ? w[0].y : w[0].x, i ? w[1].y : w[1].x, i ? w[2].y : w[2].x, i ? w[3].y : w[3].x};
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2(__byte_perm(x[0], x[1], hf ? 0x7362 : 0x5140), a0, a1);
            e4m3x4_to_f16x2(__byte_perm(x[2], x[3], hf ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              if (nb == 0 || nb < nbs) mma_f16(o[nb][2 * i + hf], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < D / 128; ++j) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = *reinterpret_cast<const uint4*>(vb + piece_offset<D, true>(t4 + 4 * i, g + 8 * j));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            auto word = [i](const uint4& v) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2(__byte_perm(word(w[0]), word(w[1]), hf ? 0x7362 : 0x5140), a0, a1);
              e4m3x4_to_f16x2(__byte_perm(word(w[2]), word(w[3]), hf ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                if (nb == 0 || nb < nbs) mma_f16(o[nb][8 * j + 2 * i + hf], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
            }
          }
        }
      }
    }
    tc::cp_async_wait<0>();

    // ---- join the warps: each leaves its scaled O^T in its own ring, as it holds it
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], d);
        if (g == 0) s_m[wid][nb * 8 + 2 * t4 + i] = m[nb][i], s_l[wid][nb * 8 + 2 * t4 + i] = l[nb][i];
      }
    __syncthreads();
    const bool whole_pair = ti0 == 0 && ti1 == nt;
    constexpr int kRingFloats = ST * C::kStageBytes / 4;
    float* mine = reinterpret_cast<float*>(ring) + wid * kRingFloats;
    const int par = wid & 1, half = wid >> 1;  // this warp's part of the sum: column parity, half of the dims
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (nb >= nbs) break;
      float mm[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = nb * 8 + 2 * t4 + i;
        mm[i] = fmaxf(fmaxf(s_m[0][c], s_m[1][c]), fmaxf(s_m[2][c], s_m[3][c]));
        const float f = fast_exp2(s_m[wid][c] - mm[i]) * vref;
#pragma unroll
        for (int k = 0; k < C::kMb; ++k) {
          mine[(4 * k + i) * 32 + lane] = o[nb][k][i] * f;
          mine[(4 * k + i + 2) * 32 + lane] = o[nb][k][i + 2] * f;
        }
      }
      __syncthreads();
      const int c = nb * 8 + 2 * t4 + par;
      const float top = par ? mm[1] : mm[0];
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += s_l[w][c] * fast_exp2(s_m[w][c] - top);
      constexpr int kHalf = C::kMb / 2;
      float y[2 * kHalf];
#pragma unroll
      for (int k = 0; k < kHalf; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = (4 * (half * kHalf + k) + par + 2 * e) * 32 + lane;
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += reinterpret_cast<const float*>(ring)[w * kRingFloats + r];
          y[2 * k + e] = v;
        }
      const int d0 = D == 256 ? half * 128 + 16 * g : (D / 8) * g + half * (D / 16);
      if (d0 >= dim) {
      } else if (c < n_cols && whole_pair) {
        const int cg = col0 + c;
        const int64_t rh = (int64_t)(job.r.r0 + cg / G) * a.heads + kvh * G + cg % G;
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + rh * dim + d0;
        uint32_t z[kHalf];
#pragma unroll
        for (int k = 0; k < kHalf; ++k) z[k] = f32x2_to_bf16x2(y[2 * k] * inv, y[2 * k + 1] * inv);
        if (a.out_vec) {
#pragma unroll
          for (int k = 0; k < kHalf; k += 2) *reinterpret_cast<uint2*>(dst + 2 * k) = make_uint2(z[k], z[k + 1]);
        } else {
#pragma unroll
          for (int k = 0; k < kHalf; ++k) dst[2 * k] = (uint16_t)z[k], dst[2 * k + 1] = (uint16_t)(z[k] >> 16);
        }
        if (a.lse && half == 0 && g == 0) a.lse[rh] = sum == 0.f ? -INFINITY : (top - kPShift + log2f(sum)) * kLn2;
      } else if (c < n_cols) {
        const int64_t slot = (2 * (int64_t)blockIdx.x + (ti0 == 0)) * CC + c;
        float* dst = a.part_o + slot * D + d0;
#pragma unroll
        for (int k = 0; k < 2 * kHalf; k += 2) *reinterpret_cast<float2*>(dst + k) = make_float2(y[k], y[k + 1]);
        if (half == 0 && g == 0) a.part_ml[2 * slot] = top, a.part_ml[2 * slot + 1] = sum;
      }
      __syncthreads();
    }
    if (tid == 0 && ti0 == 0 && ti1 < nt) {
      head[0] = 1 + (int32_t)((nt - ti1 + share - 1) / share);  // parts: this one and the next CTAs'
      head[1] = job.r.r0;
      head[2] = kvh;
      head[3] = col0;
      head[4] = n_cols;
    }
    u += job.whole ? 1 : ti1 - ti0;
  }
}

// Joins the parts of the pair that starts in CTA blockIdx.x of the deal and ends in a later one:
// part 0 in that CTA's second slot, the others in the next CTAs' first slots.
template <int D, int NB>
__global__ void __launch_bounds__(kThreads) kv8_decode_join_kernel(const Kv8AttnArgs a) {
  constexpr int CC = 8 * NB;
  pdl_trigger();
  pdl_wait();
  const int cta = blockIdx.x, c = blockIdx.y;
  const int32_t* head = a.part_head + 8 * cta;
  const int parts = head[0];
  if (parts == 0 || c >= head[4]) return;
  const int kvh = head[2], cg = head[3] + c, G = a.group;
  const int64_t rh = (int64_t)(head[1] + cg / G) * a.heads + kvh * G + cg % G;
  auto slot = [&](int i) { return (2 * (int64_t)(cta + i) + (i == 0)) * CC + c; };
  __shared__ float weight[kMaxParts];
  __shared__ float sums[kWarps][D];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  float m = -FLT_MAX;
  for (int i = lane; i < parts; i += 32) m = fmaxf(m, a.part_ml[2 * slot(i)]);
  m = warp_max(m);
  float l = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float w = fast_exp2(a.part_ml[2 * slot(i)] - m);
    l += a.part_ml[2 * slot(i) + 1] * w;
    if (wid == 0) weight[i] = w;
  }
  l = warp_sum(l);
  __syncthreads();
  // a warp every fourth part, a lane D / 32 dims
  float o[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) o[k] = 0.f;
#pragma unroll 4
  for (int i = wid; i < parts; i += kWarps) {
    const float* src = a.part_o + slot(i) * D + lane * (D / 32);
    const float w = weight[i];
#pragma unroll
    for (int k = 0; k < D / 32; k += 2) {
      const float2 v = *reinterpret_cast<const float2*>(src + k);
      o[k] += v.x * w;
      o[k + 1] += v.y * w;
    }
  }
#pragma unroll
  for (int k = 0; k < D / 32; ++k) sums[wid][lane * (D / 32) + k] = o[k];
  __syncthreads();
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  for (int d = tid; d < D; d += kThreads)
    if (d < a.cache.dim) reinterpret_cast<uint16_t*>(a.out)[rh * a.cache.dim + d] =
        f32_to_bf16(((sums[0][d] + sums[1][d]) + (sums[2][d] + sums[3][d])) * inv);
  if (a.lse && tid == 0) a.lse[rh] = l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * kLn2;
}


template <int D, int NB>
cudaError_t launch(const Kv8AttnArgs& a, cudaStream_t s) {
  static PerDevice attr;
  const cudaError_t e = with_device_slot(attr, [](int, int64_t& v) {
    if (v) return cudaSuccess;
    const cudaError_t err =
        cudaFuncSetAttribute(kv8_decode_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (err == cudaSuccess) v = 1;
    return err;
  });
  if (e != cudaSuccess) return e;
  const int32_t n = kSms * ctas_per_sm<D, NB>();
  const cudaError_t k = launch_k(kv8_decode_kernel<D, NB>, dim3(n), dim3(kThreads), Cfg<D>::kSmem, s, 0, a);
  if (k != cudaSuccess || a.whole_pairs) return k;
  return launch_k(kv8_decode_join_kernel<D, NB>, dim3(n, 8 * NB), dim3(kThreads), 0, s, 0, a);
}

template <typename F>
auto pick(int32_t dim, int32_t cols, F f) {
  if (dim <= 64)
    return cols <= 8 ? f.template run<64, 1>() : cols <= 16 ? f.template run<64, 2>() : f.template run<64, 4>();
  if (dim <= 128)
    return cols <= 8 ? f.template run<128, 1>() : cols <= 16 ? f.template run<128, 2>() : f.template run<128, 4>();
  return cols <= 8 ? f.template run<256, 1>() : f.template run<256, 2>();  // wider tiles exceed the registers
}

struct SlotsOf {  // two of 8 NB columns a CTA
  template <int D, int NB>
  size_t run() const { return 2 * (size_t)kSms * ctas_per_sm<D, NB>() * 8 * NB; }
};
struct Launch {
  const Kv8AttnArgs& a;
  cudaStream_t s;
  template <int D, int NB>
  cudaError_t run() const { return launch<D, NB>(a, s); }
};

}  // namespace

// O of every slot's columns, (max, sum) of each, then 8 words a CTA (fewer than the slots).
static int32_t tile_dim(int32_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

size_t kv8_decode_workspace(int32_t dim, int32_t cols) {
  const size_t slots = pick(dim, cols, SlotsOf{});
  return slots * tile_dim(dim) * sizeof(float) + slots * 2 * sizeof(float) + slots * 8 * sizeof(int32_t) / 2;
}

void kv8_decode_parts(Kv8AttnArgs& a, void* ws) {
  const size_t slots = pick(a.cache.dim, a.cols, SlotsOf{});
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = a.part_o + slots * tile_dim(a.cache.dim);
  a.part_head = reinterpret_cast<int32_t*>(a.part_ml + slots * 2);
}

cudaError_t launch_kv8_decode(const Kv8AttnArgs& a, cudaStream_t s) { return pick(a.cache.dim, a.cols, Launch{a, s}); }

}  // namespace csa
