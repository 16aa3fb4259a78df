// Attention of many rows a request over the 8-bit key / value cache, on tcgen05: prompt
// chunks, bf16 queries and results, heads of 64 or 128.
//
// 4 D FLOPs a row, head and key: the tensor pipe bounds it.  One CTA an SM takes 256
// query rows (tokens x query heads of one key head, token-major) as two tiles of M = 128,
// and walks the keys that its rows see in tiles of 128:
//
//   S_i [128 x 128]  = Q_i [128 x D] . K^T          both operands from shared memory
//   O_i [128 x D]   += P_i [128 x 128] . V          P from TMEM, where it replaces S_i
//
//  * TMEM: S_0, S_1 (128 columns each), O_0, O_1 (D columns each).  P_i (f16, 64 columns)
//    is written over S_i.  One thread issues S_0(t), O_1(t-1), S_1(t), O_0(t): while the
//    softmax works on one tile's scores, the pipe has the other tile's two products.
//    The pipe executes them in the order of issue, so S_i(t+1) follows O_i(t), which reads
//    P_i(t), without a wait between them.
//  * Four warps convert: codes of the next tile wait in registers, become f16 (exactly)
//    and go to the swizzled operand tiles, two stages of keys and of values.  Both query
//    tiles use each converted tile.
//  * Softmax: warps 0-3 hold the rows of tile 0, warps 4-7 those of tile 1, a thread a row,
//    so that no value crosses lanes.  The scores are read twice, 64 columns at a time (once
//    for the maximum), since 128 of them do not fit the registers.  Caps and biases are
//    compiled apart: with their code in the common loop, waiting for instructions cost more
//    than half of the time.  The row's
//    maximum is raised, and O rescaled, only when a score passes it by 2^8.  Scales are those of 16
//    tokens: the key's multiplies the scores, the value's, relative to the largest that the
//    CTA's rows see, enters the exponent, P = 2^(s - m + 7 + log2(v / v_max)), and is
//    divided out of each 16 columns' part of the sum.

#include <cfloat>

#include "csa_kernels.h"
#include "kv8.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace {

using namespace tc;

constexpr int kTile = 128;     // keys of a tile
constexpr int kM = 128;        // rows of a query tile
constexpr int kMTiles = 2;
constexpr int kSoftmax = kMTiles * 128, kConvert = 128;
constexpr int kThreads = kSoftmax + kConvert + 32;  // the last warp issues the products
constexpr int kMmaWarp = (kSoftmax + kConvert) / 32;
constexpr int kHalf = kTile / 4;  // columns of a tile that a softmax thread holds at a time
constexpr int kGroups = kTile / 16;  // tokens that share a scale
constexpr int kScaleBufs = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleMargin = 8.0f, kPShift = 7.0f;

template <int D>
struct Cfg {
  static constexpr uint32_t kAtom = kTile * 128;             // 128 rows of 64 f16
  static constexpr uint32_t kTileBytes = kAtom * (D / 64);   // a query, key or value tile
  static constexpr uint32_t kOffK = kMTiles * kTileBytes, kOffV = kOffK + 2 * kTileBytes;
  static constexpr uint32_t kOffMisc = kOffV + 2 * kTileBytes;
  static constexpr uint32_t kColS = 0, kColO = kMTiles * kTile;
  static constexpr int kUnits = kTile * (D / 16) / kConvert;  // 16-byte pieces of a tile a thread
};

struct Misc {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t q_full, s_full[kMTiles], p_full[kMTiles], o_done[kMTiles], sc_full[kScaleBufs], mma_done;
  uint32_t tmem_base;
  int32_t abort;
  int32_t owner;
  float red[kConvert / 32];
  float v_max;
  // by tile mod 8 and 16 tokens: offset of the codes (-1: none), key scale (negative: no block), log2 of the value scale
  // relative to v_max, and its inverse
  int64_t src[kScaleBufs][kGroups];
  alignas(16) float ks[kScaleBufs][kGroups], lv[kScaleBufs][kGroups], rv[kScaleBufs][kGroups];
};

template <int D>
constexpr uint32_t smem_bytes() { return Cfg<D>::kOffMisc + sizeof(Misc) + 1024; }

// Bounded wait; after the first timeout in the CTA every later wait returns at
// once, so all roles run to the end and TMEM is released.
__device__ __forceinline__ bool wait_or_abort(Misc& ms, uint64_t* bar, uint32_t parity, int32_t* err) {
  if (*reinterpret_cast<volatile int32_t*>(&ms.abort)) return false;
  if (mbar_wait(bar, parity)) return true;
  *reinterpret_cast<volatile int32_t*>(&ms.abort) = 1;
  record_error(err, CSA_ERR_TIMEOUT);
  return false;
}

// What a CTA works on: tokens [i0, i0 + nt) of request b for key head kvh.
struct Part {
  Kv8Req r;
  int32_t b, kvh, i0, tpt;  // tpt: tokens of a query tile
  int32_t n, first, pre;    // tokens stored, the lowest document start, the prefix
  Kv8Tiles tiles;
  int32_t count;            // key tiles
};

// ------------------------------------------------------------------ conversion

// Eight neighbouring lanes take four pieces (16 dims) of two rows: what they write to the
// swizzled tile together falls on different banks.
template <int D>
struct Unit {
  int row, piece;  // row: of the thread's first unit, the others kConvert 16 / D further each
  __device__ __forceinline__ explicit Unit(int ct) {
    if constexpr (D == 64) {
      row = ct >> 2, piece = ct & 3;
    } else {
      row = ((ct >> 2) & 1) + 2 * (ct >> 4), piece = (ct & 3) + ((ct >> 1) & 4);
    }
  }
};

template <int D>
__device__ __forceinline__ void load_units(const int64_t* src, const uint8_t* codes, const Unit<D>& un, uint4* x) {
  constexpr int kRows = kConvert / (D / 16);
#pragma unroll
  for (int i = 0; i < Cfg<D>::kUnits; ++i) {
    const int row = un.row + i * kRows;
    const int64_t at = src[row / 16];  // tokens past the sequence hold some code: only V needs zeros there
    x[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(codes + at + (row % 16) * D + un.piece * 16))
                   : make_uint4(0, 0, 0, 0);
  }
}

// `left`: rows of the tile that hold tokens; the others become zeros
template <int D>
__device__ __forceinline__ void store_units(uint8_t* tile, const Unit<D>& un, const uint4* x, int left) {
  constexpr int kRows = kConvert / (D / 16);
  uint8_t* at0 = tile + sw128_offset(un.row, 16 * un.piece, kTile);
  uint8_t* at1 = tile + sw128_offset(un.row, 16 * un.piece + 8, kTile);
#pragma unroll
  for (int i = 0; i < Cfg<D>::kUnits; ++i) {  // rows a multiple of 8 apart: the swizzle stays
    uint4 lo, hi;
    const bool there = un.row + i * kRows < left;
    e4m3x4_to_f16x2(there ? x[i].x : 0u, lo.x, lo.y);
    e4m3x4_to_f16x2(there ? x[i].y : 0u, lo.z, lo.w);
    e4m3x4_to_f16x2(there ? x[i].z : 0u, hi.x, hi.y);
    e4m3x4_to_f16x2(there ? x[i].w : 0u, hi.z, hi.w);
    *reinterpret_cast<uint4*>(at0 + i * kRows * 128) = lo;
    *reinterpret_cast<uint4*>(at1 + i * kRows * 128) = hi;
  }
}

template <int D>
__device__ void convert_role(const Kv8AttnArgs& a, const Part& w, uint8_t* smem, Misc& ms, int ct) {
  using C = Cfg<D>;
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.cache.k);
  const uint8_t* vc = reinterpret_cast<const uint8_t*>(a.cache.v);
  const int P = a.cache.rows_per_block, Hk = a.cache.kv_heads, shift = 31 - __clz(P);
  // the largest value scale of the blocks that the tiles touch
  float top = kKv8MinScale;
  for (int part = 0; part < 2; ++part) {
    const int t0 = (part ? w.tiles.tB : w.tiles.tA) * kTile, nt = part ? w.tiles.nB : w.tiles.nA;
    const int lb1 = (min(w.n, t0 + nt * kTile) + P - 1) >> shift;
    if (nt > 0)
#pragma unroll 4
      for (int lb = (t0 >> shift) + ct; lb < lb1; lb += kConvert) {
        const int32_t blk = kv8_block(a.bt, a.cache.num_blocks, w.b, lb);
        if (blk >= 0) top = fmaxf(top, a.cache.v_scale[(int64_t)blk * Hk + w.kvh]);
      }
  }
  top = warp_max(top);
  if ((ct & 31) == 0) ms.red[ct >> 5] = top;
  named_bar(1, kConvert);
#pragma unroll
  for (int i = 0; i < kConvert / 32; ++i) top = fmaxf(top, ms.red[i]);
  if (ct == 0) ms.v_max = top;  // read by the softmax after sc_full, or after the CTA's last barrier
  const float inv_top = 1.0f / top;

  // where the tile's tokens are, and their scales, 16 tokens a lane of the first warp
  auto look_up = [&](int t) {
    if (ct >= 32 || t >= w.count) return;
    const int sb = t % kScaleBufs;
    if (ct < kGroups) {
      const int tok = w.tiles.at(t) * kTile + 16 * ct;
      float ks = -1.f, vs = 1.f;
      int64_t src = -1;
      if (tok < w.n) {
        const int32_t blk = kv8_block(a.bt, a.cache.num_blocks, w.b, tok >> shift);
        if (blk >= 0) {
          const int64_t at = (int64_t)blk * Hk + w.kvh;
          src = (at * P + (tok & (P - 1))) * D;
          ks = a.cache.k_scale[at];
          vs = fmaxf(a.cache.v_scale[at] * inv_top, kKv8MinScale);
        } else {
          record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
        }
      }
      ms.src[sb][ct] = src;
      ms.ks[sb][ct] = ks;
      ms.lv[sb][ct] = log2f(vs);
      ms.rv[sb][ct] = 1.0f / vs;
    }
    __syncwarp();
    if (ct == 0) mbar_arrive(&ms.sc_full[sb]);
  };
  const Unit<D> un(ct);
  uint4 kx[C::kUnits], vx[C::kUnits];
  look_up(0);
  look_up(1);
  named_bar(1, kConvert);
  if (w.count > 0) {
    load_units<D>(ms.src[0], kc, un, kx);
    load_units<D>(ms.src[0], vc, un, vx);
  }
  for (int t = 0; t < w.count; ++t) {
    const int st = t & 1, left = w.n - w.tiles.at(t) * kTile;
    const uint32_t prev = ((t >> 1) & 1) ^ 1;  // the use of the stage before this one
    if (t >= 2) wait_or_abort(ms, &ms.k_free[st], prev, a.err);
    store_units<D>(smem + C::kOffK + st * C::kTileBytes, un, kx, left);
    fence_proxy_async();
    mbar_arrive(&ms.k_full[st]);
    // tile t - 3 and all before it are done with (v_free, one tile ago): its place takes tile t + 2
    look_up(t + 2);
    const int64_t* src = ms.src[(t + 1) % kScaleBufs];
    if (t + 1 < w.count) load_units<D>(src, kc, un, kx);
    if (t >= 2) wait_or_abort(ms, &ms.v_free[st], prev, a.err);
    store_units<D>(smem + C::kOffV + st * C::kTileBytes, un, vx, left);
    fence_proxy_async();
    mbar_arrive(&ms.v_full[st]);
    if (t + 1 < w.count) load_units<D>(src, vc, un, vx);
    named_bar(1, kConvert);  // the next tile's addresses
  }
}

// ------------------------------------------------------------------ products

template <int D>
__device__ void mma_role(const Kv8AttnArgs& a, const Part& w, uint8_t* smem, Misc& ms, uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t idesc_s = idesc_f16(kM, kTile, 0, 0);  // Q and K, both K-major
  constexpr uint32_t idesc_o = idesc_f16(kM, D, 0, 1);      // P from TMEM, V [token][dim] MN-major
  const uint64_t d_q = sdesc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t d_k = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
  const uint64_t d_v = sdesc_sw128(smem_u32(smem + C::kOffV), C::kAtom, 1024);
  const int n = w.count;
  bool ok = wait_or_abort(ms, &ms.q_full, 0, a.err);
  auto product_s = [&](int i, int t) {
    const uint32_t ko = ((t & 1) * C::kTileBytes) >> 4, qo = (i * C::kTileBytes) >> 4;
    if (ok) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t at = ((ks >> 2) * C::kAtom + (ks & 3) * 32) >> 4;
        mma_bf16(tmem + C::kColS + kTile * i, d_q + qo + at, d_k + ko + at, idesc_s, ks > 0);
      }
    }
    mma_commit(&ms.s_full[i]);
  };
  auto product_o = [&](int i, int t) {
    ok = ok && wait_or_abort(ms, &ms.v_full[t & 1], (t >> 1) & 1, a.err);
    ok = ok && wait_or_abort(ms, &ms.p_full[i], t & 1, a.err);
    tc_fence_after();
    const uint32_t vo = ((t & 1) * C::kTileBytes) >> 4;
    if (ok) {
#pragma unroll
      for (int ks = 0; ks < kTile / 16; ++ks)
        mma_f16_ts(tmem + C::kColO + D * i, tmem + C::kColS + kTile * i + 8 * ks, d_v + vo + ((ks * 2048) >> 4), idesc_o,
                   (t | ks) != 0);
    }
    mma_commit(&ms.o_done[i]);
  };
  for (int t = 0; t < n; ++t) {
    ok = ok && wait_or_abort(ms, &ms.k_full[t & 1], (t >> 1) & 1, a.err);
    tc_fence_after();
    product_s(0, t);
    if (t > 0) {
      product_o(1, t - 1);
      mma_commit(&ms.v_free[(t - 1) & 1]);
    }
    product_s(1, t);
    mma_commit(&ms.k_free[t & 1]);
    product_o(0, t);
  }
  if (n > 0) product_o(1, n - 1);
  // nothing may still write TMEM when it is released, even after a timeout
  mma_commit(&ms.mma_done);
  mbar_wait(&ms.mma_done, 0);
}

// ------------------------------------------------------------------ softmax

template <int D, bool CAP, bool BIAS>
__device__ __forceinline__ void softmax_role(const Kv8AttnArgs& a, const Part& w, uint8_t* smem, Misc& ms, uint32_t tmem, int st) {
  using C = Cfg<D>;
  const int i = st >> 7, m_row = st & 127, G = a.group;
  const int tok = w.i0 + i * w.tpt + m_row / G, head = w.kvh * G + m_row % G;
  const bool real = m_row < w.tpt * G && tok < w.r.rows();
  const int64_t row = w.r.r0 + tok;

  // ---- the row of Q, scaled by a power of two to [1, 2), as f16
  float p2 = 1.f;
  {
    uint8_t* tile = smem + i * C::kTileBytes;
    const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + row * a.q_stride + (int64_t)head * D;
    auto piece = [&](int c) {  // 8 dims
      if (!real) return make_uint4(0, 0, 0, 0);
      if (a.q_vec) return __ldg(reinterpret_cast<const uint4*>(q) + c);
      uint32_t e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = (uint32_t)q[8 * c + 2 * k] | (uint32_t)q[8 * c + 2 * k + 1] << 16;
      return make_uint4(e[0], e[1], e[2], e[3]);
    };
    float top = 0.f;
#pragma unroll 8
    for (int c = 0; c < D / 8; ++c) {
      const uint4 v = piece(c);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xffff0000u))));
    }
    p2 = pow2_floor(top);
    const float r2 = pow2_recip(p2);
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {  // from L1 the second time
      const uint4 v = piece(c);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      uint32_t e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        e[k] = f32x2_to_f16x2(__uint_as_float(x[k] << 16) * r2, __uint_as_float(x[k] & 0xffff0000u) * r2);
      *reinterpret_cast<uint4*>(tile + sw128_offset(m_row, 8 * c, kM)) = make_uint4(e[0], e[1], e[2], e[3]);
    }
    fence_proxy_async();
    mbar_arrive(&ms.q_full);
  }

  const float fac = p2 * a.mask.scale * (CAP ? 1.0f / a.mask.softcap : kLog2e);
  const float post = a.mask.softcap * kLog2e;
  const float slope = BIAS && real ? a.mask.slopes[head] * kLog2e : 0.f;
  // rows that do not exist see every key, so that they ask for no mask
  const int p = real ? w.r.cached + tok : INT32_MAX;
  const int first = real && a.mask.first ? max(0, a.mask.first[row]) : 0;
  const int lo = real && a.mask.window > 0 ? max(first, p - a.mask.window + 1) : first;
  const uint32_t lane_addr = tmem + ((uint32_t)(32 * ((st >> 5) & 3)) << 16);
  const uint32_t s_addr = lane_addr + C::kColS + kTile * i, o_addr = lane_addr + C::kColO + D * i;
  float m = -FLT_MAX, l = 0.f;

  for (int t = 0; t < w.count; ++t) {
    const int sb = t % kScaleBufs, t0 = w.tiles.at(t) * kTile;
    wait_or_abort(ms, &ms.sc_full[sb], (t / kScaleBufs) & 1, a.err);
    bool mapped = true;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) mapped &= ms.ks[sb][g] >= 0.f;
    const bool whole = t0 >= first && t0 + kTile <= w.n && ((t0 >= lo && t0 + kTile - 1 <= p) || t0 + kTile <= w.pre);
    const bool plain = __all_sync(0xffffffffu, whole && mapped);
    wait_or_abort(ms, &ms.s_full[i], t & 1, a.err);
    tc_fence_after();
    float x[kHalf];
    auto load = [&](int h) {
#pragma unroll
      for (int c = 0; c < kHalf; c += 16) tmem_ld16(s_addr + kHalf * h + c, x + c);
      tmem_wait_ld();
    };
    // what turns the accumulator's 16 columns into scores in log2 units, before the cap; not 0, so
    // that it leaves -inf alone
    auto factor = [&](int h, int j) { return fmaxf(fac * ms.ks[sb][h * (kHalf / 16) + j], FLT_MIN); };
    auto finish = [&](int h) {
      if constexpr (CAP || BIAS) {
#pragma unroll
        for (int j = 0; j < kHalf / 16; ++j) {
          const float f = factor(h, j);
#pragma unroll
          for (int k = 16 * j; k < 16 * j + 16; ++k) {
            float y = x[k] * f;
            if constexpr (CAP) y = post * tanh_exp(y);
            if constexpr (BIAS) y -= slope * fabsf((float)(p - t0 - kHalf * h) - (float)k);
            x[k] = y;
          }
        }
      }
      if (!plain) {
#pragma unroll
        for (int k = 0; k < kHalf; ++k) {
          const int key = t0 + kHalf * h + k;
          const bool see = key < w.n && key >= first && (key < w.pre || (key <= p && key >= lo)) &&
                           ms.ks[sb][h * (kHalf / 16) + k / 16] >= 0.f;
          x[k] = see ? x[k] : -INFINITY;
        }
      }
    };

    // ---- the tile's maximum
    float mt = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < kTile / kHalf; ++h) {
      load(h);
      // the cap rises with the accumulator: without a bias or a mask only the maximum is capped
      const bool raw = CAP && !BIAS && plain;
      if (!raw) finish(h);
#pragma unroll
      for (int j = 0; j < kHalf / 16; ++j) {
        float z = x[16 * j];
#pragma unroll
        for (int k = 1; k < 16; ++k) z = fmaxf(z, x[16 * j + k]);
        if (raw) z = post * tanh_exp(z * factor(h, j));
        else if (!CAP && !BIAS) z *= factor(h, j);
        mt = fmaxf(mt, z);
      }
    }
    if (__any_sync(0xffffffffu, mt > m + kRescaleMargin)) {
      const float mn = fmaxf(m, mt), alpha = fast_exp2(m - mn);
      m = mn;
      l *= alpha;
      if (t > 0) {
        // O holds exactly the tiles before t once O(t-1) is complete
        wait_or_abort(ms, &ms.o_done[i], (t - 1) & 1, a.err);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld16(o_addr + c, o);
          tmem_ld16(o_addr + c + 16, o + 16);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= alpha;
          tmem_st16(o_addr + c, o);
          tmem_st16(o_addr + c + 16, o + 16);
        }
      }
    }
    // ---- P over S: the first half's 32 columns end before the second half's scores begin
    const float shift = kPShift - m;
#pragma unroll 1
    for (int h = 0; h < kTile / kHalf; ++h) {
      load(h);
      finish(h);
#pragma unroll
      for (int j = 0; j < kHalf / 16; ++j) {
        const float f = factor(h, j), add = shift + ms.lv[sb][h * (kHalf / 16) + j];
        float s0 = 0.f, s1 = 0.f;
        uint32_t pw[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float x0 = x[16 * j + 2 * k], x1 = x[16 * j + 2 * k + 1];
          const float y0 = fast_exp2(CAP || BIAS ? x0 + add : fmaf(x0, f, add));
          const float y1 = fast_exp2(CAP || BIAS ? x1 + add : fmaf(x1, f, add));
          s0 += y0;
          s1 += y1;
          pw[k] = f32x2_to_f16x2(y0, y1);
        }
        l = fmaf(s0 + s1, ms.rv[sb][h * (kHalf / 16) + j], l);
        tmem_st8(s_addr + kHalf / 2 * h + 8 * j, pw);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(&ms.p_full[i]);
  }

  // ---- result
  if (w.count > 0) wait_or_abort(ms, &ms.o_done[i], (w.count - 1) & 1, a.err);
  tc_fence_after();
  const float inv = l == 0.f ? 0.f : ms.v_max / l;
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (row * a.heads + head) * D;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    float o[16];
    if (w.count > 0) {
      tmem_ld16(o_addr + 16 * c, o);
      tmem_wait_ld();
    }
    if (!real) continue;
    uint32_t z[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = w.count > 0 ? f32x2_to_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv) : 0u;
    if (a.out_vec) {
      reinterpret_cast<uint4*>(out + 16 * c)[0] = make_uint4(z[0], z[1], z[2], z[3]);
      reinterpret_cast<uint4*>(out + 16 * c)[1] = make_uint4(z[4], z[5], z[6], z[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) out[16 * c + 2 * k] = (uint16_t)z[k], out[16 * c + 2 * k + 1] = (uint16_t)(z[k] >> 16);
    }
  }
  if (real && a.lse) a.lse[row * a.heads + head] = l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * kLn2;
  tc_fence_before();
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(const Kv8AttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Misc& ms = *reinterpret_cast<Misc*>(smem + C::kOffMisc);
  const int tid = threadIdx.x, wid = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms.k_full[s], kConvert);
      mbar_init(&ms.v_full[s], kConvert);
      mbar_init(&ms.k_free[s], 1);
      mbar_init(&ms.v_free[s], 1);
    }
    for (int i = 0; i < kMTiles; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_full[i], 128);
      mbar_init(&ms.o_done[i], 1);
    }
    for (int i = 0; i < kScaleBufs; ++i) mbar_init(&ms.sc_full[i], 1);
    mbar_init(&ms.q_full, kSoftmax);
    mbar_init(&ms.mma_done, 1);
    ms.abort = 0;
    ms.v_max = 1.f;
    mbar_init_fence();
  }
  pdl_trigger();
  pdl_wait();

  // ---- the CTA's part: with T tokens a CTA and f(b) = row_start[b] / T + b, request b owns the x in
  // [f(b), f(b + 1)), at least rows / T + 1 of them.  Later parts see more keys and go first.
  Part w{};
  w.tpt = kM / a.group;
  const int T = kMTiles * w.tpt;
  const int64_t x = gridDim.x - 1 - blockIdx.x;
  auto first_x = [&](int b) { return (int64_t)a.row_start[b] / T + b; };
  if (wid == 0) {
    const int b = warp_last_le(a.bt.num_seqs, x, first_x);
    if (tid == 0) ms.owner = b;
  }
  __syncthreads();
  w.b = ms.owner;
  w.kvh = blockIdx.y;
  if (!kv8_request(a.row_start, a.cached, w.b, a.n_rows, a.bt, a.cache.rows_per_block, w.r, a.err)) return;
  const int n_new = w.r.rows();
  if ((int64_t)n_new * a.group <= a.few_cols || n_new > a.max_new || x < first_x(w.b)) return;  // the few-row kernel's
  w.i0 = (int)min((x - first_x(w.b)) * T, (int64_t)n_new);
  if (w.i0 >= n_new) return;
  const int last = min(n_new, w.i0 + T) - 1;  // token
  w.n = w.r.len();
  w.pre = a.mask.prefix ? min(a.mask.prefix[w.b], w.n) : 0;
  if (a.mask.first) {
    w.first = INT32_MAX;
    for (int i = w.i0; i <= last; ++i) w.first = min(w.first, a.mask.first[w.r.r0 + i]);
    w.first = max(w.first, 0);
  }
  const int lo = a.mask.window > 0 ? max(w.first, w.r.cached + w.i0 - a.mask.window + 1) : w.first;
  w.tiles = kv8_tiles(kTile, w.first, w.pre, lo, w.r.cached + last);
  w.count = w.tiles.count();

  if (wid == kMmaWarp) tmem_alloc(&ms.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  if (tid < kSoftmax) {
    softmax_role<D, CAP, BIAS>(a, w, smem, ms, tmem, tid);
  } else {
    if (tid < kSoftmax + kConvert) convert_role<D>(a, w, smem, ms, tid - kSoftmax);
    else if (tid == kSoftmax + kConvert) mma_role<D>(a, w, smem, ms, tmem);
    __syncwarp();
  }
  __syncthreads();
  tc_fence_after();
  if (wid == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, bool CAP, bool BIAS>
cudaError_t launch(const Kv8AttnArgs& a, cudaStream_t s) {
  static PerDevice attr;
  const cudaError_t e = with_device_slot(attr, [](int, int64_t& v) {
    if (v) return cudaSuccess;
    const cudaError_t err = cudaFuncSetAttribute(kv8_prefill_kernel<D, CAP, BIAS>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>());
    if (err == cudaSuccess) v = 1;
    return err;
  });
  if (e != cudaSuccess) return e;
  const unsigned gx = (unsigned)(a.n_rows / (kMTiles * (kM / a.group)) + a.bt.num_seqs);
  return launch_k(kv8_prefill_kernel<D, CAP, BIAS>, dim3(gx, a.cache.kv_heads), dim3(kThreads), smem_bytes<D>(), s, 0,
                  a);
}

template <int D>
cudaError_t launch_dim(const Kv8AttnArgs& a, cudaStream_t s) {
  const bool cap = a.mask.softcap > 0.f, bias = a.mask.slopes != nullptr;
  if (cap) return bias ? launch<D, true, true>(a, s) : launch<D, true, false>(a, s);
  return bias ? launch<D, false, true>(a, s) : launch<D, false, false>(a, s);
}

}  // namespace

bool kv8_prefill_eligible(int32_t dim, int32_t group) { return (dim == 64 || dim == 128) && group <= kM; }

cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, cudaStream_t s) {
  return a.cache.dim == 64 ? launch_dim<64>(a, s) : launch_dim<128>(a, s);
}

}  // namespace csa
