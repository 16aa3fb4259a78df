// Attention of many rows a request over the 8-bit key / value cache, on tcgen05: prompt
// chunks, bf16 queries and results.
//
// 4 D FLOPs a row, head and key: the tensor pipe bounds it.  A part is 256 query rows
// (tokens x query heads of one key head, token-major) as two tiles of M = 128 (one for
// heads of more than 128 dims), which meet the keys that they see in tiles of 64:
//
//   S_i [128 x 64]  = Q_i [128 x D] . K^T          both operands from shared memory
//   O_i [128 x D]  += P_i [128 x 64] . V           P from TMEM
//
//  * TMEM: S_0 and S_1 (64 columns each, two buffers, one for heads of 128, which leave no
//    room for more), O_0, O_1 (D columns each) and P_i (f16, 32 columns, two buffers).  One lane
//    issues S_0(t+1), S_1(t+1), O_0(t), O_1(t): the scores of the next tile are there when the
//    softmax comes to them.  S_i(t+1) waits until S_i(t) is in registers where it shares its
//    columns.  (P_i over S_i instead, with two buffers, is 5 to 10 % faster for heads of 128, but
//    then S_i(t+1) overwrites the P_i(t-1) that O_i(t-1) reads, and products of different shapes
//    are not promised to run in the order of issue.  A warp for the S and one for the O
//    took 14 % more time, the order S_0(t+1), O_1(t-1), S_1(t+1), O_0(t) 13 %; with tiles of 128
//    keys and one S_i, each softmax waited for two products and their hand-over.)  The
//    whole warp runs the loop, so that descriptors stay in uniform registers: issued by a
//    lane on its own, each product cost 125 cycles.
//  * Four warps convert: codes of the next two tiles wait in registers, become f16 (exactly)
//    and go to the swizzled operand tiles, four of keys and four of values.  Both query
//    tiles use each converted tile.  (Eight such warps took registers and issue slots from
//    the softmax: 1.30 ms against 1.37 without a cap, but 1.99 against 1.81 with one.)
//  * Softmax: warps 0-3 hold the rows of tile 0, warps 4-7 those of tile 1, a thread a row,
//    so that no value crosses lanes.  The maximum is raised, and O rescaled, only when a score
//    passes it by 2^8.  Caps and biases are compiled apart: with their code in the common
//    loop, waiting for instructions cost a third of the time.  Scales are those of 16
//    tokens: the key's multiplies the scores, the value's, relative to the largest that the
//    part's rows see, enters the exponent, P = 2^(s - m + 7 + log2(v / v_max)), and is
//    divided out of each 16 columns' part of the sum.
//  * CTAs stay, one an SM, and take parts from a queue.  The roles go from part to part on
//    their own, so that a part's first copies are under way before the last part's result
//    is stored: 1.37 -> 1.17 ms without a cap when it came in.
//  * What bounds it now: two chunks of 2048 tokens at 4k to 16k, 64 query heads on 8 key
//    heads of 128, take 1.26 ms without a cap, 925 TFLOP/s (0.49 of the measured rate; ncu:
//    tensor pipe 43 % busy, issue slots 43 %), and 2.08 ms with one, 561.  The conversion
//    and the softmax each need about the time that the products leave them, and wait for
//    TMEM and for each other the rest of it.

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "csa_kernels.h"
#include "kv8.cuh"
#include "tc_ptx.cuh"

namespace csa {
namespace {

using namespace tc;

constexpr int kTile = 64;      // keys of a tile
constexpr int kM = 128;        // rows of a query tile
constexpr int kStages = 2;     // of key tiles, and of value tiles, in shared memory
constexpr int kSoftmax = 256, kConvert = 128;
constexpr int kThreads = kSoftmax + kConvert + 64;
constexpr int kMmaWarp = (kSoftmax + kConvert) / 32, kLookWarp = kMmaWarp + 1;
constexpr int kGroups = kTile / 16;  // tokens that share a scale
constexpr int kPairBufs = 8;         // pairs of tiles whose addresses and scales are kept
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleMargin = 8.0f, kPShift = 7.0f;

// D: the head size, rounded up to 64, 128 or 256 (the rest are zeros)
template <int D>
struct Cfg {
  static constexpr int kMT = D == 256 ? 1 : 2;   // query tiles: O takes kMT D columns of TMEM
  static constexpr int kPer = D == 256 ? 1 : 2;  // tiles of a stage, as shared memory allows
  static constexpr uint32_t kQAtom = kM * 128, kAtom = kTile * 128;  // rows of 64 f16
  static constexpr uint32_t kQBytes = kQAtom * (D / 64), kTileBytes = kAtom * (D / 64);
  static constexpr uint32_t kOffK = kMT * kQBytes, kOffV = kOffK + kPer * kStages * kTileBytes;
  static constexpr uint32_t kOffMisc = kOffV + kPer * kStages * kTileBytes;
  static constexpr int kSBufs = D == 128 ? 1 : 2;  // buffers of S_i: TMEM has no more room beside two heads of 128
  static constexpr uint32_t kColO = kMT * kSBufs * kTile;
  static constexpr int kUnits = kTile * (D / 16) / kConvert;  // 16-byte pieces of a tile a thread
  __host__ __device__ static constexpr uint32_t col_s(int i, int t) { return kTile * (kSBufs * i + t % kSBufs); }
  __host__ __device__ static constexpr uint32_t col_p(int i, int t) {
    return kColO + kMT * D + (kTile / 2) * (2 * i + t % 2);
  }
  static_assert(kColO + kMT * D + kTile * kMT <= 512, "TMEM");
};

// What a CTA works on: tokens i0 .. of request b for key head kvh.
struct Part {
  Kv8Req r;
  int32_t b, kvh, x, i0, tpt;  // x: of the grid; tpt: tokens of a query tile
  int32_t n, first, pre;    // tokens stored, the lowest document start, the prefix
  int32_t all_first, all_lo, all_p;  // what all rows have in common: see from here on, to here
  Kv8Tiles tiles;
  int32_t begin, count;     // of the key tiles: this part's share
  int32_t split;
  float v_max;              // the largest value scale of its blocks
  int32_t end;              // no part: there are no more
  __device__ __forceinline__ int32_t tile(int32_t t) const { return tiles.at(begin + t); }
};

struct Misc {
  uint64_t k_full[kStages], k_free[kStages], v_full[kStages], v_free[kStages];
  // by the parity of t within its part: who waits for a tile may be one tile behind, never two
  uint64_t s_full[2][2], s_read[2][2], p_full[2][2], o_done[2][2];
  uint64_t at_full[kPairBufs], at_free[kPairBufs], mma_done;
  // by the parity of the part: a role may be one part ahead of another (after one that sees nothing)
  uint64_t part_full[2], part_free[2], q_full[2], o_free[2][2];
  uint32_t tmem_base;
  int32_t abort;
  Part part[2];
  // of the last tiles, by 16 tokens: offset of the codes (-1: none), key scale (negative: no block),
  // log2 of the value scale relative to the part's largest, and its inverse
  int64_t src[2 * kPairBufs][kGroups];
  alignas(16) float ks[2 * kPairBufs][kGroups];
  alignas(16) float lv[2 * kPairBufs][kGroups];
  alignas(16) float rv[2 * kPairBufs][kGroups];
  int32_t t0[2 * kPairBufs];     // first token
  int32_t plain[2 * kPairBufs];  // every row of the part sees every key of the tile
};

template <int D>
constexpr uint32_t smem_bytes() { return Cfg<D>::kOffMisc + sizeof(Misc) + 1024; }

// Bounded wait; after the first timeout in the CTA every later wait that is not over
// already returns at once, so all roles run to the end and TMEM is released.
__device__ __forceinline__ bool wait_or_abort(Misc& ms, uint64_t* bar, uint32_t parity, int32_t* err) {
  if (mbar_test(bar, parity)) return true;
  if (*reinterpret_cast<volatile int32_t*>(&ms.abort)) return false;
  if (mbar_wait(bar, parity)) return true;
  *reinterpret_cast<volatile int32_t*>(&ms.abort) = 1;
  record_error(err, CSA_ERR_TIMEOUT);
  return false;
}

// Where a role stands after the parts it has been through: what the barriers' phases follow.
struct Past {
  uint32_t parts = 0, pairs = 0, tiles = 0, even = 0, odd = 0;
  __device__ __forceinline__ void add(int32_t count) {
    ++parts;
    pairs += (count + 1) / 2;
    tiles += count;
    even += (count + 1) / 2;
    odd += count / 2;
  }
  // of the buffers by parity: the uses before tile t's
  __device__ __forceinline__ uint32_t uses(int32_t t) const { return (t & 1 ? odd : even) + (t >> 1); }
};

// The next part, or null: there is none, or a wait gave up.
__device__ __forceinline__ const Part* next_part(Misc& ms, const Past& past, int32_t* err) {
  const uint32_t slot = past.parts & 1;
  if (!wait_or_abort(ms, &ms.part_full[slot], past.parts >> 1 & 1, err)) return nullptr;
  return ms.part[slot].end ? nullptr : &ms.part[slot];
}

// ------------------------------------------------------------------ conversion

// Eight neighbouring lanes take four pieces (16 dims) of two rows: what they write to the
// swizzled tile together falls on different banks.
template <int D>
struct Unit {
  int row, piece;  // row: of the thread's first unit, the others kConvert 16 / D further each
  int off, step;   // within 16 tokens' codes; step: of every other unit, when rows are 8 apart
  bool there;      // the piece is not past the head size
  __device__ __forceinline__ Unit(int ct, int dim) {
    if constexpr (D == 64) {  // 32 rows of 4 pieces
      row = ct >> 2, piece = ct & 3;
    } else if constexpr (D == 128) {  // 16 rows of 8
      row = ((ct >> 2) & 1) + 2 * (ct >> 4), piece = (ct & 3) + ((ct >> 1) & 4);
    } else {  // 8 rows of 16
      row = ((ct >> 2) & 1) + 2 * (ct >> 5), piece = (ct & 3) + ((ct >> 1) & 12);
    }
    off = row % 16 * dim + piece * 16;
    step = D == 256 ? 8 * dim : 0;
    there = piece * 16 < dim;
  }
};

template <int D>
__device__ __forceinline__ void load_units(const int64_t* src, const uint8_t* codes, const Unit<D>& un, uint4* x) {
  constexpr int kRows = kConvert / (D / 16);
#pragma unroll
  for (int i = 0; i < Cfg<D>::kUnits; ++i) {
    const int row = un.row + i * kRows;
    const int64_t at = src[row / 16];  // tokens past the sequence hold any code
    x[i] = at >= 0 && un.there ? __ldg(reinterpret_cast<const uint4*>(codes + at + un.off + (i & 1) * un.step))
                               : make_uint4(0, 0, 0, 0);
  }
}

// `left`: rows of the tile that hold tokens; the others become zeros
template <int D, bool WHOLE>
__device__ __forceinline__ void store_units(uint8_t* tile, const Unit<D>& un, const uint4* x, int left) {
  constexpr int kRows = kConvert / (D / 16);
  uint8_t* at0 = tile + sw128_offset(un.row, 16 * un.piece, kTile);
  uint8_t* at1 = tile + sw128_offset(un.row, 16 * un.piece + 8, kTile);
#pragma unroll
  for (int i = 0; i < Cfg<D>::kUnits; ++i) {  // rows a multiple of 8 apart: the swizzle stays
    uint4 lo, hi;
    const bool there = WHOLE || un.row + i * kRows < left;
    e4m3x4_to_f16x2(there ? x[i].x : 0u, lo.x, lo.y);
    e4m3x4_to_f16x2(there ? x[i].y : 0u, lo.z, lo.w);
    e4m3x4_to_f16x2(there ? x[i].z : 0u, hi.x, hi.y);
    e4m3x4_to_f16x2(there ? x[i].w : 0u, hi.z, hi.w);
    *reinterpret_cast<uint4*>(at0 + i * kRows * 128) = lo;
    *reinterpret_cast<uint4*>(at1 + i * kRows * 128) = hi;
  }
}

template <int D>
__device__ __forceinline__ void convert_role(const Kv8AttnArgs& a, uint8_t* smem, Misc& ms, int ct) {
  using C = Cfg<D>;
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.cache.k);
  const uint8_t* vc = reinterpret_cast<const uint8_t*>(a.cache.v);
  const Unit<D> un(ct, a.cache.dim);
  Past past;
  while (const Part* next = next_part(ms, past, a.err)) {
    const Part& w = *next;
    const int count = w.count, n = w.n;
    uint4 kx[C::kPer][C::kUnits], vx[C::kPer][C::kUnits];  // a stage on its way
    const uint32_t stage0 = C::kPer == 2 ? past.pairs : past.tiles;
    auto load = [&](int u, const uint8_t* codes, uint4 (&x)[C::kPer][C::kUnits]) {
      const uint32_t pair = past.pairs + u * C::kPer / 2;
      if (C::kPer * u < count) wait_or_abort(ms, &ms.at_full[pair % kPairBufs], (pair / kPairBufs) & 1, a.err);
#pragma unroll
      for (int j = 0; j < C::kPer; ++j) {
        const int t = C::kPer * u + j;
        if (t < count) load_units<D>(ms.src[2 * (pair % kPairBufs) + (t & 1)], codes, un, x[j]);
      }
    };
    auto store = [&](int u, uint32_t off, uint64_t* full, uint64_t* free, const int (&left)[C::kPer],
                     const uint4 (&x)[C::kPer][C::kUnits]) {
      const uint32_t at = stage0 + u, st = at % kStages;
      if (at >= kStages) wait_or_abort(ms, &free[st], (at / kStages - 1) & 1, a.err);
#pragma unroll
      for (int j = 0; j < C::kPer; ++j) {
        const int t = C::kPer * u + j;
        if (t >= count) break;
        uint8_t* tile = smem + off + (C::kPer * st + j) * C::kTileBytes;
        if (left[j] >= kTile) store_units<D, true>(tile, un, x[j], kTile);
        else store_units<D, false>(tile, un, x[j], left[j]);
      }
      fence_proxy_async();
      mbar_arrive(&full[st]);
    };
    load(0, kc, kx);
    load(0, vc, vx);
    for (int u = 0; C::kPer * u < count; ++u) {
      int left[C::kPer];  // tokens from each tile on; kept for V, by whose turn the softmax may have let go of the tile
#pragma unroll
      for (int j = 0; j < C::kPer; ++j) {
        const int t = C::kPer * u + j;
        left[j] = t < count ? n - ms.t0[2 * ((past.pairs + (t >> 1)) % kPairBufs) + (t & 1)] : 0;
      }
      store(u, C::kOffK, ms.k_full, ms.k_free, left, kx);
      load(u + 1, kc, kx);
      store(u, C::kOffV, ms.v_full, ms.v_free, left, vx);
      load(u + 1, vc, vx);
    }
    __syncwarp();
    if ((ct & 31) == 0) mbar_arrive(&ms.part_free[past.parts & 1]);
    past.add(count);
  }
}

// ------------------------------------------------------------------ products

// The whole warp runs this, so that descriptors stay in uniform registers; one lane issues.
template <int D>
__device__ __forceinline__ void mma_role(const Kv8AttnArgs& a, uint8_t* smem, Misc& ms, uint32_t tmem_v) {
  using C = Cfg<D>;
  constexpr uint32_t idesc_s = idesc_f16(kM, kTile, 0, 0);  // Q and K, both K-major
  constexpr uint32_t idesc_o = idesc_f16(kM, D, 0, 1);      // P from TMEM, V [token][dim] MN-major
  const uint32_t base = uniform(smem_u32(smem)), tmem = uniform(tmem_v);
  const uint64_t d_q = sdesc_sw128(base, 16, 1024);
  const uint64_t d_k = sdesc_sw128(base + C::kOffK, 16, 1024);
  const uint64_t d_v = sdesc_sw128(base + C::kOffV, C::kAtom, 1024);
  const bool lead = elect_one();
  Past past;
  while (const Part* next = next_part(ms, past, a.err)) {
    const Part& w = *next;
    const int n = uniform(w.count);
    const uint32_t stage0 = uniform(C::kPer == 2 ? past.pairs : past.tiles);
    bool ok = wait_or_abort(ms, &ms.q_full[past.parts & 1], past.parts >> 1 & 1, a.err);
    auto products_s = [&](int t) {  // S_0(t), S_1(t)
      const uint32_t at = stage0 + t / C::kPer, st = at % kStages;
      if (t % C::kPer == 0) ok = ok && wait_or_abort(ms, &ms.k_full[st], at / kStages & 1, a.err);
      const uint32_t ko = ((C::kPer * st + t % C::kPer) * C::kTileBytes) >> 4;
      if (C::kSBufs == 1 && t > 0) {  // (two buffers: S_i(t-2) was read before P_i(t-2) came)
#pragma unroll
        for (int i = 0; i < C::kMT; ++i)
          ok = ok && wait_or_abort(ms, &ms.s_read[i][(t - 1) & 1], past.uses(t - 1) & 1, a.err);
        tc_fence_after();
      }
      if (lead) {
#pragma unroll
        for (int i = 0; i < C::kMT; ++i) {
          if (ok) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              mma_bf16(tmem + C::col_s(i, t), d_q + ((i * C::kQBytes + (ks >> 2) * C::kQAtom + (ks & 3) * 32) >> 4),
                       d_k + ko + (((ks >> 2) * C::kAtom + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
          }
          mma_commit(&ms.s_full[i][t & 1]);
        }
        if (t % C::kPer == C::kPer - 1 || t == n - 1) mma_commit(&ms.k_free[st]);
      }
      __syncwarp();
    };
    if (n > 0) products_s(0);
    // the last part's O has been read
    if (past.parts > 0)
      for (int i = 0; i < C::kMT; ++i)
        ok = ok && wait_or_abort(ms, &ms.o_free[i][(past.parts - 1) & 1], (past.parts - 1) >> 1 & 1, a.err);
    for (int t = 0; t < n; ++t) {
      if (t + 1 < n) products_s(t + 1);
      const uint32_t at = stage0 + t / C::kPer, st = at % kStages;
      if (t % C::kPer == 0) ok = ok && wait_or_abort(ms, &ms.v_full[st], at / kStages & 1, a.err);
      const uint32_t vo = ((C::kPer * st + t % C::kPer) * C::kTileBytes) >> 4;
      const uint32_t use = past.uses(t) & 1;
#pragma unroll
      for (int i = 0; i < C::kMT; ++i) {
        ok = ok && wait_or_abort(ms, &ms.p_full[i][t & 1], use, a.err);
        tc_fence_after();
        if (lead) {
          if (ok) {
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              mma_f16_ts(tmem + C::kColO + D * i, tmem + C::col_p(i, t) + 8 * ks, d_v + vo + ((ks * 2048) >> 4),
                         idesc_o, (t | ks) != 0);
          }
          mma_commit(&ms.o_done[i][t & 1]);
          if (i == C::kMT - 1 && (t % C::kPer == C::kPer - 1 || t == n - 1)) mma_commit(&ms.v_free[st]);
        }
        __syncwarp();
      }
    }
    if (lead) mbar_arrive(&ms.part_free[past.parts & 1]);
    past.add(n);
  }
  // nothing may still write TMEM when it is released, even after a timeout
  if (lead) mma_commit(&ms.mma_done);
  __syncwarp();
  mbar_wait(&ms.mma_done, 0);
}

// ------------------------------------------------------------------ softmax

// First row of a CTA's partial results.
template <int D>
__device__ __forceinline__ int64_t part_slot(int64_t gx, int64_t x, int kvh, int split, int n_splits) {
  return ((kvh * gx + x) * n_splits + split) * (Cfg<D>::kMT * kM);
}

// Bits [a, b) of 64, whatever a and b are.
__device__ __forceinline__ uint64_t key_bits(int64_t a, int64_t b) {
  a = max((int64_t)0, min((int64_t)64, a));
  b = max(a, min((int64_t)64, b));
  return (b >= 64 ? ~0ull : (1ull << b) - 1) & ~(a >= 64 ? ~0ull : (1ull << a) - 1);
}

template <int D, bool CAP, bool BIAS>
__device__ __forceinline__ void softmax_part(const Kv8AttnArgs& a, const Part& w, int count, const Past& past, uint8_t* smem,
                                             Misc& ms, uint32_t tmem, int st) {
  using C = Cfg<D>;
  const int i = st >> 7, m_row = st & 127, G = a.group, dim = a.cache.dim;
  const int tok = w.i0 + i * w.tpt + m_row / G, head = w.kvh * G + m_row % G;
  const bool real = m_row < w.tpt * G && tok < w.r.rows();
  const int64_t row = w.r.r0 + tok;

  // ---- Q, each row scaled by a power of two to [1, 2), as f16.  A warp reads its 32 rows together,
  // D / 8 lanes a row: alone, a thread would touch its row's lines one after the other.
  float p2 = 1.f;
  {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes a row, rows at a time
    uint8_t* tile = smem + i * C::kQBytes;
    const int lane = st & 31, piece = lane % kLanes, sub = lane / kLanes, row0 = m_row - lane;
    // a row's offset, or -1, from the lane that holds it
    const int64_t mine = real ? row * a.q_stride + (int64_t)head * dim : -1;
#pragma unroll 1
    for (int c0 = 0; c0 < 32 / kRows; c0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int64_t at = __shfl_sync(0xffffffffu, mine, (c0 + c) * kRows + sub);
        const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + at + 8 * piece;
        v[c] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && 8 * piece < dim) {
          if (a.q_vec) {
            v[c] = __ldg(reinterpret_cast<const uint4*>(q));
          } else {
            v[c] = make_uint4(q[0] | (uint32_t)q[1] << 16, q[2] | (uint32_t)q[3] << 16, q[4] | (uint32_t)q[5] << 16,
                              q[6] | (uint32_t)q[7] << 16);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xffff0000u))));
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float f = pow2_floor(top), r2 = pow2_recip(f);
        uint32_t e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          e[k] = f32x2_to_f16x2(__uint_as_float(x[k] << 16) * r2, __uint_as_float(x[k] & 0xffff0000u) * r2);
        const int r = (c0 + c) * kRows + sub;
        *reinterpret_cast<uint4*>(tile + sw128_offset(row0 + r, 8 * piece, kM)) = make_uint4(e[0], e[1], e[2], e[3]);
        const float back = __shfl_sync(0xffffffffu, f, lane % kRows * kLanes);
        if (lane / kRows == c0 + c) p2 = back;
      }
    }
    fence_proxy_async();
    mbar_arrive(&ms.q_full[past.parts & 1]);
  }

  const float fac = p2 * a.mask.scale * (CAP ? 2.0f * kLog2e / a.mask.softcap : kLog2e);
  const float post = a.mask.softcap * kLog2e;
  const float slope = BIAS && real ? a.mask.slopes[head] * kLog2e : 0.f;
  const int p = real ? w.r.cached + tok : INT32_MAX;
  const int first = real && a.mask.first ? max(0, a.mask.first[row]) : 0;
  const int lo = real && a.mask.window > 0 ? max(first, p - a.mask.window + 1) : first;
  const uint32_t lane_addr = tmem + ((uint32_t)(32 * ((st >> 5) & 3)) << 16);
  const uint32_t o_addr = lane_addr + C::kColO + D * i;
  float m = -FLT_MAX, l = 0.f;

  for (int t = 0; t < count; ++t) {
    const uint32_t pair = past.pairs + (t >> 1), sb = 2 * (pair % kPairBufs) + (t & 1), use = past.uses(t) & 1;
    const uint32_t s_addr = lane_addr + C::col_s(i, t), p_addr = lane_addr + C::col_p(i, t);
    wait_or_abort(ms, &ms.at_full[pair % kPairBufs], (pair / kPairBufs) & 1, a.err);
    // what turns the accumulator's 16 columns into scores in log2 units, before the cap; not 0, so
    // that it leaves -inf alone
    const float4 ks4 = *reinterpret_cast<const float4*>(ms.ks[sb]);
    const float f[kGroups] = {fmaxf(fac * ks4.x, FLT_MIN), fmaxf(fac * ks4.y, FLT_MIN), fmaxf(fac * ks4.z, FLT_MIN),
                              fmaxf(fac * ks4.w, FLT_MIN)};
    const int t0 = ms.t0[sb];
    const bool plain = ms.plain[sb];
    wait_or_abort(ms, &ms.s_full[i][t & 1], use, a.err);
    tc_fence_after();
    float x[kTile];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) tmem_ld16(s_addr + 16 * g, x + 16 * g);
    tmem_wait_ld();
    if constexpr (C::kSBufs == 1) {
      tc_fence_before();
      __syncwarp();
      if ((st & 31) == 0) mbar_arrive(&ms.s_read[i][t & 1]);
    }
    if (CAP && (BIAS || !plain)) {  // the cap comes before a bias, and -inf would not pass it
      bool small = true;
#pragma unroll
      for (int k = 0; k < kTile; ++k) small &= fabsf(x[k]) * f[k / 16] <= kTanhSmall * 2.0f * kLog2e;
      small = __all_sync(0xffffffffu, small);
#pragma unroll
      for (int k = 0; k < kTile; k += 2) {
        float2 y = mul2(make_float2(x[k], x[k + 1]), make_float2(f[k / 16], f[k / 16]));
        y = small ? tanh_small2(mul2(y, make_float2(0.5f / kLog2e, 0.5f / kLog2e)))
                  : make_float2(tanh_exp2(y.x), tanh_exp2(y.y));
        x[k] = post * y.x;
        x[k + 1] = post * y.y;
      }
    }
    if constexpr (BIAS) {
#pragma unroll
      for (int k = 0; k < kTile; ++k)
        x[k] = (CAP ? x[k] : x[k] * f[k / 16]) - slope * fabsf((float)(p - t0) - (float)k);
    }
    if (!plain) {
      // a bit for each key that the row sees
      uint64_t see = key_bits(lo - t0, (int64_t)p + 1 - t0) | key_bits(first - t0, w.pre - t0);
      see &= key_bits(first - t0, w.n - t0);
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if (ms.ks[sb][g] < 0.f) see &= ~(0xffffull << (16 * g));
#pragma unroll
      for (int k = 0; k < kTile; ++k) x[k] = see >> k & 1 ? x[k] : -INFINITY;
    }
    // the cap rises with the accumulator: without a bias or a mask only the maximum is capped here
    float mt = -INFINITY;
    bool small = true;  // scores that tanh_small2 takes
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float* y = x + 16 * g;
      float z[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = fmaxf(fmaxf(y[k], y[k + 4]), fmaxf(y[k + 8], y[k + 12]));
      const float top = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
      mt = fmaxf(mt, BIAS || (CAP && !plain) ? top : CAP ? post * tanh_exp2(top * f[g]) : top * f[g]);
      if constexpr (CAP && !BIAS) {
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = fminf(fminf(y[k], y[k + 4]), fminf(y[k + 8], y[k + 12]));
        const float low = fminf(fminf(z[0], z[1]), fminf(z[2], z[3]));
        small &= fmaxf(top, -low) * f[g] <= kTanhSmall * 2.0f * kLog2e;
      }
    }
    small = CAP && !BIAS && __all_sync(0xffffffffu, small);
    if (__any_sync(0xffffffffu, mt > m + kRescaleMargin)) {
      const float mn = fmaxf(m, mt), alpha = fast_exp2(m - mn);
      m = mn;
      l *= alpha;
      if (t > 0) {
        // O holds exactly the tiles before t once O(t-1) is complete
        wait_or_abort(ms, &ms.o_done[i][(t - 1) & 1], past.uses(t - 1) & 1, a.err);
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tmem_ld16(o_addr + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] *= alpha;
          tmem_st16(o_addr + c, o);
        }
      }
    }
    // ---- P(t), over P(t-2): O(t-2) was issued before S(t), so its product is done
    const float4 lv4 = *reinterpret_cast<const float4*>(ms.lv[sb]), rv4 = *reinterpret_cast<const float4*>(ms.rv[sb]);
    const float lv[kGroups] = {lv4.x, lv4.y, lv4.z, lv4.w}, rv[kGroups] = {rv4.x, rv4.y, rv4.z, rv4.w};
    const float shift = kPShift - m;
    auto write_p = [&](auto how) {  // of 0: the accumulator; 1: scores; 2, 3: what the cap is for, 3: all small
      constexpr int kHow = decltype(how)::value;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float add = shift + lv[g];
        const float* y = x + 16 * g;
        float2 sum = make_float2(0.f, 0.f);
        uint32_t pw[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float2 e = make_float2(y[2 * k], y[2 * k + 1]);
          if constexpr (kHow == 1) {
            e = add2(e, make_float2(add, add));
          } else if constexpr (kHow == 3) {
            const float fu = f[g] * (0.5f / kLog2e);
            e = fma2(tanh_small2(mul2(e, make_float2(fu, fu))), make_float2(post, post), make_float2(add, add));
          } else if constexpr (kHow == 2) {  // post tanh + add
            e = make_float2(fast_exp2(e.x * f[g]), fast_exp2(e.y * f[g]));
            e = add2(e, make_float2(1.f, 1.f));
            e = make_float2(fast_rcp(e.x), fast_rcp(e.y));
            e = fma2(e, make_float2(-2.f * post, -2.f * post), make_float2(post + add, post + add));
          } else {
            e = fma2(e, make_float2(f[g], f[g]), make_float2(add, add));
          }
          e = make_float2(fast_exp2(e.x), fast_exp2(e.y));
          sum = k ? add2(sum, e) : e;
          pw[k] = f32x2_to_f16x2(e.x, e.y);
        }
        l = fmaf(sum.x + sum.y, rv[g], l);
        tmem_st8(p_addr + 8 * g, pw);
      }
    };
    if constexpr (BIAS) {
      write_p(std::integral_constant<int, 1>{});
    } else if constexpr (CAP) {
      if (!plain) write_p(std::integral_constant<int, 1>{});
      else if (small) write_p(std::integral_constant<int, 3>{});
      else write_p(std::integral_constant<int, 2>{});
    } else {
      write_p(std::integral_constant<int, 0>{});
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((st & 31) == 0) mbar_arrive(&ms.p_full[i][t & 1]);
    if ((t & 1) || t == count - 1) {  // the pair's scales are read
      __syncwarp();
      if ((st & 31) == 0) mbar_arrive(&ms.at_free[pair % kPairBufs]);
    }
  }

  // ---- result
  if (count > 0) wait_or_abort(ms, &ms.o_done[i][(count - 1) & 1], past.uses(count - 1) & 1, a.err);
  tc_fence_after();
  const bool part = a.n_splits > 1;  // one of several shares of the keys: O and l as they are
  const float inv = part ? w.v_max : l == 0.f ? 0.f : w.v_max / l;
  const int64_t slot = part_slot<D>(a.parts_x, w.x, w.kvh, w.split, a.n_splits) + st;
  // bf16 rows go out through the place of Q, which no product reads any more: a warp's 32 rows, D / 8
  // lanes a row
  uint8_t* tile = smem + i * C::kQBytes;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    float o[16];
    if (count > 0) {
      tmem_ld16(o_addr + 16 * c, o);
      tmem_wait_ld();
    }
    if (part) {
      if (real && 16 * c < dim && l != 0.f) {  // else it is not read
        float4* dst = reinterpret_cast<float4*>(a.part_o + slot * D + 16 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dst[k] = make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv, o[4 * k + 3] * inv);
      }
      continue;
    }
    uint32_t z[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = count > 0 ? f32x2_to_bf16x2(o[2 * k] * inv, o[2 * k + 1] * inv) : 0u;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      *reinterpret_cast<uint4*>(tile + sw128_offset(m_row, 16 * c + 8 * k, kM)) =
          make_uint4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]);
  }
  tc_fence_before();
  mbar_arrive(&ms.o_free[i][past.parts & 1]);
  if (!part) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;
    const int lane = st & 31, piece = lane % kLanes, sub = lane / kLanes, row0 = m_row - lane;
    const int64_t mine = real ? (row * a.heads + head) * dim : -1;
    __syncwarp();
#pragma unroll 4
    for (int c = 0; c < 32 / kRows; ++c) {
      const int r = c * kRows + sub;
      const int64_t at = __shfl_sync(0xffffffffu, mine, r);
      const uint4 v = *reinterpret_cast<const uint4*>(tile + sw128_offset(row0 + r, 8 * piece, kM));
      if (at < 0 || 8 * piece >= dim) continue;
      uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + at + 8 * piece;
      if (a.out_vec) {
        *reinterpret_cast<uint4*>(out) = v;
      } else {
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) out[2 * k] = (uint16_t)x[k], out[2 * k + 1] = (uint16_t)(x[k] >> 16);
      }
    }
    __syncwarp();  // before the next part's Q
  }
  if (real && part) {
    a.part_ml[2 * slot] = m;
    a.part_ml[2 * slot + 1] = l;
  } else if (real && a.lse) {
    a.lse[row * a.heads + head] = l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * kLn2;
  }
}

template <int D, bool CAP, bool BIAS>
__device__ __forceinline__ void softmax_role(const Kv8AttnArgs& a, uint8_t* smem, Misc& ms, uint32_t tmem, int st) {
  if ((st >> 7) >= Cfg<D>::kMT) return;
  Past past;
  while (const Part* next = next_part(ms, past, a.err)) {
    const Part& w = *next;
    const int count = w.count;
    softmax_part<D, CAP, BIAS>(a, w, count, past, smem, ms, tmem, st);
    __syncwarp();
    if ((st & 31) == 0) mbar_arrive(&ms.part_free[past.parts & 1]);
    past.add(count);
  }
}

// ------------------------------------------------------------------ parts, addresses and scales

// Part x of key head kvh: with T tokens a part and f(b) = row_start[b] / T + b, request b owns the x in
// [f(b), f(b + 1)), at least rows / T + 1 of them.  False: no rows there, or the few-row kernel's.
// Called by a whole warp.
template <int D>
__device__ __forceinline__ bool find_part(const Kv8AttnArgs& a, int64_t x, int kvh, Part& w) {
  w.tpt = kM / a.group;
  const int T = Cfg<D>::kMT * w.tpt;
  auto first_x = [&](int b) { return (int64_t)a.row_start[b] / T + b; };
  w.b = warp_last_le(a.bt.num_seqs, x, first_x);
  w.kvh = kvh;
  w.x = (int32_t)x;
  if (!kv8_request(a.row_start, a.cached, w.b, a.n_rows, a.bt, a.cache.rows_per_block, w.r, a.err)) return false;
  const int n_new = w.r.rows();
  if (n_new > a.max_new) {
    record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
    return false;
  }
  if ((int64_t)n_new * a.group <= a.few_cols || x < first_x(w.b)) return false;
  w.i0 = (int)min((x - first_x(w.b)) * T, (int64_t)n_new);
  return w.i0 < n_new;
}

// One warp hands the parts out, as the CTAs come to them (an order that no result depends on), and
// runs ahead of the other roles: what the part sees, then, 16 tokens a lane and four pairs of
// tiles at a time, where the keys are, their scales, and which tiles need no mask.
template <int D>
__device__ __forceinline__ void look_up_role(const Kv8AttnArgs& a, Misc& ms) {
  const int lane = threadIdx.x & 31, g = lane % kGroups, P = a.cache.rows_per_block, shift = 31 - __clz(P);
  const int Hk = a.cache.kv_heads;
  const int64_t total = (int64_t)a.parts_x * Hk * a.n_splits;
  Past past;
  for (int64_t turn = blockIdx.x;; turn += gridDim.x) {
    int64_t id = turn;
    if (a.part_next) {
      int next = 0;
      if (lane == 0) next = atomicAdd(a.part_next, 1);
      id = __shfl_sync(0xffffffffu, next, 0);
    }
    Part w{};
    w.end = id >= total;
    if (!w.end) {
      // parts that see more keys go first
      if (!find_part<D>(a, a.parts_x - 1 - id % a.parts_x, (int)(id / a.parts_x % Hk), w)) continue;
      w.split = (int32_t)(id / a.parts_x / Hk);
      const int last = min(w.r.rows(), w.i0 + Cfg<D>::kMT * w.tpt) - 1;  // token
      w.n = w.r.len();
      w.pre = a.mask.prefix ? min(a.mask.prefix[w.b], w.n) : 0;
      if (a.mask.first) {
        int32_t low = INT32_MAX, high = 0;
        for (int i = w.i0 + lane; i <= last; i += 32) {
          const int32_t f = max(a.mask.first[w.r.r0 + i], 0);
          low = min(low, f);
          high = max(high, f);
        }
        w.first = __reduce_min_sync(0xffffffffu, low);
        w.all_first = __reduce_max_sync(0xffffffffu, high);
      }
      w.all_p = w.r.cached + w.i0;
      w.all_lo = a.mask.window > 0 ? max(w.all_first, w.r.cached + last - a.mask.window + 1) : w.all_first;
      const int lo = a.mask.window > 0 ? max(w.first, w.r.cached + w.i0 - a.mask.window + 1) : w.first;
      w.tiles = kv8_tiles(kTile, w.first, w.pre, lo, w.r.cached + last);
      const int64_t all = w.tiles.count();
      w.begin = (int32_t)(all * w.split / a.n_splits);
      w.count = (int32_t)(all * (w.split + 1) / a.n_splits) - w.begin;
      float top = kKv8MinScale;
      for (int part = 0; part < 2; ++part) {
        const int i0 = part ? max(w.begin, w.tiles.nA) : w.begin;
        const int nt = (part ? w.begin + w.count : min(w.begin + w.count, w.tiles.nA)) - i0, t0 = w.tiles.at(i0) * kTile;
        const int lb1 = (min(w.n, t0 + nt * kTile) + P - 1) >> shift;
        if (nt > 0)
#pragma unroll 4
          for (int lb = (t0 >> shift) + lane; lb < lb1; lb += 32) {
            const int32_t blk = kv8_block(a.bt, a.cache.num_blocks, w.b, lb);
            if (blk >= 0) top = fmaxf(top, a.cache.v_scale[(int64_t)blk * Hk + w.kvh]);
          }
      }
      w.v_max = warp_max(top);
    }
    const uint32_t slot = past.parts & 1;
    if (past.parts >= 2 && !wait_or_abort(ms, &ms.part_free[slot], ((past.parts >> 1) - 1) & 1, a.err)) return;
    if (lane == 0) {
      ms.part[slot] = w;
      mbar_arrive(&ms.part_full[slot]);
    }
    if (w.end) return;
    const float inv_top = 1.0f / w.v_max;
    for (int u0 = 0; 2 * u0 < w.count; u0 += 4) {
      const int t = 2 * u0 + lane / kGroups, sb = (int)((past.pairs + (t >> 1)) % kPairBufs) * 2 + (t & 1);
      float ks = -1.f, vs = 1.f;
      int64_t src = -1;
      if (t < w.count) {
        const int tok = w.tile(t) * kTile + 16 * g;
        if (tok < w.n) {
          const int32_t blk = kv8_block(a.bt, a.cache.num_blocks, w.b, tok >> shift);
          if (blk >= 0) {
            const int64_t at = (int64_t)blk * Hk + w.kvh;
            src = (at * P + (tok & (P - 1))) * a.cache.dim;
            ks = a.cache.k_scale[at];
            vs = a.cache.v_scale[at];
          } else {
            record_error(a.err, CSA_ERR_DEVICE_BOUNDS);
          }
        }
      }
      for (int u = u0; u < u0 + 4 && 2 * u < w.count; ++u) {
        const uint32_t at = past.pairs + u;
        if (at >= kPairBufs) wait_or_abort(ms, &ms.at_free[at % kPairBufs], (at / kPairBufs - 1) & 1, a.err);
      }
      if (t < w.count) {
        if (src >= 0) vs = fmaxf(vs * inv_top, kKv8MinScale);
        ms.src[sb][g] = src;
        ms.ks[sb][g] = ks;
        ms.lv[sb][g] = log2f(vs);
        ms.rv[sb][g] = 1.0f / vs;
      }
      // of the four lanes of a tile: all of its tokens are there, and no row's mask cuts it
      const uint32_t there = __ballot_sync(0xffffffffu, src >= 0);
      if (t < w.count && g == 0) {
        const int t0 = w.tile(t) * kTile;
        ms.t0[sb] = t0;
        ms.plain[sb] = (there >> lane & 15u) == 15u && t0 + kTile <= w.n && t0 >= w.all_first &&
                       ((t0 >= w.all_lo && t0 + kTile - 1 <= w.all_p) || t0 + kTile <= w.pre);
      }
      __syncwarp();
      if (lane == 0)
        for (int u = u0; u < u0 + 4 && 2 * u < w.count; ++u) mbar_arrive(&ms.at_full[(past.pairs + u) % kPairBufs]);
    }
    past.add(w.count);
  }
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(const Kv8AttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Misc& ms = *reinterpret_cast<Misc*>(smem + C::kOffMisc);
  const int tid = threadIdx.x, wid = uniform(tid >> 5);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ms.k_full[s], kConvert);
      mbar_init(&ms.v_full[s], kConvert);
      mbar_init(&ms.k_free[s], 1);
      mbar_init(&ms.v_free[s], 1);
    }
    for (int i = 0; i < C::kMT; ++i) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&ms.s_full[i][s], 1);
        mbar_init(&ms.s_read[i][s], 4);
        mbar_init(&ms.p_full[i][s], 4);
        mbar_init(&ms.o_done[i][s], 1);
      }
    }
    for (int u = 0; u < kPairBufs; ++u) {
      mbar_init(&ms.at_full[u], 1);
      mbar_init(&ms.at_free[u], C::kMT * 4);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&ms.part_full[k], 1);
      // the warps of the softmax, of the conversion, the products'
      mbar_init(&ms.part_free[k], C::kMT * 4 + kConvert / 32 + 1);
      mbar_init(&ms.o_free[0][k], 128);
      mbar_init(&ms.o_free[1][k], 128);
      mbar_init(&ms.q_full[k], C::kMT * 128);
    }
    mbar_init(&ms.mma_done, 1);
    ms.abort = 0;
    mbar_init_fence();
  }
  if (wid == kMmaWarp) tmem_alloc(&ms.tmem_base, 512);
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem_base;
  if (wid < kSoftmax / 32) {
    softmax_role<D, CAP, BIAS>(a, smem, ms, tmem, tid);
  } else {
    if (wid < kMmaWarp) convert_role<D>(a, smem, ms, tid - kSoftmax);
    else if (wid == kLookWarp) look_up_role<D>(a, ms);
    else mma_role<D>(a, smem, ms, tmem);
  }
  __syncthreads();
  tc_fence_after();
  if (wid == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the shares of the keys, a warp a row.
template <int D>
__global__ void __launch_bounds__(128) kv8_prefill_join_kernel(const Kv8AttnArgs a) {
  pdl_trigger();
  pdl_wait();
  Part w{};
  if (!find_part<D>(a, blockIdx.x, blockIdx.y, w)) return;
  const int lane = threadIdx.x & 31, G = a.group, dim = a.cache.dim, S = a.n_splits;
  const int st = blockIdx.z * 4 + (threadIdx.x >> 5), m_row = st & (kM - 1);
  const int tok = w.i0 + (st / kM) * w.tpt + m_row / G, head = w.kvh * G + m_row % G;
  if (m_row >= w.tpt * G || tok >= w.r.rows()) return;
  auto slot = [&](int s) { return part_slot<D>(a.parts_x, w.x, w.kvh, s, S) + st; };
  float m = -FLT_MAX;
  for (int s = 0; s < S; ++s) m = fmaxf(m, a.part_ml[2 * slot(s)]);
  float l = 0.f, o[D / 32];
#pragma unroll
  for (int k = 0; k < D / 32; ++k) o[k] = 0.f;
  for (int s = 0; s < S; ++s) {
    const float ls = a.part_ml[2 * slot(s) + 1], f = fast_exp2(a.part_ml[2 * slot(s)] - m);
    if (ls == 0.f) continue;  // saw nothing
    l += ls * f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
      if (lane + 32 * k < dim) o[k] += a.part_o[slot(s) * D + lane + 32 * k] * f;
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int64_t rh = (int64_t)(w.r.r0 + tok) * a.heads + head;
#pragma unroll
  for (int k = 0; k < D / 32; ++k)
    if (lane + 32 * k < dim) reinterpret_cast<uint16_t*>(a.out)[rh * dim + lane + 32 * k] = f32_to_bf16(o[k] * inv);
  if (a.lse && lane == 0) a.lse[rh] = l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * kLn2;
}

constexpr int kSms = 152;  // of a GB300

// The head size of the kernel that takes `dim`.
int32_t tile_dim(int32_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

int64_t grid_x(int32_t n_rows, int32_t num_seqs, int32_t group, int32_t dim) {
  const int32_t tiles = tile_dim(dim) == 256 ? Cfg<256>::kMT : Cfg<128>::kMT;
  return (int64_t)n_rows / (tiles * (kM / group)) + num_seqs;
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
  const int64_t parts = (int64_t)a.parts_x * a.cache.kv_heads * a.n_splits;
  const cudaError_t k = launch_k(kv8_prefill_kernel<D, CAP, BIAS>, dim3((unsigned)std::min<int64_t>(parts, kSms)),
                                 dim3(kThreads), smem_bytes<D>(), s, 0, a);
  if (k != cudaSuccess || a.n_splits == 1) return k;
  return launch_k(kv8_prefill_join_kernel<D>, dim3(a.parts_x, a.cache.kv_heads, Cfg<D>::kMT * kM / 4), dim3(128), 0, s,
                  0, a);
}

template <int D>
cudaError_t launch_dim(const Kv8AttnArgs& a, cudaStream_t s) {
  const bool cap = a.mask.softcap > 0.f, bias = a.mask.slopes != nullptr;
  if (cap) return bias ? launch<D, true, true>(a, s) : launch<D, true, false>(a, s);
  return bias ? launch<D, false, true>(a, s) : launch<D, false, false>(a, s);
}

}  // namespace

bool kv8_prefill_eligible(int32_t group) { return group <= kM; }

// A few parts over long sequences leave most SMs idle, so their keys are shared out: to as many
// CTAs as one wave holds, each with 8 tiles or more of the `max_len` tokens that the table can
// map, and 16 at most.  16 new tokens behind 128k, 64 query and 8 key heads: 3.4 ms with one
// CTA a part, 0.17 ms with 16.
int32_t kv8_prefill_splits(int32_t n_rows, int32_t num_seqs, int32_t heads, int32_t kv_heads, int32_t dim,
                           int64_t max_len) {
  const int64_t ctas = grid_x(n_rows, num_seqs, heads / kv_heads, dim) * kv_heads;
  int64_t s = kSms / ctas;
  const int64_t most = max_len / (8 * kTile);
  if (s > most) s = most;
  return (int32_t)(s < 1 ? 1 : s > 16 ? 16 : s);
}

size_t kv8_prefill_workspace(int32_t n_rows, int32_t num_seqs, int32_t heads, int32_t kv_heads, int32_t dim,
                             int32_t splits) {
  if (splits <= 1) return 0;
  const int32_t D = tile_dim(dim), rows = (D == 256 ? Cfg<256>::kMT : Cfg<128>::kMT) * kM;
  return (size_t)grid_x(n_rows, num_seqs, heads / kv_heads, dim) * kv_heads * splits * rows * (D + 2) * sizeof(float);
}

void kv8_prefill_parts(Kv8AttnArgs& a, void* ws) {
  a.parts_x = (int32_t)grid_x(a.n_rows, a.bt.num_seqs, a.group, a.cache.dim);
  const int32_t D = tile_dim(a.cache.dim), rows = (D == 256 ? Cfg<256>::kMT : Cfg<128>::kMT) * kM;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = a.part_o + (size_t)a.parts_x * a.cache.kv_heads * a.n_splits * rows * D;
}

cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, cudaStream_t s) {
  const int32_t D = tile_dim(a.cache.dim);
  return D == 64 ? launch_dim<64>(a, s) : D == 128 ? launch_dim<128>(a, s) : launch_dim<256>(a, s);
}

}  // namespace csa
