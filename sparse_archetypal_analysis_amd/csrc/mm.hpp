// Matrix products of 16-bit elements on the matrix cores (gfx950): one tiled
// loop for the token model's block and head, with the work on each tile of
// results left to the caller (an Epilogue). Nothing here is exported.
#pragma once

#include "token.hpp"

namespace seacells {
namespace mm {

// How an operand lies in memory: rows of elements along the product's inner
// index k, or rows (one per k) of elements along its outer index.
enum Side : uint32_t { kAlongK = 0, kAcrossK = 1 };

constexpr uint32_t kMaxSegs = 12;
constexpr uint32_t kTileK = 32;
constexpr uint32_t kStages = 4;
constexpr uint32_t kThreads = 256;
constexpr uint32_t kOutside = 0x80000000u;  // a byte offset past every operand's range

// C[m, n] = sum over segments and k of A[., k] B[., k]. Every row starts on 16
// bytes (base and strides), and a row has a multiple of 8 elements. A segment
// is a pair of offsets in elements; all segments have k elements (along K: a
// multiple of 8, the caller's zeros behind its own).
struct Args {
  const uint16_t *a, *b;
  uint64_t lda, ldb;
  uint32_t m, n;
  uint32_t ka, kb;  // k that A and B hold; past it they read as zeros
  uint32_t seg_tiles, tiles;  // tiles of kTileK in a segment, in all
  uint32_t per_split;         // tiles of a part of k (tiles: one part)
  uint32_t tiles_m, tiles_n;
  uint64_t a_off[kMaxSegs], b_off[kMaxSegs];
};

typedef int Srd __attribute__((ext_vector_type(4)));
typedef short Half4 __attribute__((ext_vector_type(4)));
typedef short Half8 __attribute__((ext_vector_type(8)));
typedef float Acc __attribute__((ext_vector_type(4)));
typedef float Row8 __attribute__((ext_vector_type(8)));

// c += a b on the matrix cores. In assembly so that the results stay in the
// accumulation registers that they are given: with all 256 of them taken the
// compiler's own form moves results about between products. Its result is not
// read before settle().
template <class T>
__device__ __forceinline__ void mfma(Half8 a, Half8 b, Acc &c);
template <>
__device__ __forceinline__ void mfma<_Float16>(Half8 a, Half8 b, Acc &c) {
  asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
template <>
__device__ __forceinline__ void mfma<__bf16>(Half8 a, Half8 b, Acc &c) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// Wait states between writes of accumulation registers and products, and
// between products and readers of their results (at most 19 for 8 passes).
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// One wave load of 1 KB (16 bytes a lane) into LDS, from the lane's offsets
// behind a descriptor; past its range it reads zeros. It is in flight until a
// counted wait (landed). In assembly because the compiler makes every LDS read
// behind a builtin's load wait for it, the ring of stages notwithstanding. The
// wait state is M0's; the descriptor is older than settled() below.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(uint32_t lds, const Srd &srd, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(at), "s"(srd)
               : "m0");
}
#pragma clang diagnostic pop

// The wait states between a vector instruction's scalar result, should one be
// part of a descriptor, and the loads that use it.
__device__ __forceinline__ void settled(Srd &a, Srd &b) {
  asm volatile("s_nop 4" : "+s"(a), "+s"(b));
}

// Waits until at most kLeft of the wave's loads are in flight, then for the
// block's other waves.
template <uint32_t kLeft>
__device__ __forceinline__ void landed() {
  static_assert(kLeft < 64, "vmcnt");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLeft) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A lane's outer index behind its tile of 16 and its lane i = lane % 16: two
// neighbouring tiles interleave by fours, so that the results that a lane has
// of both (4 each, of consecutive indexes) are 8 neighbours in memory.
__device__ __forceinline__ constexpr uint32_t outer_of(uint32_t tile, uint32_t i) {
  return (tile / 2) * 32 + (i / 4) * 8 + (tile & 1) * 4 + (i & 3);
}

// One operand's way into registers. kSize: outer indexes of the block's tile.
// LDS holds a stage as 1 KB pieces, one per wave load, 16 bytes a lane; the
// order of the 16-byte chunks within a row is what keeps the banks apart:
//   along K:  rows of 64 bytes (4 chunks) per outer index, chunk ^ s(row).
//             The 16 lanes of a fragment read rows {0-3, 8-11, 16-19, 24-27}
//             of a pair of tiles; s gives them 16 places of the 256 bytes that
//             4 rows span, and 8 places of 128 bytes to each 8 of them.
//   across K: rows of kSize elements per k, chunk ^ 4 (k % 4). A transposing
//             read takes 4 k and 4 chunks' halves: 4 times 64 bytes apart.
template <Side kSide, uint32_t kSize>
struct Lane {
  static constexpr uint32_t kBytes = kSize * kTileK * 2;  // of a stage
  static constexpr uint32_t kLoads = kBytes / 4096;       // of a wave and stage
  static constexpr uint32_t kTiles = kSize / 32;          // of 16, of a wave (half the block's)
  static constexpr uint32_t kChunks = kSize / 8;          // of a row across K

  uint32_t at[kLoads];      // byte offsets of the lane's loads behind the tile's corner
  uint32_t k_of;            // the lane's first k of a stage (across K: of its first load)
  uint32_t read[kTiles / 2];  // byte offsets of the lane's LDS reads, per pair of tiles

  // outer: first outer index of the tile; limit: outer indexes that there are.
  // half: which half of the tile's outer indexes the wave multiplies. row_of(r)
  // gives the outer index of LDS row r (kOutside: none) for operands along K.
  template <class RowOf>
  __device__ __forceinline__ void init(uint64_t ld, uint32_t outer, uint32_t limit, uint32_t half,
                                       RowOf row_of) {
    const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
    if constexpr (kSide == kAlongK) {
      const uint32_t r0 = wave * 16 + lane / 4;
      const uint32_t s = ((r0 >> 3) & 1) + 2 * (((r0 >> 4) ^ (r0 >> 1)) & 1);
      const uint32_t chunk = (lane & 3) ^ s;
      k_of = chunk * 8;
#pragma unroll
      for (uint32_t j = 0; j < kLoads; ++j) {
        const uint32_t row = row_of(j * 64 + r0);
        at[j] = row == kOutside ? kOutside : (uint32_t)(row * ld * 2 + chunk * 16);
      }
      const uint32_t i = lane & 15;
      const uint32_t sr = ((i >> 2) & 1) + 2 * (((i >> 3) ^ (i >> 1)) & 1);
      const uint32_t slot = (lane / 16) ^ sr;
#pragma unroll
      for (uint32_t p = 0; p < kTiles / 2; ++p)
        read[p] = (half * (kSize / 2) + p * 32 + (i / 4) * 8 + (i & 3)) * 64 + slot * 16;
    } else {
      constexpr uint32_t kRows = 1024 / (kSize * 2);  // k of a wave load
      const uint32_t row = wave * kRows + lane / kChunks;
      const uint32_t chunk = (lane % kChunks) ^ ((row & 3) * 4);
      const bool in = outer + chunk * 8 < limit;
      k_of = row;
  #pragma unroll
      for (uint32_t j = 0; j < kLoads; ++j)
        at[j] = in ? (uint32_t)((j * 4 * kRows + row) * ld * 2 + chunk * 16) : kOutside;
      const uint32_t r = (lane & 15) / 4, q = lane & 3;
#pragma unroll
      for (uint32_t p = 0; p < kTiles / 2; ++p) {
        const uint32_t c = (half * (kChunks / 2) + p * 4 + q) ^ (r * 4);
        read[p] = ((lane / 16) * 8 + r) * (kSize * 2) + c * 16;
      }
    }
  }

  static __device__ __forceinline__ Srd srd(const char *base) {
    Srd s;
    s.x = (int)(uint32_t)(uintptr_t)base;
    s.y = (int)((uint32_t)((uintptr_t)base >> 32) & 0xFFFFu);
    s.z = 0x7FFFFFFF;
    s.w = 0x00020000;
    return s;
  }

  // The wave's load j of a stage. k_left: k that the operand still has at the
  // descriptor's base (0: zeros are loaded).
  __device__ __forceinline__ void load(uint32_t j, uint32_t lds, const Srd &srd,
                                       uint32_t k_left) const {
    const uint32_t k = k_of + (kSide == kAlongK ? 0 : j * (4096 / (kSize * 2)));
    load_to_lds(lds + j * 4096, srd, k < k_left ? at[j] : kOutside);
  }

  // The fragment of one tile of 16 from a stage: 8 k of one outer index.
  __device__ __forceinline__ Half8 fragment(const char *stage, uint32_t tile) const {
    typedef __attribute__((address_space(3))) Half4 *At;
    if constexpr (kSide == kAlongK) {
      return *reinterpret_cast<const Half8 *>(stage + read[tile / 2] + (tile & 1) * 256);
    } else {
      const char *p = stage + read[tile / 2] + (tile & 1) * 8;
      const Half4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(p));
      const Half4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(p + 4 * kSize * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Bytes to an operand's element (outer, k).
template <Side kSide>
__device__ __forceinline__ uint64_t corner(uint64_t ld, uint32_t outer, uint32_t k) {
  return (kSide == kAlongK ? outer * ld + k : k * ld + outer) * 2;
}

// Which tile a block takes. Blocks go round robin over the 8 XCDs, each with
// an L2 of its own: an XCD gets consecutive tiles, and consecutive tiles are
// 8 rows of tiles high, so that the blocks that run together share operands.
__device__ __forceinline__ void tile_of(uint32_t block, uint32_t tiles_m, uint32_t tiles_n,
                                        uint32_t *tm, uint32_t *tn) {
  const uint32_t total = tiles_m * tiles_n;
  const uint32_t xcd = block & 7, q = total / 8, r = total & 7;
  const uint32_t id = xcd * q + min(xcd, r) + block / 8;
  const uint32_t band = id / (8 * tiles_n);
  const uint32_t high = min(8u, tiles_m - band * 8);
  const uint32_t in = id - band * 8 * tiles_n;
  *tm = band * 8 + in % high;
  *tn = in / high;
}

// The rows of a tile of B along K: kTile consecutive ones, or for a gated
// product kTile / 2 of the gate and the kTile / 2 up rows `pair` behind them,
// 64 (32) and 64 (32) to each wave's half.
template <uint32_t kTile, bool kGated>
__device__ __forceinline__ uint32_t b_row(uint32_t r, uint32_t outer, uint32_t limit,
                                          uint32_t pair) {
  if (!kGated) return outer + r < limit ? r : kOutside;
  const uint32_t half = r / (kTile / 2), in = r % (kTile / 2);
  const uint32_t up = in / (kTile / 4);
  const uint32_t row = half * (kTile / 4) + in % (kTile / 4);
  return outer + row < limit ? row + up * pair : kOutside;
}

// A block of 4 waves computes kTile x kTile results, each wave a quarter. The
// LDS holds a ring of 4 stages of 32 k; loads run 3 tiles ahead, and the
// fragments of the next tile are read while the present one multiplies, so
// one barrier per tile is all that the waves wait for.
// epi(acc, row, col): all results of the wave; see Epilogue use below.
template <class T, uint32_t kTile, Side kA, Side kB, bool kGated, class Epilogue>
__global__ __launch_bounds__(kThreads, kTile == 256 ? 1 : 2) void product(Args g, Epilogue epi) {
  constexpr uint32_t kSub = kTile / 32;  // tiles of 16 of a wave, each way
  typedef Lane<kA, kTile> LaneA;
  typedef Lane<kB, kTile> LaneB;
  constexpr uint32_t kStage = LaneA::kBytes + LaneB::kBytes;
  constexpr uint32_t kLoads = LaneA::kLoads + LaneB::kLoads;
  __shared__ __attribute__((aligned(1024))) char ring[kStages * kStage];

  const uint32_t wave = threadIdx.x / kWave;
  const uint32_t wm = wave & 1, wn = wave >> 1;
  uint32_t tm, tn;
  tile_of(blockIdx.x, g.tiles_m, g.tiles_n, &tm, &tn);
  const uint32_t row0 = tm * kTile;
  const uint32_t col0 = tn * (kGated ? kTile / 2 : kTile);
  const uint32_t t0 = blockIdx.y * g.per_split;
  const uint32_t tiles = min(g.per_split, g.tiles - t0);

  LaneA la;
  LaneB lb;
  la.init(g.lda, row0, g.m, wm, [&](uint32_t r) { return row0 + r < g.m ? r : kOutside; });
  lb.init(g.ldb, col0, g.n, wn,
          [&](uint32_t r) { return b_row<kTile, kGated>(r, col0, g.n, g.n); });

  // where the loads are: segment, k, corners of the tile there, and in the
  // next segment
  const uint64_t step_a = kA == kAlongK ? kTileK * 2 : g.lda * (kTileK * 2);
  const uint64_t step_b = kB == kAlongK ? kTileK * 2 : g.ldb * (kTileK * 2);
  const uint32_t seg_k = g.seg_tiles * kTileK;
  uint32_t seg = t0 / g.seg_tiles, ahead = tiles;
  uint32_t k = (t0 - seg * g.seg_tiles) * kTileK;
  const char *const at_a = reinterpret_cast<const char *>(g.a) + corner<kA>(g.lda, row0, 0);
  const char *const at_b = reinterpret_cast<const char *>(g.b) + corner<kB>(g.ldb, col0, 0);
  const char *pa = at_a + g.a_off[seg] * 2 + corner<kA>(g.lda, 0, k);
  const char *pb = at_b + g.b_off[seg] * 2 + corner<kB>(g.ldb, 0, k);
  uint32_t known = min(seg + 1, kMaxSegs - 1);
  const char *next_a = at_a + g.a_off[known] * 2;
  const char *next_b = at_b + g.b_off[known] * 2;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)ring +
                        __builtin_amdgcn_readfirstlane(wave) * 1024;

  Srd srd_a, srd_b;
  uint32_t left_a, left_b, at;
  auto aim = [&](uint32_t stage) {
    srd_a = LaneA::srd(pa);
    srd_b = LaneB::srd(pb);
    settled(srd_a, srd_b);
    at = lds0 + stage * kStage;
    left_a = ahead && g.ka > k ? g.ka - k : 0;
    left_b = ahead && g.kb > k ? g.kb - k : 0;
  };
  auto load = [&](uint32_t j) {
    if (j < LaneA::kLoads) la.load(j, at, srd_a, left_a);
    else lb.load(j - LaneA::kLoads, at + LaneA::kBytes, srd_b, left_b);
  };
  auto advance = [&]() {
    ahead -= ahead != 0;
    k += kTileK;
    const bool over = k == seg_k;
    k = over ? 0 : k;
    seg += over;
    pa = over ? next_a : pa + step_a;
    pb = over ? next_b : pb + step_b;
  };
  // (outside of the tiles' straight code)
  auto look_ahead = [&]() {
    if (seg < known) return;
    known = min(seg + 1, kMaxSegs - 1);
    next_a = at_a + g.a_off[known] * 2;
    next_b = at_b + g.b_off[known] * 2;
  };

  Acc acc[kSub][kSub];
#pragma unroll
  for (uint32_t i = 0; i < kSub; ++i)
#pragma unroll
    for (uint32_t j = 0; j < kSub; ++j) acc[i][j] = Acc{0.0f, 0.0f, 0.0f, 0.0f};

  // A tile's products, row by row of fragments of A; the next tile's fragments
  // come in behind: B's with the first rows into registers of their own, a row
  // of A's into its own once that is multiplied.
  Half8 fa[kSub], fb[2][kSub];
  auto step = [&](uint32_t stage, uint32_t now) {
    landed<kLoads>();
    aim((stage + 3) & 3);
    const char *s = ring + ((stage + 1) & 3) * kStage;
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
#pragma unroll
      for (uint32_t j = 0; j < kSub; ++j) {
        mfma<T>(fb[now][j], fa[i], acc[i][j]);
        if (j == 1) load(i);
      }
      if (i < kSub / 2) {
        fb[now ^ 1][2 * i] = lb.fragment(s + LaneA::kBytes, 2 * i);
        fb[now ^ 1][2 * i + 1] = lb.fragment(s + LaneA::kBytes, 2 * i + 1);
      }
      fa[i] = la.fragment(s, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    advance();
  };

  static_assert(kLoads == kSub, "a load per row of fragments");
#pragma unroll
  for (uint32_t s = 0; s < 3; ++s) {
    aim(s);
#pragma unroll
    for (uint32_t j = 0; j < kLoads; ++j) load(j);
    advance();
    look_ahead();
  }
  landed<2 * kLoads>();
#pragma unroll
  for (uint32_t i = 0; i < kSub; ++i) {
    fa[i] = la.fragment(ring, i);
    fb[0][i] = lb.fragment(ring + LaneA::kBytes, i);
  }
  // (the compiler's count of reads in flight starts the loop from none)
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  settle();
  uint32_t stage = 0;
  for (uint32_t t = 0; t < tiles; t += 2) {
    step(stage, 0);
    look_ahead();
    step(stage + 1, 1);
    stage ^= 2;
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  settle();
  epi.template run<kTile, kGated>(acc, row0 + wm * (kTile / 2),
                                  col0 + wn * (kGated ? kTile / 4 : kTile / 2), blockIdx.y);
}

// --- what becomes of the results ---------------------------------------------

// A lane's results of a tile of fragments: row, and 8 neighbouring columns.
__device__ __forceinline__ Row8 eight(const Acc &lo, const Acc &hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// put(row, col, v) for every 8 results inside of m rows and n columns, or
// put(row, col, gate, up) for those of a gated product.
template <class Put>
struct Each {
  Put put;
  uint32_t m, n;

  template <uint32_t kTile, bool kGated, uint32_t kSub>
  __device__ __forceinline__ void run(const Acc (&acc)[kSub][kSub], uint32_t row0, uint32_t col0,
                                      uint32_t) const {
    const uint32_t lane = lane_id();
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
      const uint32_t row = row0 + outer_of(i, lane & 15);
      if (row >= m) continue;
#pragma unroll
      for (uint32_t j = 0; j < (kGated ? kSub / 2 : kSub); j += 2) {
        const uint32_t col = col0 + outer_of(j, (lane / 16) * 4);
        if (col >= n) continue;
        if constexpr (kGated)
          put(row, col, eight(acc[i][j], acc[i][j + 1]),
              eight(acc[i][j + kSub / 2], acc[i][j + kSub / 2 + 1]));
        else
          put(row, col, eight(acc[i][j], acc[i][j + 1]));
      }
    }
  }
};

// A part of k: f32 sums to rows of `wide` columns (a gated product's up
// columns behind the gate's), a plane of m rows per part.
struct Parts {
  float *to;
  uint32_t m, n, wide;

  template <uint32_t kTile, bool kGated, uint32_t kSub>
  __device__ __forceinline__ void run(const Acc (&acc)[kSub][kSub], uint32_t row0, uint32_t col0,
                                      uint32_t part) const {
    const uint32_t lane = lane_id();
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
      const uint32_t row = row0 + outer_of(i, lane & 15);
      if (row >= m) continue;
      float *const at = to + ((uint64_t)part * m + row) * wide;
#pragma unroll
      for (uint32_t j = 0; j < kSub; j += 2) {
        const bool up = kGated && j >= kSub / 2;
        const uint32_t col = col0 + outer_of(up ? j - kSub / 2 : j, (lane / 16) * 4);
        if (col >= n) continue;
        *reinterpret_cast<Row8 *>(at + (up ? wide / 2 : 0) + col) = eight(acc[i][j], acc[i][j + 1]);
      }
    }
  }
};

// The parts' sums, in their order, to put.
template <bool kGated, class Put>
__global__ __launch_bounds__(kThreads) void join_parts(const float *__restrict__ parts,
                                                       uint32_t count, uint32_t m, uint32_t n,
                                                       uint32_t wide, Put put) {
  const uint32_t chunks = (n + 7) / 8;
  const uint64_t id = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= (uint64_t)m * chunks) return;
  const uint32_t row = (uint32_t)(id / chunks), col = (uint32_t)(id - (uint64_t)row * chunks) * 8;
  const float *at = parts + (uint64_t)row * wide + col;
  Row8 a = *reinterpret_cast<const Row8 *>(at);
  Row8 b = a;
  if (kGated) b = *reinterpret_cast<const Row8 *>(at + wide / 2);
  for (uint32_t s = 1; s < count; ++s) {
    at += (uint64_t)m * wide;
    a += *reinterpret_cast<const Row8 *>(at);
    if (kGated) b += *reinterpret_cast<const Row8 *>(at + wide / 2);
  }
  if constexpr (kGated) put(row, col, a, b);
  else put(row, col, a);
}

// --- f32 as three 16-bit numbers ---------------------------------------------

// f32 operands are multiplied as sums of three bf16 numbers (8 bits each, so
// x = x0 + x1 + x2 to 2^-25 of x), with the six products whose size is above
// 2^-24 of the whole; sums are f32. The matrix cores multiply bf16 at 16 times
// f32's rate. An infinity or NaN stays in x0.
constexpr uint32_t kPlanes = 3, kPairs = 6;
constexpr uint8_t kPairA[kPairs] = {0, 2, 1, 0, 1, 0}, kPairB[kPairs] = {2, 0, 1, 1, 0, 0};

__device__ __forceinline__ void split(float x, __bf16 out[kPlanes]) {
  __bf16 a = (__bf16)x;
  // (a finite x next to the type's end is not rounded up to infinity)
  if (!__builtin_isfinite((float)a) && __builtin_isfinite(x))
    a = __builtin_bit_cast(__bf16, (uint16_t)(__float_as_uint(x) >> 16));
  const float r = __builtin_isfinite(x) ? x - (float)a : 0.0f;
  out[0] = a;
  out[1] = (__bf16)r;
  out[2] = (__bf16)(r - (float)out[1]);
}

// 8 values of an operand that a kernel here writes for a product here: rows of
// T, or f32 as planes `plane` elements apart.
template <class O>
__device__ __forceinline__ void put_operand(uint16_t *at, uint64_t plane, Row8 v) {
  typedef uint16_t Word8 __attribute__((ext_vector_type(8)));
  if constexpr (sizeof(O) == 4) {
    Word8 w[kPlanes];
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      __bf16 x[kPlanes];
      split(v[e], x);
#pragma unroll
      for (uint32_t p = 0; p < kPlanes; ++p) w[p][e] = __builtin_bit_cast(uint16_t, x[p]);
    }
#pragma unroll
    for (uint32_t p = 0; p < kPlanes; ++p) *reinterpret_cast<Word8 *>(at + p * plane) = w[p];
  } else {
    typedef O Out8 __attribute__((ext_vector_type(8)));
    *reinterpret_cast<Out8 *>(at) = __builtin_convertvector(v, Out8);
  }
}

// --- host side ---------------------------------------------------------------

// An operand as products take it: 16-bit rows on 16 bytes of whole chunks of 8
// (zeros behind the row's own elements), f32 as planes.
struct Matrix {
  const uint16_t *p;
  uint64_t ld, plane;
};

inline uint32_t up8(uint32_t x) { return (x + 7u) & ~7u; }
inline uint64_t planes_of(uint32_t dtype) { return dtype == 0u ? kPlanes : 1u; }
inline uint64_t matrix_bytes(uint32_t dtype, uint64_t rows, uint32_t len) {
  return align_up(rows * up8(len) * 2 * planes_of(dtype), 256);
}

// Longest row of an operand, and most bytes between the rows of one tile:
// lanes' offsets are 31 bits.
constexpr uint32_t kMaxInner = 1u << 20;
constexpr uint64_t kMaxSpan = 1ull << 31;

// Whether a caller's rows can be multiplied where they are. `apart`: rows
// between those of one tile (beside the tile's own).
inline bool in_place(const void *p, uint32_t dtype, uint64_t ld, uint32_t len, uint32_t apart = 0) {
  return dtype != 0u && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0 &&
         len % 8 == 0 && ld < kMaxSpan / 512 && (apart + 256ull) * ld * 2 < kMaxSpan;
}

// Copies of operands that cannot be, all in one launch.
struct PackItem {
  const void *from;
  uint64_t from_ld;
  uint16_t *to;
  uint64_t chunks;  // rows * chunks of 8 of a row
  uint64_t plane;
  uint32_t row_chunks, len;
};
struct Pack3 {
  PackItem item[4];
  uint32_t count;
};
hipError_t launch_pack(const Pack3 &items, uint32_t dtype, hipStream_t stream);

// Takes the next free piece of a workspace (or only counts).
struct Room {
  char *base;
  size_t used = 0;
  void *take(size_t bytes) {
    char *const at = base == nullptr ? nullptr : base + used;
    used += align_up(bytes, 256);
    return at;
  }
};

// The caller's matrix, or room for its copy (added to the list).
inline Matrix operand(const void *p, uint32_t dtype, uint64_t ld, uint32_t rows, uint32_t len,
                      bool stays, Room &room, Pack3 &list) {
  if (stays) return Matrix{static_cast<const uint16_t *>(p), ld, 0};
  const uint32_t wide = up8(len);
  const uint64_t plane = (uint64_t)rows * wide;
  uint16_t *const to = static_cast<uint16_t *>(room.take(matrix_bytes(dtype, rows, len)));
  list.item[list.count++] = PackItem{p, ld, to, (uint64_t)rows * (wide / 8), plane, wide / 8, len};
  return Matrix{to, wide, plane};
}

// How a product of m x n results over `tiles` tiles of k is spread over the
// card. Times in ns, measured at 8192^3: a step of 32 k of a round of 256 x 256
// tiles (one a CU) takes 800, of 128 x 128 tiles (two a CU) 590, and of half
// such a round 350; a round costs about 4000 besides. Parts of k fill the card
// where tiles are few; their sums are written and read once more.
struct Shape {
  uint32_t tile, parts, per_part;
};
Shape plan_shape(uint64_t m, uint64_t n, uint32_t tiles);

inline size_t parts_bytes(const Shape &s, uint64_t m, uint64_t wide) {
  return s.parts > 1 ? s.parts * m * wide * 4 : 0;
}

// Segments of a product: `bases` pairs of offsets, times the pairs of planes.
inline uint32_t seg_tiles_of(uint32_t k) { return (k + 2 * kTileK - 1) / (2 * kTileK) * 2; }
inline uint32_t tiles_of(uint32_t dtype, uint32_t bases, uint32_t k) {
  return seg_tiles_of(k) * bases * (dtype == 0u ? kPairs : 1u);
}

inline Args make_args(uint32_t dtype, const Matrix &a, const Matrix &b, uint32_t m, uint32_t n,
                      uint32_t ka, uint32_t kb, uint32_t bases, const uint64_t *a_base,
                      const uint64_t *b_base, const Shape &s, uint32_t columns) {
  Args g = {};
  g.a = a.p;
  g.b = b.p;
  g.lda = a.ld;
  g.ldb = b.ld;
  g.m = m;
  g.n = n;
  g.ka = ka;
  g.kb = kb;
  g.seg_tiles = seg_tiles_of(ka > kb ? ka : kb);
  g.tiles = tiles_of(dtype, bases, ka > kb ? ka : kb);
  g.per_split = s.per_part;
  g.tiles_m = div_up(m, s.tile);
  g.tiles_n = div_up(columns, s.tile);
  const uint32_t pairs = dtype == 0u ? kPairs : 1u;
  for (uint32_t q = 0; q < pairs; ++q)
    for (uint32_t i = 0; i < bases; ++i) {
      g.a_off[q * bases + i] = (a_base ? a_base[i] : 0) + (pairs > 1 ? kPairA[q] * a.plane : 0);
      g.b_off[q * bases + i] = (b_base ? b_base[i] : 0) + (pairs > 1 ? kPairB[q] * b.plane : 0);
    }
  return g;
}

// Calls f with the element type of results and that of the products.
template <class F>
hipError_t with_types(uint32_t dtype, F &&f) {
  switch (static_cast<Dtype>(dtype)) {
    case Dtype::f32:
      return f(float{}, __bf16{});
    case Dtype::f16:
      return f(_Float16{}, _Float16{});
    default:
      return f(__bf16{}, __bf16{});
  }
}

// C = A B to an epilogue.
template <class T, Side kA, Side kB, bool kGated, class Epilogue>
hipError_t launch_tiles(const Args &g, const Shape &s, const Epilogue &epi, hipStream_t stream) {
  if ((uint64_t)g.tiles_m * g.tiles_n > 0x7FFFFFFFull) return hipErrorInvalidConfiguration;
  const dim3 grid(g.tiles_m * g.tiles_n, s.parts);
  if (s.tile == 256)
    product<T, 256, kA, kB, kGated, Epilogue><<<grid, kThreads, 0, stream>>>(g, epi);
  else
    product<T, 128, kA, kB, kGated, Epilogue><<<grid, kThreads, 0, stream>>>(g, epi);
  return hipGetLastError();
}

// C = A B to put, over parts of k where the shape has some.
template <class T, Side kA, Side kB, bool kGated, class Put>
hipError_t launch_product(const Args &g, const Shape &s, const Put &put, float *parts,
                          hipStream_t stream) {
  if (s.parts == 1)
    return launch_tiles<T, kA, kB, kGated>(g, s, Each<Put>{put, g.m, g.n}, stream);
  const uint32_t wide = up8(g.n) * (kGated ? 2 : 1);
  hipError_t e = launch_tiles<T, kA, kB, kGated>(g, s, Parts{parts, g.m, g.n, wide}, stream);
  if (e != hipSuccess) return e;
  const uint64_t chunks = (uint64_t)g.m * div_up(g.n, 8);
  join_parts<kGated, Put><<<div_up(chunks, kThreads), kThreads, 0, stream>>>(parts, s.parts, g.m, g.n,
                                                                           wide, put);
  return hipGetLastError();
}

// Results of type O to the caller's rows (any element-aligned address).
template <class O>
struct ToRows {
  O *out;
  uint64_t ld;
  uint32_t n;
  __device__ __forceinline__ void operator()(uint32_t row, uint32_t col, Row8 v) const {
    store_pack_tail<O, 8>(out + row * ld, col, n, __builtin_convertvector(v, Pack<O, 8>));
  }
};

}  // namespace mm
}  // namespace seacells
