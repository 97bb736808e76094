// Matrix products of 16-bit elements on the matrix cores (gfx950): one tiled
// loop for the token model's block and head, with the work on each tile of
// results left to the caller (an Epilogue). Nothing here is exported.
#pragma once

#include <type_traits>
#include <utility>

#include "token.hpp"

namespace seacells {
namespace mm {

// How an operand lies in memory: rows of elements along the product's inner
// index k, or rows (one per k) of elements along its outer index.
enum Side : uint32_t { kAlongK = 0, kAcrossK = 1 };

constexpr uint32_t kMaxSegs = 12;
constexpr uint32_t kTileK = 32;
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
  const uint32_t *only;  // or nullptr: left out where this is 0 (products that may_skip)
};

// The products whose launch the device may leave out: f16's of dh (the check at
// the start of all of them cost bf16's gradients 0.5 to 2 %).
template <class T, Side kA, Side kB>
constexpr bool may_skip = std::is_same<T, _Float16>::value && kA == kAlongK && kB == kAcrossK;

// f(0), f(1), ... as constants.
template <class F, uint32_t... kI>
__device__ __forceinline__ void each_of(F &&f, std::integer_sequence<uint32_t, kI...>) {
  (f(std::integral_constant<uint32_t, kI>{}), ...);
}
template <uint32_t kCount, class F>
__device__ __forceinline__ void each(F &&f) {
  each_of(f, std::make_integer_sequence<uint32_t, kCount>{});
}

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
template <uint32_t kOffset>
__device__ __forceinline__ void load_to_lds(uint32_t lds, const Srd &srd, uint32_t at) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(at), "s"(srd), "n"(kOffset)
               : "m0", "scc");
}
#pragma clang diagnostic pop

// The wait states between a vector instruction's scalar result, should one be
// part of a descriptor, and the loads that use it.
__device__ __forceinline__ void settled(Srd &a, Srd &b) {
  asm volatile("s_nop 4" : "+s"(a), "+s"(b));
}

// Waits until at most kLeft of the wave's loads are in flight (and, kReads, its
// LDS reads are done), then for the block's other waves.
template <uint32_t kLeft, bool kReads>
__device__ __forceinline__ void landed() {
  static_assert(kLeft < 64, "vmcnt");
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (kReads)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLeft) : "memory");
  else
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
// LDS holds two pairs of tiles of 32 k, as 1 KB pieces, one per wave load, 16
// bytes a lane; the order of the 16-byte chunks within a row is what keeps the
// banks apart:
//   along K:  a pair of tiles is loaded as one, rows of 128 bytes (8 chunks, a
//             cache line) per outer index, chunk ^ s(row). 16 lanes of a
//             fragment read rows {0-3, 8-11, 16-19, 24-27} of a pair of tiles of
//             16; s gives them 16 places of the 256 bytes that 2 rows span, and
//             each 8 of them 8 places of 128 bytes.
//   across K: tiles are loaded one by one, rows of kSize elements per k, chunk ^
//             4 (k % 4). A transposing read takes 4 k and 4 chunks' halves: 4
//             times 64 bytes apart.
template <Side kSide, uint32_t kSize>
struct Lane {
  static constexpr bool kPairs = kSide == kAlongK;            // what is loaded at once
  static constexpr uint32_t kPair = kSize * kTileK * 4;       // bytes of a pair of tiles
  static constexpr uint32_t kBytes = 2 * kPair;               // of the ring
  static constexpr uint32_t kLoads = kPair / (kPairs ? 4096 : 8192);  // of a wave at once
  static constexpr uint32_t kStep = kPairs ? 2 * kTileK : kTileK;     // k of them
  static constexpr uint32_t kChunks = kSize / 8;              // of a row across K
  static constexpr uint32_t kRows = 1024 / (kSize * 2);       // k of a wave load across K
  static constexpr uint32_t kReads = kPairs ? 2 : kSize / 64;

  uint32_t at[kLoads];    // byte offsets of the lane's loads behind the tile's corner
  uint32_t k_of;          // the lane's first k (across K: of its first load)
  uint32_t read[kReads];  // byte offsets of the lane's LDS reads: along K per tile of the pair,
                          // across K per two tiles of 16

  // outer: first outer index of the tile; limit: outer indexes that there are.
  // half: which half of the tile's outer indexes the wave multiplies. row_of(r)
  // gives the outer index of LDS row r (kOutside: none) for operands along K.
  template <class RowOf>
  __device__ __forceinline__ void init(uint64_t ld, uint32_t outer, uint32_t limit, uint32_t half,
                                       RowOf row_of) {
    const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
    if constexpr (kPairs) {
      const uint32_t r0 = wave * 8 + lane / 8;
      const uint32_t chunk = (lane & 7) ^ swizzle(r0);
      k_of = chunk * 8;
#pragma unroll
      for (uint32_t j = 0; j < kLoads; ++j) {
        const uint32_t row = row_of(j * 32 + r0);
        at[j] = row == kOutside ? kOutside : (uint32_t)(row * ld * 2 + chunk * 16);
      }
      const uint32_t r = outer_of(0, lane & 15);
      read[0] = (half * (kSize / 2) + r) * 128 + ((lane / 16) ^ swizzle(r)) * 16;
      read[1] = read[0] ^ 64;
    } else {
      const uint32_t row = wave * kRows + lane / kChunks;
      const uint32_t chunk = (lane % kChunks) ^ ((row & 3) * 4);
      const bool in = outer + chunk * 8 < limit;
      k_of = row;
#pragma unroll
      for (uint32_t j = 0; j < kLoads; ++j)
        at[j] = in ? (uint32_t)((j * 4 * kRows + row) * ld * 2 + chunk * 16) : kOutside;
      const uint32_t r = (lane & 15) / 4, q = lane & 3;
#pragma unroll
      for (uint32_t p = 0; p < kReads; ++p) {
        const uint32_t c = (half * (kChunks / 2) + p * 4 + q) ^ (r * 4);
        read[p] = ((lane / 16) * 8 + r) * (kSize * 2) + c * 16;
      }
    }
  }

  static __device__ __forceinline__ uint32_t swizzle(uint32_t row) {
    return ((row >> 1) & 1) + ((row >> 3) & 1) * 2 + (((row >> 4) ^ row) & 1) * 4;
  }

  // The wave's load j. left: k that the operand still has at the descriptor's
  // base (below 1: zeros are loaded).
  template <uint32_t j>
  __device__ __forceinline__ void load(uint32_t lds, const Srd &srd, int32_t left) const {
    const int32_t k = (int32_t)(k_of + (kPairs ? 0 : j * 4 * kRows));
    load_to_lds<j * 4096>(lds, srd, k < left ? at[j] : kOutside);
  }

  // The fragment of one tile of 16 from tile `odd` of the pair at `pair`: 8 k of
  // one outer index.
  template <uint32_t kOdd>
  __device__ __forceinline__ Half8 fragment(const char *pair, uint32_t tile) const {
    typedef __attribute__((address_space(3))) Half4 *At;
    if constexpr (kPairs) {
      return *reinterpret_cast<const Half8 *>(pair + read[kOdd] + (tile / 2) * 4096 + (tile & 1) * 512);
    } else {
      const char *p = pair + kOdd * (kPair / 2) + read[tile / 2] + (tile & 1) * 8;
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

// The rows of a tile of B along K: kTile consecutive ones, or for a gated product
// half of them of the gate and half the up rows `pair` behind them, as many of
// each to a wave's columns.
template <uint32_t kTile, bool kGated>
__device__ __forceinline__ uint32_t b_row(uint32_t r, uint32_t outer, uint32_t limit,
                                          uint32_t pair) {
  if (!kGated) return outer + r < limit ? r : kOutside;
  const uint32_t half = r / (kTile / 2), in = r % (kTile / 2);
  const uint32_t up = in / (kTile / 4);
  const uint32_t row = half * (kTile / 4) + in % (kTile / 4);
  return outer + row < limit ? row + up * pair : kOutside;
}

// A block of 4 waves computes kTile x kTile results, each wave a quarter: of 256
// x 256 (128 KB of LDS) one block a CU, of 128 x 128 (64 KB) two. The LDS holds
// two pairs of tiles of 32 k. While the products of tile t run, the fragments of
// tile t + 1 are read, and loads go out: operands across K one tile at a time,
// into the half that tile t - 1 has left; operands along K a pair at a time, in
// odd t, into the pair that is then read to its end. One or two barriers a pair
// are all that the waves wait for.
// epi.run(acc, row0, col0, whole, part): the wave's results from (row0, col0)
// on, the last of them inside of the whole or not, of part `part` of k.
template <class T, uint32_t kTile, Side kA, Side kB, bool kGated, class Epilogue>
__global__ __launch_bounds__(kThreads, kTile == 256 ? 1 : 2) void product(Args g, Epilogue epi) {
  constexpr uint32_t kPart = kTile / 2;  // rows and columns of a wave
  constexpr uint32_t kSub = kPart / 16;  // in tiles of 16
  typedef Lane<kA, kTile> LaneA;
  typedef Lane<kB, kTile> LaneB;
  // loads that go out with an even and with an odd tile
  constexpr uint32_t kEven = (LaneA::kPairs ? 0 : LaneA::kLoads) + (LaneB::kPairs ? 0 : LaneB::kLoads);
  constexpr uint32_t kOdd = LaneA::kLoads + LaneB::kLoads;
  constexpr bool kAnyPairs = LaneA::kPairs || LaneB::kPairs;
  __shared__ __attribute__((aligned(1024))) char ring[LaneA::kBytes + LaneB::kBytes];
  if constexpr (may_skip<T, kA, kB>) {
    if (g.only != nullptr && *g.only == 0) return;
  }

  const uint32_t wave = threadIdx.x / kWave;
  const uint32_t wm = wave & 1, wn = wave >> 1;
  uint32_t tm, tn;
  tile_of(blockIdx.x, g.tiles_m, g.tiles_n, &tm, &tn);
  const uint32_t row0 = tm * kTile;
  const uint32_t col0 = tn * (kGated ? kPart : kTile);
  const uint32_t t0 = blockIdx.y * g.per_split;
  const uint32_t tiles = min(g.per_split, g.tiles - t0);

  LaneA la;
  LaneB lb;
  la.init(g.lda, row0, g.m, wm, [&](uint32_t r) { return row0 + r < g.m ? r : kOutside; });
  lb.init(g.ldb, col0, g.n, wn,
          [&](uint32_t r) { return b_row<kTile, kGated>(r, col0, g.n, g.n); });

  // Where the loads are: a descriptor of each operand whose base is the tile's
  // corner, how much k it has from there on, and in how many pairs the segment
  // (or the block's part of k) ends. That is looked at between two tiles.
  const uint64_t step_a = LaneA::kPairs ? LaneA::kStep * 2 : g.lda * (LaneA::kStep * 2);
  const uint64_t step_b = LaneB::kPairs ? LaneB::kStep * 2 : g.ldb * (LaneB::kStep * 2);
  const char *const at_a = reinterpret_cast<const char *>(g.a) + corner<kA>(g.lda, row0, 0);
  const char *const at_b = reinterpret_cast<const char *>(g.b) + corner<kB>(g.ldb, col0, 0);
  uint32_t seg = t0 / g.seg_tiles;
  const uint32_t in_seg = t0 - seg * g.seg_tiles;
  uint32_t until = min(g.seg_tiles - in_seg, tiles) / 2, remain = tiles / 2 - until;
  uint64_t base_a = (uint64_t)(at_a + g.a_off[seg] * 2 + corner<kA>(g.lda, 0, in_seg * kTileK));
  uint64_t base_b = (uint64_t)(at_b + g.b_off[seg] * 2 + corner<kB>(g.ldb, 0, in_seg * kTileK));
  int32_t left_a = (int32_t)g.ka - (int32_t)(in_seg * kTileK);
  int32_t left_b = (int32_t)g.kb - (int32_t)(in_seg * kTileK);

  // (addresses have 47 bits: a base's upper word is a descriptor's as it is)
  Srd srd_a, srd_b;
  auto aim_a = [&]() {
    srd_a = Srd{(int)(uint32_t)base_a, (int)(uint32_t)(base_a >> 32), 0x7FFFFFFF, 0x00020000};
  };
  auto aim_b = [&]() {
    srd_b = Srd{(int)(uint32_t)base_b, (int)(uint32_t)(base_b >> 32), 0x7FFFFFFF, 0x00020000};
  };
  auto advance_a = [&]() {
    base_a += step_a;
    left_a -= LaneA::kStep;
    aim_a();
  };
  auto advance_b = [&]() {
    base_b += step_b;
    left_b -= LaneB::kStep;
    aim_b();
  };
  // Behind the loads of a pair: the next segment, or no more of k.
  auto look = [&]() {
    if (--until > 0) return;
    if (remain == 0) {
      left_a = left_b = 0;
      until = 0x7FFFFFFF;
      return;
    }
    ++seg;
    base_a = (uint64_t)(at_a + g.a_off[seg] * 2);
    base_b = (uint64_t)(at_b + g.b_off[seg] * 2);
    left_a = (int32_t)g.ka;
    left_b = (int32_t)g.kb;
    until = min(g.seg_tiles / 2, remain);
    remain -= until;
    aim_a();
    aim_b();
    settled(srd_a, srd_b);
  };

  // Byte offsets: of the pair that is multiplied and of the other, and of the
  // wave's loads.
  uint32_t cur_a = 0, cur_b = LaneA::kBytes;
  uint32_t next_a = LaneA::kPair, next_b = LaneA::kBytes + LaneB::kPair;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)ring +
                        __builtin_amdgcn_readfirstlane(wave) * 1024;
  // load q of those that go out with a tile
  auto load = [&](auto odd, auto which) {
    constexpr uint32_t q = decltype(which)::value;
    constexpr bool is_odd = decltype(odd)::value != 0;
    constexpr uint32_t of_a = is_odd || !LaneA::kPairs ? LaneA::kLoads : 0;
    constexpr uint32_t of_b = is_odd || !LaneB::kPairs ? LaneB::kLoads : 0;
    if constexpr (q < of_a)
      la.template load<q>(lds0 + (is_odd ? cur_a : next_a + LaneA::kPair / 2), srd_a, left_a);
    else if constexpr (q < of_a + of_b)
      lb.template load<q - of_a>(lds0 + (is_odd ? cur_b : next_b + LaneB::kPair / 2), srd_b, left_b);
  };

  Acc acc[kSub][kSub];
#pragma unroll
  for (uint32_t i = 0; i < kSub; ++i)
#pragma unroll
    for (uint32_t j = 0; j < kSub; ++j) acc[i][j] = Acc{0.0f, 0.0f, 0.0f, 0.0f};

  // A tile's products, row by row of fragments of A, with the next tile's
  // fragments and loads between them. An even tile's reads are of its own pair,
  // which loads overwrite next where an operand comes in pairs: they are done
  // before the last rows then, and waited for.
  Half8 fa[2][kSub], fb[2][kSub];
  auto step = [&](auto odd) {
    constexpr uint32_t now = decltype(odd)::value;
    if constexpr (now == 1) landed<kEven, kAnyPairs>();
    else if constexpr (kEven > 0) landed<kOdd, false>();
    else __builtin_amdgcn_sched_barrier(0);
    const char *const from_a = ring + (now ? next_a : cur_a), *const from_b = ring + (now ? next_b : cur_b);
    constexpr uint32_t kOut = now ? kOdd : kEven;
    constexpr uint32_t kPerRow = (kOut + kSub - 1) / kSub;  // loads
    constexpr uint32_t kReads = now == 0 && kAnyPairs ? 3 : 2;
    each<kSub>([&](auto row) {
      constexpr uint32_t i = decltype(row)::value;
      each<kReads>([&](auto which) {
        constexpr uint32_t q = i * kReads + decltype(which)::value;  // B's and A's in turn
        if constexpr (q < 2 * kSub) {
          if constexpr (q % 2 == 0)
            fb[now ^ 1][q / 2] = lb.template fragment<now ^ 1>(from_b, q / 2);
          else
            fa[now ^ 1][q / 2] = la.template fragment<now ^ 1>(from_a, q / 2);
        }
      });
      each<kSub>([&](auto column) {
        constexpr uint32_t j = decltype(column)::value;
        mfma<T>(fb[now][j], fa[now][i], acc[i][j]);
        if constexpr (j == kSub / 4 && kPerRow > 0) load(odd, std::integral_constant<uint32_t, i * kPerRow>{});
        if constexpr (j == 3 * kSub / 4 && kPerRow > 1)
          load(odd, std::integral_constant<uint32_t, i * kPerRow + 1>{});
        if constexpr (i == kSub - 1 && j == kSub - 2) {
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (now == 0 || !LaneA::kPairs) advance_a();
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (i == kSub - 1 && j == kSub - 1) {
          if constexpr (now == 0 || !LaneB::kPairs) advance_b();
          if constexpr (now == 0 || kEven > 0) settled(srd_a, srd_b);
        }
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (now == 0) {
      look();
    } else {
      const uint32_t a = cur_a, b = cur_b;
      cur_a = next_a;
      cur_b = next_b;
      next_a = a;
      next_b = b;
    }
  };
  static_assert(kOdd <= 2 * kSub && kEven <= 2 * kSub, "loads of a row");

  // pairs 0 and 1 along K, tiles 0 to 2 across K
  const std::integral_constant<uint32_t, 0> even;
  const std::integral_constant<uint32_t, 1> odd;
  aim_a();
  aim_b();
  settled(srd_a, srd_b);
  each<kOdd>([&](auto q) { load(odd, q); });  // into the present pair
  if constexpr (kEven > 0) {
    if constexpr (!LaneA::kPairs) advance_a();
    if constexpr (!LaneB::kPairs) advance_b();
    settled(srd_a, srd_b);
    next_a = cur_a;  // (tile 1 belongs to the present pair)
    next_b = cur_b;
    each<kEven>([&](auto q) { load(even, q); });
    next_a = LaneA::kPair;
    next_b = LaneA::kBytes + LaneB::kPair;
  }
  advance_a();
  advance_b();
  settled(srd_a, srd_b);
  look();
  cur_a = next_a;
  cur_b = next_b;
  each<kOdd>([&](auto q) { load(odd, q); });
  cur_a = 0;
  cur_b = LaneA::kBytes;
  if constexpr (!LaneA::kPairs) advance_a();
  if constexpr (!LaneB::kPairs) advance_b();
  settled(srd_a, srd_b);
  landed<kEven + kOdd, false>();
#pragma unroll
  for (uint32_t i = 0; i < kSub; ++i) {
    fa[0][i] = la.template fragment<0>(ring + cur_a, i);
    fb[0][i] = lb.template fragment<0>(ring + cur_b, i);
  }
  // (the compiler's count of reads in flight starts the loop from none)
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  settle();
  for (uint32_t t = 0; t < tiles; t += 2) {
    step(even);
    step(odd);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  settle();
  constexpr uint32_t kWide = kGated ? kPart / 2 : kPart;
  const uint32_t row = row0 + wm * kPart, col = col0 + wn * kWide;
  const bool whole = row + kPart <= g.m && col + kWide <= g.n;
  epi.template run<kGated>(acc, row, col, __builtin_amdgcn_readfirstlane(whole) != 0, blockIdx.y);
}

// --- what becomes of the results ---------------------------------------------

// One result. Read where it is used: left to itself the compiler moves all 256
// out of the accumulation registers first, and has none left to work with.
__device__ __forceinline__ float result(const Acc &acc, uint32_t e) {
  float x;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(x) : "a"(acc[e]));
  return x;
}

// A lane's results of two neighbouring tiles: 8 columns of a row.
__device__ __forceinline__ Row8 eight(const Acc &lo, const Acc &hi) {
  Row8 v;
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) v[e] = result(e < 4 ? lo : hi, e & 3);
  return v;
}

// put<whole>(row, col, v) for every 8 results inside of m rows and n columns, or
// put<whole>(row, col, gate, up) for those of a gated product. whole: all 8 are.
// A Put that reads (Put::Ahead is not void) has ahead<whole>(row, col) called a
// row of fragments before, and its result given to put. (dh of 16384 x 8192 x
// 2048 bf16: 490 us without what it reads and writes, 750 with 1.34 GB of it at
// 5 TB/s; four rows ahead 770.)
template <class Put>
struct Each {
  Put put;
  uint32_t m, n;

  template <bool kGated, bool kWhole, uint32_t kSub>
  __device__ __forceinline__ void go(const Acc (&acc)[kSub][kSub], uint32_t row0,
                                     uint32_t col0) const {
    constexpr uint32_t kChunks = kGated ? kSub / 4 : kSub / 2;
    constexpr bool kReads = !std::is_void<typename Put::Ahead>::value;
    typedef typename std::conditional<kReads, typename Put::Ahead, int>::type Ahead;
    const uint32_t lane = lane_id();
    auto row_of = [&](uint32_t i) { return row0 + outer_of(i, lane & 15); };
    auto col_of = [&](uint32_t q) { return col0 + outer_of(2 * q, (lane / 16) * 4); };
    Ahead next[kChunks];
    auto look = [&](uint32_t i) {
      if constexpr (kReads) {
#pragma unroll
        for (uint32_t q = 0; q < kChunks; ++q)
          next[q] = put.template ahead<kWhole>(kWhole ? row_of(i) : min(row_of(i), m - 1), col_of(q));
      }
    };
    look(0);
    each<kSub>([&](auto index) {
      constexpr uint32_t i = decltype(index)::value;
      Ahead now[kChunks];
      if constexpr (kReads) {
#pragma unroll
        for (uint32_t q = 0; q < kChunks; ++q) now[q] = next[q];
        if constexpr (i + 1 < kSub) look(i + 1);
      }
      const uint32_t row = row_of(i);
      if (!kWhole && row >= m) return;
#pragma unroll
      for (uint32_t q = 0; q < kChunks; ++q) {
        const uint32_t col = col_of(q);
        if (!kWhole && col >= n) continue;
        const Row8 v = eight(acc[i][2 * q], acc[i][2 * q + 1]);
        if constexpr (kGated)
          put.template put<kWhole>(row, col, v,
                                   eight(acc[i][2 * q + kSub / 2], acc[i][2 * q + 1 + kSub / 2]));
        else if constexpr (kReads)
          put.template put<kWhole>(row, col, v, now[q]);
        else
          put.template put<kWhole>(row, col, v);
      }
    });
  }

  template <bool kGated, uint32_t kSub>
  __device__ __forceinline__ void run(const Acc (&acc)[kSub][kSub], uint32_t row0, uint32_t col0,
                                      bool whole, uint32_t) const {
    if (whole) go<kGated, true>(acc, row0, col0);
    else go<kGated, false>(acc, row0, col0);
  }
};

// A part of k: f32 sums to rows of `wide` columns (a gated product's up
// columns behind the gate's), a plane of m rows per part; `add` to what is
// there.
struct Parts {
  float *to;
  uint32_t m, n, wide;
  bool add;

  template <bool kGated, uint32_t kSubM, uint32_t kSubN>
  __device__ __forceinline__ void run(const Acc (&acc)[kSubM][kSubN], uint32_t row0, uint32_t col0,
                                      bool, uint32_t part) const {
    const uint32_t lane = lane_id();
#pragma unroll
    for (uint32_t i = 0; i < kSubM; ++i) {
      const uint32_t row = row0 + outer_of(i, lane & 15);
      if (row >= m) continue;
      float *const at = to + ((uint64_t)part * m + row) * wide;
      Row8 v[kSubN / 2];
      uint32_t col[kSubN / 2];
#pragma unroll
      for (uint32_t j = 0; j < kSubN; j += 2) {
        const bool up = kGated && j >= kSubN / 2;
        const uint32_t c = col0 + outer_of(up ? j - kSubN / 2 : j, (lane / 16) * 4);
        col[j / 2] = c < n ? c + (up ? wide / 2 : 0) : kOutside;
        v[j / 2] = eight(acc[i][j], acc[i][j + 1]);
      }
      if (add) {
        Row8 old[kSubN / 2];
#pragma unroll
        for (uint32_t j = 0; j < kSubN / 2; ++j)  // (all in flight together)
          old[j] = *reinterpret_cast<const Row8 *>(at + (col[j] == kOutside ? 0 : col[j]));
#pragma unroll
        for (uint32_t j = 0; j < kSubN / 2; ++j) v[j] += old[j];
      }
#pragma unroll
      for (uint32_t j = 0; j < kSubN / 2; ++j)
        if (col[j] != kOutside) *reinterpret_cast<Row8 *>(at + col[j]) = v[j];
    }
  }
};

// The parts' sums, in a fixed order, to put: kLanes threads for every 8 results,
// each with every kLanes-th part (1300 x 64 in 32 parts: one thread each 10.7
// us, eight 4.8; 2048 x 256 in 16 6.8 and 10.1).
template <bool kGated, uint32_t kLanes, class Put>
__global__ __launch_bounds__(kThreads) void join_parts(const float *__restrict__ parts,
                                                       uint32_t count, uint32_t m, uint32_t n,
                                                       uint32_t wide, Put put,
                                                       const uint32_t *__restrict__ only) {
  if (only != nullptr && *only == 0) return;
  const uint32_t chunks = (n + 7) / 8, lane = threadIdx.x % kLanes;
  const uint64_t id = (uint64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const bool in = id < (uint64_t)m * chunks;
  const uint32_t row = in ? (uint32_t)(id / chunks) : 0;
  const uint32_t col = in ? (uint32_t)(id - (uint64_t)row * chunks) * 8 : 0;
  const float *at = parts + ((uint64_t)lane * m + row) * wide + col;
  Row8 a = 0.0f, b = 0.0f;
#pragma unroll 4
  for (uint32_t s = lane; s < count; s += kLanes) {
    a += *reinterpret_cast<const Row8 *>(at);
    if (kGated) b += *reinterpret_cast<const Row8 *>(at + wide / 2);
    at += (uint64_t)kLanes * m * wide;
  }
  if constexpr (kLanes > 1) {
#pragma unroll
    for (uint32_t step = 1; step < kLanes; step *= 2)
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        a[e] += __shfl_xor(a[e], step, kWave);
        if (kGated) b[e] += __shfl_xor(b[e], step, kWave);
      }
  }
  if (!in || lane > 0) return;
  if constexpr (kGated)
    put.template put<false>(row, col, a, b);
  else if constexpr (!std::is_void<typename Put::Ahead>::value)
    put.template put<false>(row, col, a, put.template ahead<false>(row, col));
  else
    put.template put<false>(row, col, a);
}

template <bool kGated, class Put>
hipError_t launch_join(const float *parts, uint32_t count, uint32_t m, uint32_t n, uint32_t wide,
                       const Put &put, hipStream_t stream, const uint32_t *only = nullptr) {
  const uint64_t chunks = (uint64_t)m * ((n + 7) / 8);
  if (count >= 8 && chunks < (1u << 15))
    join_parts<kGated, 8><<<(uint32_t)((chunks + kThreads / 8 - 1) / (kThreads / 8)), kThreads, 0, stream>>>(
        parts, count, m, n, wide, put, only);
  else
    join_parts<kGated, 1><<<(uint32_t)((chunks + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
        parts, count, m, n, wide, put, only);
  return hipGetLastError();
}

// --- f32 as three 16-bit numbers ---------------------------------------------

// f32 operands are multiplied as sums of three bf16 numbers (8 bits each, so
// x = x0 + x1 + x2 to 2^-25 of x), with the six products whose size is above
// 2^-24 of the whole; sums are f32. The matrix cores multiply bf16 at 16 times
// f32's rate. An infinity or NaN goes on to x1 and x2, where it is NaN.
constexpr uint32_t kPlanes = 3, kPairs = 6;
constexpr uint8_t kPairA[kPairs] = {0, 2, 1, 0, 1, 0}, kPairB[kPairs] = {2, 0, 1, 1, 0, 0};

__device__ __forceinline__ void split(float x, __bf16 out[kPlanes]) {
  // (a finite x next to the type's end is not rounded up to infinity)
  constexpr float kMost = 0x1.fep127f;  // bf16's largest
  out[0] = (__bf16)__builtin_amdgcn_fmed3f(x, -kMost, kMost);
  const float r = x - (float)out[0];
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
// A row of the workspace's matrices starts on a cache line (8192 x 4096 x 16384
// bf16 780 us, with rows on half lines 930).
inline uint32_t up64(uint32_t x) { return (x + 63u) & ~63u; }
// One that only products here read: and not all rows on the same memory channels
// (8192 x 4096 x 16384 803 us with rows 32 KB apart, 784 with 128 bytes more).
inline uint32_t apart64(uint32_t x) { return up64(x) + (up64(x) % 2048 == 0 ? 64u : 0u); }
inline uint64_t planes_of(uint32_t dtype) { return dtype == 0u ? kPlanes : 1u; }
inline uint64_t matrix_bytes(uint32_t dtype, uint64_t rows, uint32_t len) {
  return align_up(rows * apart64(len) * 2 * planes_of(dtype), 256);
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
  uint64_t to_ld, plane;
  uint32_t row_chunks, len;
};
struct PackList {
  PackItem item[4];
  uint32_t count;
};
hipError_t launch_pack(const PackList &items, uint32_t dtype, hipStream_t stream);

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
                      bool stays, Room &room, PackList &list) {
  if (stays) return Matrix{static_cast<const uint16_t *>(p), ld, 0};
  const uint32_t wide = apart64(len), chunks = up8(len) / 8;
  const uint64_t plane = (uint64_t)rows * wide;
  uint16_t *const to = static_cast<uint16_t *>(room.take(matrix_bytes(dtype, rows, len)));
  list.item[list.count++] = PackItem{p, ld, to, (uint64_t)rows * chunks, wide, plane, chunks, len};
  return Matrix{to, wide, plane};
}

// How a product of m x n results over `tiles` tiles of k is spread over the
// card: the least time by what rounds of blocks take, measured (ns, bf16): of
// 256 x 256 tiles (one a CU) 8000 + 690 a step of 32 k; of 128 x 128 (two a CU)
// 3500 + 440, alone 7000 + 440, with one a CU 5000 + 300. Parts of k fill the card where tiles
// are few; their sums are written and read once more. heavy: the results are
// worked on (10000 and 5000 a round more), in one part of k.
struct Shape {
  uint32_t tile, parts, per_part;
};
Shape plan_shape(uint64_t m, uint64_t n, uint32_t tiles, bool heavy = false);

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
  hipError_t e = launch_tiles<T, kA, kB, kGated>(g, s, Parts{parts, g.m, g.n, wide, false}, stream);
  if (e != hipSuccess) return e;
  return launch_join<kGated>(parts, s.parts, g.m, g.n, wide, put, stream, g.only);
}

// Results of type O to the caller's rows (any element-aligned address).
template <bool kWhole, class O>
__device__ __forceinline__ void put_row(O *row, uint32_t col, uint32_t n, Row8 v) {
  const Pack<O, 8> w = __builtin_convertvector(v, Pack<O, 8>);
  if (kWhole) *reinterpret_cast<Pack<O, 8> *>(row + col) = w;
  else store_pack_tail<O, 8>(row, col, n, w);
}

template <class O>
struct ToRows {
  typedef void Ahead;
  O *out;
  uint64_t ld;
  uint32_t n;
  template <bool kWhole>
  __device__ __forceinline__ void put(uint32_t row, uint32_t col, Row8 v) const {
    put_row<kWhole>(out + row * ld, col, n, v);
  }
};

// f16's range is narrow: what it holds between two products is times a power of
// two, here with its inverse (on the device).
struct Scale {
  float by, back;
  uint32_t past;  // something got past f16 by it (the block's gradient)
};

inline bool is_f16(uint32_t dtype) { return static_cast<Dtype>(dtype) == Dtype::f16; }

// Products of one to the caller's rows.
template <class O>
struct ToScaledRows {
  typedef void Ahead;
  O *out;
  uint64_t ld;
  uint32_t n;
  const Scale *scale;  // or nullptr
  template <bool kWhole>
  __device__ __forceinline__ void put(uint32_t row, uint32_t col, Row8 v) const {
    if (scale != nullptr) v *= scale->back;
    put_row<kWhole>(out + row * ld, col, n, v);
  }
};

}  // namespace mm
}  // namespace seacells
