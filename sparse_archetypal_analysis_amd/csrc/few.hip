// The gated block and the log probabilities for few rows (a serving step), on
// gfx950: bound by reading the weights once, so no tile is staged. 16 rows of
// weights and 16 rows of x meet in one matrix instruction (weights as its
// rows), each lane reading 16 bytes of one row straight from memory, at any
// element alignment; rows of x come from the caches. f32 multiplies in f32.
#include <type_traits>

#include "few.hpp"

namespace seacells {
namespace {

typedef float Acc __attribute__((ext_vector_type(4)));
constexpr uint32_t kWaves = 8;
constexpr uint32_t kThreads = kWaves * kWave;

// c += 16 x 16 products of 4 vectors' length of k; the k of a lane's vector is
// any, as long as it is the same in both.
__device__ __forceinline__ void multiply(Vec<float> w, Vec<float> x, Acc &c) {
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(w[e], x[e], c, 0, 0, 0);
}
__device__ __forceinline__ void multiply(Vec<_Float16> w, Vec<_Float16> x, Acc &c) {
  typedef _Float16 V __attribute__((ext_vector_type(8)));
  c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, w), __builtin_bit_cast(V, x), c, 0, 0,
                                             0);
}
__device__ __forceinline__ void multiply(Vec<__bf16> w, Vec<__bf16> x, Acc &c) {
  typedef __bf16 V __attribute__((ext_vector_type(8)));
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, w), __builtin_bit_cast(V, x), c, 0, 0,
                                              0);
}

// The vector of a row at `at`, zeros from `end` on.
template <class T>
__device__ __forceinline__ Vec<T> load_to(const T *row, uint32_t at, uint32_t end) {
  Vec<T> v;
#pragma unroll
  for (uint32_t j = 0; j < kVec<T>; ++j) v[j] = (T)0.0f;
  return at < end ? load_vec_tail(row, at, end, (T)0.0f) : v;
}

// Products of kW rows of weights a lane (one of a tile of 16 each) and kX
// tiles of 16 rows of x, over the vectors first, first + step, ... of a row's
// kAhead * 4 vectors at a time, then the row's last ones one by one.
template <uint32_t kAhead, class T, uint32_t kW, uint32_t kX>
__device__ __forceinline__ void walk(const T *const (&w)[kW], const T *const (&x)[kX], uint32_t k,
                                     uint32_t first, uint32_t step, Acc (&acc)[kW][kX]) {
  constexpr uint32_t kOne = 4 * kVec<T>, kGroup = kAhead * kOne;
  const uint32_t in = (lane_id() / 16) * kVec<T>;
  const uint32_t groups = k / kGroup;
  for (uint32_t g = first; g < groups; g += step) {
    Vec<T> a[kW][kAhead], b[kX][kAhead];
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u) {
#pragma unroll
      for (uint32_t i = 0; i < kW; ++i) a[i][u] = load_vec(w[i] + g * kGroup + u * kOne + in);
#pragma unroll
      for (uint32_t j = 0; j < kX; ++j) b[j][u] = load_vec(x[j] + g * kGroup + u * kOne + in);
    }
#pragma unroll
    for (uint32_t u = 0; u < kAhead; ++u)
#pragma unroll
      for (uint32_t i = 0; i < kW; ++i)
#pragma unroll
        for (uint32_t j = 0; j < kX; ++j) multiply(a[i][u], b[j][u], acc[i][j]);
  }
  for (uint32_t at = groups * kGroup + first * kOne; at < k; at += step * kOne) {
    Vec<T> a[kW], b[kX];
#pragma unroll
    for (uint32_t i = 0; i < kW; ++i) a[i] = load_to(w[i], at + in, k);
#pragma unroll
    for (uint32_t j = 0; j < kX; ++j) b[j] = load_to(x[j], at + in, k);
#pragma unroll
    for (uint32_t i = 0; i < kW; ++i)
#pragma unroll
      for (uint32_t j = 0; j < kX; ++j) multiply(a[i], b[j], acc[i][j]);
  }
}

// A block has kTiles times 16 rows of weights (gated: of gate and up each) and
// all rows of x; its waves split k and join through the LDS. Two tiles a block
// halve the reads of x, which are as many as the weights' for 32 rows. `per`
// below 16 (one tile): as many rows of weights, the others of the tile read the
// last one again, so that a small matrix occupies every CU (one row of x, 1024 x
// 4096 bf16: 64 blocks 6.6 us, 256 blocks 5.1).
template <class T, uint32_t kX, bool kGated, uint32_t kWaves, uint32_t kTiles>
__global__ __launch_bounds__(kWaves * kWave) void few_product(FewProduct g, uint32_t per) {
  constexpr uint32_t kKinds = kGated ? 2 : 1, kW = kKinds * kTiles, kThreads = kWaves * kWave;
  __shared__ float part[kWaves][kW][kX][256];
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave, i = lane & 15;
  const uint32_t base = blockIdx.x * (kTiles > 1 ? 16 * kTiles : per);
  const T *w[kW], *x[kX];
#pragma unroll
  for (uint32_t q = 0; q < kW; ++q)
    w[q] = static_cast<const T *>(g.w) +
           ((uint64_t)(q / kTiles) * g.rows + min(base + (q % kTiles) * 16 + min(i, per - 1), g.rows - 1)) * g.w_ld;
#pragma unroll
  for (uint32_t t = 0; t < kX; ++t)
    x[t] = static_cast<const T *>(g.x) + (uint64_t)min(t * 16 + i, g.n - 1) * g.x_ld;
  Acc acc[kW][kX] = {};
  walk<(kW > 1 || kX > 2 ? 4 : 8)>(w, x, g.k, wave, kWaves, acc);
  // a lane has rows 4 (lane / 16) + 0..3 of weights and row lane % 16 of x
#pragma unroll
  for (uint32_t q = 0; q < kW; ++q)
#pragma unroll
    for (uint32_t t = 0; t < kX; ++t)
      *reinterpret_cast<Acc *>(&part[wave][q][t][i * 16 + (lane / 16) * 4]) = acc[q][t];
  __syncthreads();
  for (uint32_t id = threadIdx.x; id < kTiles * kX * 256; id += kThreads) {
    const uint32_t in = id & 255, t = (id / 256) % kX, tile = id / 256 / kX;
    const uint32_t token = t * 16 + in / 16, row = base + tile * 16 + (in & 15);
    if (token >= g.n || row >= g.rows || (in & 15) >= per) continue;
    float s[kKinds];
#pragma unroll
    for (uint32_t q = 0; q < kKinds; ++q) {
      s[q] = 0.0f;
#pragma unroll
      for (uint32_t v = 0; v < kWaves; ++v) s[q] += part[v][q * kTiles + tile][t][in];
    }
    T *const out = static_cast<T *>(g.out) + token * g.out_ld + row;
    if constexpr (kGated) {
      if (g.pre != nullptr) {
        T *const pre = static_cast<T *>(g.pre) + token * g.pre_ld + row;
        pre[0] = (T)s[0];
        pre[g.rows] = (T)s[1];
      }
      const float a = g.act == Act::silu   ? act<Act::silu>(s[0])
                      : g.act == Act::gelu ? act<Act::gelu>(s[0])
                                           : act<Act::relu>(s[0]);
      *out = (T)(a * s[1]);
    } else {
      *out = (T)s[0];
    }
  }
}

// A wave takes 16 classes after the other, with all rows of x; a lane keeps of
// its row of x the sums over its classes (4 of 16). Lanes, then waves join; a
// block leaves one slice.
template <class T, uint32_t kX>
__global__ __launch_bounds__(kThreads) void few_sums(FewSums g) {
  __shared__ Sums part[kWaves][kX][16];
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave, i = lane & 15;
  const T *x[kX];
  uint32_t target[kX];
  Sums sums[kX];
#pragma unroll
  for (uint32_t t = 0; t < kX; ++t) {
    const uint32_t row = min(t * 16 + i, g.n - 1);
    x[t] = static_cast<const T *>(g.x) + (uint64_t)row * g.x_ld;
    target[t] = g.targets != nullptr && t * 16 + i < g.n ? (uint32_t)g.targets[row] : ~0u;
    sums[t] = Sums{-kInf, 0.0f, 0.0f};
  }
  const uint32_t tiles = (g.v + 15) / 16;
  for (uint32_t tile = blockIdx.x * kWaves + wave; tile < tiles; tile += gridDim.x * kWaves) {
    const T *w[1] = {static_cast<const T *>(g.table) + (uint64_t)min(tile * 16 + i, g.v - 1) * g.table_ld};
    Acc acc[1][kX] = {};
    walk<(kX > 2 ? 4 : 8)>(w, x, g.d, 0, 1, acc);
    const uint32_t first = tile * 16 + (lane / 16) * 4;
    float bias[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const float b = g.bias != nullptr ? g.bias[min(first + e, g.v - 1)] : 0.0f;
      bias[e] = first + e < g.v ? b : -kInf;
    }
#pragma unroll
    for (uint32_t t = 0; t < kX; ++t) {
      float z[4], m = sums[t].m;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        z[e] = bias[e] == -kInf ? -kInf : acc[0][t][e] + bias[e];
        m = nan_max(m, z[e]);
        if (first + e < g.v && target[t] == first + e) g.at_target[t * 16 + i] = z[e];
      }
      rescale(sums[t], m);
      const float base = m == -kInf ? 0.0f : m;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        const float d = not_below(z[e] - base);
        const float p = exp_neg(d);
        sums[t].s += p;
        sums[t].u = fmaf(d, p, sums[t].u);
      }
    }
  }
#pragma unroll
  for (uint32_t t = 0; t < kX; ++t) {
#pragma unroll
    for (uint32_t step = 16; step <= 32; step *= 2)
      sums[t] = joined(sums[t], Sums{__shfl_xor(sums[t].m, step, kWave), __shfl_xor(sums[t].s, step, kWave),
                                     __shfl_xor(sums[t].u, step, kWave)});
    if (lane < 16) part[wave][t][lane] = sums[t];
  }
  __syncthreads();
  if (threadIdx.x >= kX * 16 || threadIdx.x >= g.n) return;
  Sums a = part[0][threadIdx.x / 16][threadIdx.x & 15];
  for (uint32_t w = 1; w < kWaves; ++w) a = joined(a, part[w][threadIdx.x / 16][threadIdx.x & 15]);
  float *const out = g.sums + (uint64_t)blockIdx.x * 3 * g.n + threadIdx.x;
  out[0] = a.m;
  out[g.n] = a.s;
  out[2 * g.n] = a.u;
}

// Calls f with the count of tiles of 16 rows.
template <class F>
hipError_t with_tiles(uint32_t n, F &&f) {
  if (n <= 16) return f(std::integral_constant<uint32_t, 1>{});
  if (n <= 32) return f(std::integral_constant<uint32_t, 2>{});
  return f(std::integral_constant<uint32_t, 4>{});
}

}  // namespace

hipError_t launch_few_product(const FewProduct &g, bool gated, uint32_t dtype, hipStream_t stream) {
  return with_type(dtype, [&](auto t) {
    return with_tiles(g.n, [&](auto x) {
      constexpr uint32_t kX = decltype(x)::value, kTwo = kX > 2 ? 1 : 2;
      typedef decltype(t) T;
      const uint32_t tiles = div_up(g.rows, 16);
      uint32_t per = 16;
      while (kX == 1 && per > 4 && div_up(g.rows, per) < 256) per /= 2;
      const uint32_t blocks = div_up(g.rows, per);
      // up to two blocks a CU: more waves each; more: two tiles each
      if (gated && tiles < 256)
        few_product<T, kX, true, 16, 1><<<blocks, 16 * kWave, 0, stream>>>(g, per);
      else if (gated && (tiles < 512 || kX == 1))
        few_product<T, kX, true, 8, 1><<<tiles, 8 * kWave, 0, stream>>>(g, 16);
      else if (gated)
        few_product<T, kX, true, 8, kTwo><<<div_up(tiles, kTwo), 8 * kWave, 0, stream>>>(g, 16);
      else if (tiles < 512)
        few_product<T, kX, false, 16, 1><<<blocks, 16 * kWave, 0, stream>>>(g, per);
      else
        few_product<T, kX, false, 8, kTwo><<<div_up(tiles, kTwo), 8 * kWave, 0, stream>>>(g, 16);
      return hipGetLastError();
    });
  });
}

uint32_t few_slices(uint32_t v) {
  const uint32_t blocks = div_up(v, 16 * kWaves);
  return blocks < 512 ? blocks : 512;
}

hipError_t launch_few_sums(const FewSums &g, uint32_t dtype, hipStream_t stream) {
  return with_type(dtype, [&](auto t) {
    return with_tiles(g.n, [&](auto x) {
      few_sums<decltype(t), decltype(x)::value><<<few_slices(g.v), kThreads, 0, stream>>>(g);
      return hipGetLastError();
    });
  });
}

}  // namespace seacells
