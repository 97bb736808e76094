// Layer norm and its gradient, with the sums of the weight's and the bias'
// gradient.
//
//   h = (x - mean) rstd                    y = h weight + bias
//   g = d_y weight                         d_x = rstd (g - mean(g) - h mean(g h))
//   d_weight = sum over rows of d_y h      d_bias = sum over rows of d_y
//
// All are bound by memory: forward reads x and writes y (16384 x 4096 bf16
// 48 us, 5.6 TB/s), the gradient reads d_y and x and writes d_x (32768 x 2048
// bf16 with f32 weights 82 us, 4.9 TB/s). A row is read once and stays in registers between
// its statistics and its output; the gradient's column sums stay in the
// registers of the lanes that own the columns, over all rows a block takes.
#include "token.hpp"

namespace seacells {

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kLongThreads = 1024;  // rows that no block can hold
constexpr uint32_t kMaxBlocks = 1u << 20;
// Threads of a forward launch at most: two rounds of the card, so that a
// group's weight and bias serve several rows (60499 x 940 f16 with f32 weights
// 64 -> 49 us, 131072 x 500 bf16 103 -> 69; 1024 to 4096 blocks within 4 %).
constexpr uint32_t kFillThreads = 4096 * kThreads;

// A row of d elements over kStride lanes, kR packs of kN each: x[k] holds the
// elements from (k * kStride + at) * kN, those past the end `fill` (in the
// row's one broken pack its first element, if kRepeat). The broken pack has a
// branch of its own, its elements loaded at clamped places (a branch in each
// load: 4096 bf16 65 us against 50, 2001 64 against 41).
template <class T, uint32_t kN, uint32_t kStride, uint32_t kR, bool kRepeat = false>
__device__ __forceinline__ void load_row(const T *row, uint32_t at, uint32_t d, bool live, T fill,
                                         Pack<T, kN> (&x)[kR]) {
#pragma unroll
  for (uint32_t k = 0; k < kR; ++k) {
    const uint32_t c = (k * kStride + at) * kN;
    x[k] = fill;
    if (live && c + kN <= d) x[k] = *reinterpret_cast<const Pack<T, kN> *>(row + c);
  }
  const uint32_t last = d / kN;  // the broken pack, if there is one
  if (d % kN != 0 && live && at == last % kStride) {
    Pack<T, kN> y;
#pragma unroll
    for (uint32_t j = 0; j < kN; ++j) y[j] = row[last * kN + j < d ? last * kN + j : d - 1];
#pragma unroll
    for (uint32_t j = 0; j < kN; ++j) y[j] = last * kN + j < d ? y[j] : kRepeat ? y[0] : fill;
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k)
      if (k == last / kStride) x[k] = y;
  }
}

// Sums of kN values over the kWaves waves of a row's group in a fixed order,
// the results in every thread. kWaves > 1: the group is the block; buf holds
// kN * kWaves floats, and a caller alternates two of them so that one barrier
// per call is enough.
template <uint32_t kLanes, uint32_t kWaves, uint32_t kN>
__device__ __forceinline__ void row_sums(float (&x)[kN], float *buf) {
#pragma unroll
  for (uint32_t q = 0; q < kN; ++q) x[q] = group_sum<kLanes>(x[q]);
  if constexpr (kWaves > 1) {
    const uint32_t wave = threadIdx.x / kWave;
    if (lane_id() == 0)
#pragma unroll
      for (uint32_t q = 0; q < kN; ++q) buf[q * kWaves + wave] = x[q];
    __syncthreads();
#pragma unroll
    for (uint32_t q = 0; q < kN; ++q) {
      float s = buf[q * kWaves];
#pragma unroll
      for (uint32_t w = 1; w < kWaves; ++w) s += buf[q * kWaves + w];
      x[q] = s;
    }
  }
}

// A sum's mean, rounded to f32: the residuals' sum corrects exactly this number,
// so the product may not be fused into what takes or adds it (the mean was off
// by up to a whole step then).
__device__ __forceinline__ float mean_of(float sum, float inv_d) {
#pragma clang fp contract(off)
  return sum * inv_d;
}

// Sum over the block in a fixed order, the result in every thread.
__device__ __forceinline__ float block_sum(float x, float *lds) {
  x = group_sum<kWave>(x);
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x / kWave] = x;
  __syncthreads();
  float s = 0.0f;
  for (uint32_t w = 0; w < kLongThreads / kWave; ++w) s += lds[w];
  return s;
}

// --- forward ------------------------------------------------------------------

// A row per kLanes lanes (kWaves > 1: per block of kWaves waves), kR vectors
// per lane in registers, weight and bias too over all rows of the group.
template <class T, class W, uint32_t kLanes, uint32_t kWaves, uint32_t kR>
__global__ void __launch_bounds__(kWaves > 1 ? kWaves *kWave : kThreads)
    layer_norm_kernel(const T *x, uint32_t n, uint32_t d, uint64_t x_ld,
                      const W *__restrict__ weight, const W *__restrict__ bias, float eps, T *out,
                      uint64_t out_ld, float *__restrict__ mean, float *__restrict__ rstd) {
  constexpr uint32_t kV = kVec<T>;
  constexpr uint32_t kRow = kLanes * kWaves;  // threads per row
  constexpr uint32_t kGroups = kWaves > 1 ? 1 : kThreads / kLanes;
  __shared__ float buf[2][2 * kWaves];
  const uint32_t at = threadIdx.x % kRow;
  const float inv_d = 1.0f / (float)d;
  Pack<W, kV> w[kR], b[kR];
  load_row<W, kV, kRow, kR>(weight, at, d, weight != nullptr, (W)1.0f, w);
  load_row<W, kV, kRow, kR>(bias, at, d, bias != nullptr, (W)0.0f, b);
  const uint64_t step = (uint64_t)gridDim.x * kGroups;
  // every lane of a wave runs the same rounds: the sums take whole waves
  for (uint64_t i0 = (uint64_t)blockIdx.x * kGroups; i0 < n; i0 += step) {
    const uint64_t i = i0 + threadIdx.x / kRow;
    const bool live = i < n;
    const T *row = x + (live ? i : 0) * x_ld;
    Vec<T> v[kR];
    load_row<T, kV, kRow, kR>(row, at, d, live, (T)0.0f, v);
    float s[1] = {0.0f};
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k)
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) s[0] += (float)v[k][j];
    row_sums<kLanes, kWaves, 1>(s, buf[0]);
    float mu = mean_of(s[0], inv_d);
    // the residuals' sum takes out the rounding of the first one
    float q[2] = {0.0f, 0.0f};
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      const uint32_t c = (k * kRow + at) * kV;
      const bool whole = (k + 1) * kRow * kV <= d;
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) {
        const float t = whole || c + j < d ? (float)v[k][j] - mu : 0.0f;
        q[0] += t * t;
        q[1] += t;
      }
    }
    row_sums<kLanes, kWaves, 2>(q, buf[1]);
    const float shift = q[1] * inv_d;
    const float var = nan_max(q[0] * inv_d - shift * shift, 0.0f);
    mu += shift;
    const float rs = 1.0f / sqrtf(var + eps);
    if (!live) continue;
    T *to = out + i * out_ld;
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      const uint32_t c = (k * kRow + at) * kV;
      Vec<T> y;
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j)
        y[j] = (T)(((float)v[k][j] - mu) * rs * (float)w[k][j] + (float)b[k][j]);
      if (c < d) store_vec_tail<T, true>(to, c, d, y);
    }
    if (at == 0) {
      if (mean != nullptr) mean[i] = mu;
      if (rstd != nullptr) rstd[i] = rs;
    }
  }
}

// Rows beyond a block's registers: a block per row that reads it three times.
template <class T, class W>
__global__ void __launch_bounds__(kLongThreads)
    layer_norm_long_kernel(const T *x, uint32_t n, uint32_t d, uint64_t x_ld,
                           const W *__restrict__ weight, const W *__restrict__ bias, float eps,
                           T *out, uint64_t out_ld, float *__restrict__ mean,
                           float *__restrict__ rstd) {
  __shared__ float lds[kLongThreads / kWave];
  const float inv_d = 1.0f / (float)d;
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T *row = x + i * x_ld;
    float s = 0.0f;
    for (uint32_t c = threadIdx.x; c < d; c += kLongThreads) s += (float)row[c];
    float mu = mean_of(block_sum(s, lds), inv_d);
    float q = 0.0f, r = 0.0f;
    for (uint32_t c = threadIdx.x; c < d; c += kLongThreads) {
      const float t = (float)row[c] - mu;
      q += t * t;
      r += t;
    }
    const float shift = block_sum(r, lds) * inv_d;
    const float var = nan_max(block_sum(q, lds) * inv_d - shift * shift, 0.0f);
    mu += shift;
    const float rs = 1.0f / sqrtf(var + eps);
    // out may be x: a thread writes only what it alone reads
    for (uint32_t c = threadIdx.x; c < d; c += kLongThreads) {
      const float w = weight != nullptr ? (float)weight[c] : 1.0f;
      const float b = bias != nullptr ? (float)bias[c] : 0.0f;
      out[i * out_ld + c] = (T)(((float)row[c] - mu) * rs * w + b);
    }
    if (threadIdx.x == 0) {
      if (mean != nullptr) mean[i] = mu;
      if (rstd != nullptr) rstd[i] = rs;
    }
  }
}

// --- gradient -----------------------------------------------------------------

// Blocks of 8 waves; a row per kLanes lanes of a wave, or per kWaves waves.
// Each lane adds d_y h and d_y of its columns over all rows that its group
// takes; at the end the groups that own the same columns are added in order
// (lanes of a wave by exchange, waves through LDS) into the block's part.
constexpr uint32_t kGradWaves = 8;
constexpr uint32_t kGradThreads = kGradWaves * kWave;

template <class T, class W, uint32_t kLanes, uint32_t kWaves, uint32_t kR>
__global__ void __launch_bounds__(kWaves > kGradWaves ? kWaves *kWave : kGradThreads)
    layer_norm_grad_kernel(const T *d_out, uint64_t d_out_ld, const T *x, uint32_t n, uint32_t d,
                           uint64_t x_ld, const float *__restrict__ mean,
                           const float *__restrict__ rstd, const W *__restrict__ weight, T *d_x,
                           uint64_t d_x_ld, float *__restrict__ part, W *__restrict__ d_weight,
                           W *__restrict__ d_bias) {
  constexpr uint32_t kV = kVec<T>;
  constexpr uint32_t kBlockWaves = kWaves > kGradWaves ? kWaves : kGradWaves;
  constexpr uint32_t kRow = kLanes * kWaves;
  constexpr uint32_t kGroups = kBlockWaves * kWave / kRow;  // rows side by side
  constexpr uint32_t kCols = kR * kRow * kV;                // columns held
  __shared__ float buf[2][2 * kBlockWaves];
  __shared__ float sums[kGroups > 1 ? kCols : 1];
  const uint32_t at = threadIdx.x % kRow, group = threadIdx.x / kRow;
  const float inv_d = 1.0f / (float)d;
  Pack<W, kV> w[kR];
  float sw[kR][kV] = {}, sb[kR][kV] = {};
  load_row<W, kV, kRow, kR>(weight, at, d, weight != nullptr, (W)1.0f, w);
  const uint64_t step = (uint64_t)gridDim.x * kGroups;
  uint32_t round = 0;
  for (uint64_t i0 = (uint64_t)blockIdx.x * kGroups; i0 < n; i0 += step, ++round) {
    const uint64_t i = i0 + group;
    const bool live = i < n;
    const T *row = x + (live ? i : 0) * x_ld, *dy = d_out + (live ? i : 0) * d_out_ld;
    Vec<T> v[kR], g[kR];
    load_row<T, kV, kRow, kR>(dy, at, d, live, (T)0.0f, g);
    load_row<T, kV, kRow, kR, true>(row, at, d, live, (T)0.0f, v);
    const float mu = live ? mean[i] : 0.0f, rs = live ? rstd[i] : 0.0f;
    // (columns past the end have d_y = 0 and add nothing to any sum: their h is
    // another column's, or 0, for mean * rstd may be past f32's range; d_x takes
    // the same h, another one costs 16 registers: 100000 x 543 bf16 148 us for 95)
    float s[2] = {0.0f, 0.0f}, r[kR];
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      r[k] = (k * kRow + at) * kV < d ? rs : 0.0f;
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) {
        const float y = (float)g[k][j], h = ((float)v[k][j] - mu) * r[k];
        const float t = y * (float)w[k][j];
        s[0] += t;
        s[1] += t * h;
        sw[k][j] += y * h;
        sb[k][j] += y;
      }
    }
    if (d_x == nullptr) continue;
    if constexpr (kWaves > 1) {
      // groups of several waves: each its own part of the buffer
      float *mine = buf[round & 1] + 2 * kWaves * group;
#pragma unroll
      for (uint32_t q = 0; q < 2; ++q) s[q] = group_sum<kLanes>(s[q]);
      if (lane_id() == 0) {
        mine[threadIdx.x / kWave % kWaves] = s[0];
        mine[kWaves + threadIdx.x / kWave % kWaves] = s[1];
      }
      __syncthreads();
#pragma unroll
      for (uint32_t q = 0; q < 2; ++q) {
        s[q] = mine[q * kWaves];
#pragma unroll
        for (uint32_t u = 1; u < kWaves; ++u) s[q] += mine[q * kWaves + u];
      }
    } else {
      row_sums<kLanes, 1, 2>(s, nullptr);
    }
    if (!live) continue;
    const float a = s[0] * inv_d, b = s[1] * inv_d;
    T *to = d_x + i * d_x_ld;
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      const uint32_t c = (k * kRow + at) * kV;
      Vec<T> y;
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) {
        const float h = ((float)v[k][j] - mu) * r[k];
        y[j] = (T)(rs * ((float)g[k][j] * (float)w[k][j] - a - h * b));
      }
      if (c < d) store_vec_tail<T, true>(to, c, d, y);
    }
  }
  if (part == nullptr && d_weight == nullptr && d_bias == nullptr) return;

  // part == nullptr: the only block, its sums are the result
#pragma unroll
  for (uint32_t half = 0; half < 2; ++half) {
    float(&acc)[kR][kV] = half == 0 ? sw : sb;
    if constexpr (kLanes < kWave) {
#pragma unroll
      for (uint32_t k = 0; k < kR; ++k)
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j)
          for (uint32_t off = kLanes; off < kWave; off *= 2)
            acc[k][j] += __shfl_xor(acc[k][j], off, kWave);
    }
    if constexpr (kGroups > 1) {
      constexpr uint32_t kPerWave = kLanes < kWave ? kWave / kLanes : 1;
      constexpr uint32_t kTurns = kGroups / kPerWave;  // holders of the same columns
      for (uint32_t turn = 0; turn < kTurns; ++turn) {
        __syncthreads();
        if (group / kPerWave == turn && group % kPerWave == 0) {
#pragma unroll
          for (uint32_t k = 0; k < kR; ++k)
#pragma unroll
            for (uint32_t j = 0; j < kV; ++j) {
              float *to = sums + (k * kV + j) * kRow + at;
              *to = turn == 0 ? acc[k][j] : *to + acc[k][j];
            }
        }
      }
      if (group != (kTurns - 1) * kPerWave) continue;
#pragma unroll
      for (uint32_t k = 0; k < kR; ++k)
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j) acc[k][j] = sums[(k * kV + j) * kRow + at];
    } else if (group != 0) {
      continue;
    }
    W *to = half == 0 ? d_weight : d_bias;
    float *to_part = part == nullptr ? nullptr : part + ((uint64_t)blockIdx.x * 2 + half) * d;
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      const uint32_t c = (k * kRow + at) * kV;
      if (c >= d) continue;
      if (to_part != nullptr) {
        Pack<float, kV> y;
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j) y[j] = acc[k][j];
        store_pack_tail<float, kV>(to_part, c, d, y);
      } else if (to != nullptr) {
        Pack<W, kV> y;
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j) y[j] = (W)acc[k][j];
        store_pack_tail<W, kV>(to, c, d, y);
      }
    }
  }
}

// Rows beyond a block's registers: the column sums in one kernel, d_x (a block
// per row that reads it twice) in another.
template <class T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_long_parts_kernel(const T *__restrict__ d_out, uint64_t d_out_ld,
                                 const T *__restrict__ x, uint32_t n, uint32_t d, uint64_t x_ld,
                                 const float *__restrict__ mean, const float *__restrict__ rstd,
                                 uint32_t rows, float *__restrict__ part) {
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= d) return;
  const uint64_t i0 = (uint64_t)blockIdx.y * rows;
  const uint64_t i1 = i0 + rows < n ? i0 + rows : n;
  float sw = 0.0f, sb = 0.0f;
  for (uint64_t i = i0; i < i1; ++i) {
    const float dy = (float)d_out[i * d_out_ld + c];
    sw += dy * (((float)x[i * x_ld + c] - mean[i]) * rstd[i]);
    sb += dy;
  }
  part[((uint64_t)blockIdx.y * 2) * d + c] = sw;
  part[((uint64_t)blockIdx.y * 2 + 1) * d + c] = sb;
}

template <class T, class W>
__global__ void __launch_bounds__(kLongThreads)
    layer_norm_long_dx_kernel(const T *d_out, uint64_t d_out_ld, const T *x, uint32_t n,
                              uint32_t d, uint64_t x_ld, const float *__restrict__ mean,
                              const float *__restrict__ rstd, const W *__restrict__ weight, T *d_x,
                              uint64_t d_x_ld) {
  __shared__ float lds[kLongThreads / kWave];
  const float inv_d = 1.0f / (float)d;
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T *row = x + i * x_ld, *dy = d_out + i * d_out_ld;
    const float mu = mean[i], rs = rstd[i];
    float s = 0.0f, q = 0.0f;
    for (uint32_t c = threadIdx.x; c < d; c += kLongThreads) {
      const float w = weight != nullptr ? (float)weight[c] : 1.0f;
      const float g = (float)dy[c] * w, h = ((float)row[c] - mu) * rs;
      s += g;
      q += g * h;
    }
    const float a = block_sum(s, lds) * inv_d, b = block_sum(q, lds) * inv_d;
    // d_x may be either input: a thread writes only what it alone reads
    for (uint32_t c = threadIdx.x; c < d; c += kLongThreads) {
      const float w = weight != nullptr ? (float)weight[c] : 1.0f;
      const float g = (float)dy[c] * w, h = ((float)row[c] - mu) * rs;
      d_x[i * d_x_ld + c] = (T)(rs * (g - a - h * b));
    }
  }
}

// The parts of 64 columns: 16 waves take every 16th part, their sums are added
// in order.
constexpr uint32_t kJoinWaves = 16;

template <class W>
__global__ void __launch_bounds__(kJoinWaves *kWave)
    layer_norm_join_kernel(const float *__restrict__ part, uint32_t parts, uint32_t d,
                           W *__restrict__ d_weight, W *__restrict__ d_bias) {
  constexpr uint32_t kUnroll = 8;
  __shared__ float sums[kJoinWaves][kWave];
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
  const uint64_t c = (uint64_t)blockIdx.x * kWave + lane, width = 2 * (uint64_t)d;
  float s = 0.0f;
  if (c < width) {
    for (uint32_t p = wave; p < parts; p += kJoinWaves * kUnroll) {
      float y[kUnroll];
#pragma unroll
      for (uint32_t u = 0; u < kUnroll; ++u) {
        const uint32_t q = p + u * kJoinWaves;
        y[u] = q < parts ? part[q * width + c] : 0.0f;
      }
#pragma unroll
      for (uint32_t u = 0; u < kUnroll; ++u) s += y[u];
    }
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= width) return;
#pragma unroll
  for (uint32_t w = 1; w < kJoinWaves; ++w) s += sums[w][lane];
  W *to = c < d ? d_weight : d_bias;
  if (to != nullptr) to[c < d ? c : c - d] = (W)s;
}

// --- choice of the group --------------------------------------------------------

template <uint32_t kLanes_, uint32_t kWaves_, uint32_t kR_>
struct Group {
  static constexpr uint32_t lanes = kLanes_, waves = kWaves_, vecs = kR_;
  static constexpr uint32_t holds = kLanes_ * kWaves_ * kR_;  // vectors of 16 bytes
};

// f(Group) with the smallest group that holds `vecs` vectors: two vectors per
// lane, then more lanes (a reduction over half the lanes serves twice the
// rows: 131072 x 500 bf16 69 -> 59 us), then more vectors, then more waves.
// Forward, a lane holds up to 4 vectors (weight and bias beside them).
template <class F>
bool forward_group(uint32_t vecs, F &&f) {
  if (vecs <= 8) f(Group<8, 1, 1>{});
  else if (vecs <= 16) f(Group<8, 1, 2>{});
  else if (vecs <= 32) f(Group<16, 1, 2>{});
  else if (vecs <= 64) f(Group<32, 1, 2>{});
  else if (vecs <= 128) f(Group<64, 1, 2>{});
  else if (vecs <= 256) f(Group<64, 1, 4>{});
  else if (vecs <= 512) f(Group<64, 4, 2>{});
  else if (vecs <= 1024) f(Group<64, 4, 4>{});
  else if (vecs <= 2048) f(Group<64, 16, 2>{});
  else if (vecs <= 4096) f(Group<64, 16, 4>{});
  else return false;
  return true;
}

template <class F>
bool grad_group(uint32_t vecs, F &&f) {
  if (vecs <= 8) f(Group<8, 1, 1>{});
  else if (vecs <= 16) f(Group<8, 1, 2>{});
  else if (vecs <= 32) f(Group<16, 1, 2>{});
  else if (vecs <= 64) f(Group<32, 1, 2>{});
  else if (vecs <= 128) f(Group<64, 1, 2>{});
  else if (vecs <= 256) f(Group<64, 1, 4>{});
  else if (vecs <= 512) f(Group<64, 2, 4>{});
  else if (vecs <= 1024) f(Group<64, 4, 4>{});
  else if (vecs <= 2048) f(Group<64, 8, 4>{});
  else if (vecs <= 4096) f(Group<64, 16, 4>{});
  else return false;
  return true;
}

uint32_t least(uint32_t a, uint32_t b) { return a < b ? a : b; }
uint32_t capped(uint64_t blocks) { return (uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks); }

}  // namespace

hipError_t launch_layer_norm(const void *x, uint32_t dtype, uint32_t n, uint32_t d, uint64_t x_ld,
                             const void *weight, const void *bias, uint32_t weight_type, float eps,
                             void *out, uint64_t out_ld, float *mean, float *rstd,
                             hipStream_t stream) {
  if (n == 0) return hipSuccess;
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto wt) {
      using W = decltype(wt);
      auto launch = [&](auto kernel, uint32_t blocks, uint32_t threads) {
        hipLaunchKernelGGL(kernel, dim3(blocks), dim3(threads), 0, stream,
                           static_cast<const T *>(x), n, d, x_ld, static_cast<const W *>(weight),
                           static_cast<const W *>(bias), eps, static_cast<T *>(out), out_ld, mean,
                           rstd);
      };
      const bool held = forward_group(div_up(d, kVec<T>), [&](auto g) {
        using G = decltype(g);
        constexpr uint32_t threads = G::waves > 1 ? G::waves * kWave : kThreads;
        constexpr uint32_t rows = G::waves > 1 ? 1 : kThreads / G::lanes;
        launch(layer_norm_kernel<T, W, G::lanes, G::waves, G::vecs>, least(div_up(n, rows), kFillThreads / threads),
               threads);
      });
      if (!held) launch(layer_norm_long_kernel<T, W>, capped(n), kLongThreads);
      return hipGetLastError();
    };
    return weight_type == (uint32_t)Dtype::f32 ? go(float{}) : go(t);
  });
}

// Parts: a block of 8 rows or more, up to one per compute unit, or two where a
// lane holds up to 2 vectors and registers leave room for both (100000 x 130
// f32 74 -> 52 us; 32768 x 2048 bf16, 4 vectors, 82 -> 90 with two).
constexpr uint32_t kMaxParts = 512;

NormGradPlan plan_layer_norm_grad(uint32_t n, uint32_t d) {
  NormGradPlan p{};
  const uint32_t parts = div_up(n, 8);
  p.parts = parts < kMaxParts ? parts : kMaxParts;
  p.ws_bytes = (size_t)p.parts * 2 * d * sizeof(float);
  return p;
}

hipError_t launch_layer_norm_grad(const NormGradPlan &plan, const void *d_out, uint64_t d_out_ld,
                                  const void *x, uint32_t dtype, uint32_t n, uint32_t d,
                                  uint64_t x_ld, const float *mean, const float *rstd,
                                  const void *weight, uint32_t weight_type, void *d_x,
                                  uint64_t d_x_ld, void *d_weight, void *d_bias, void *ws,
                                  hipStream_t stream) {
  float *part = static_cast<float *>(ws);
  const bool sums = d_weight != nullptr || d_bias != nullptr;
  if (!sums && (d_x == nullptr || n == 0)) return hipSuccess;
  return with_type(dtype, [&](auto t) -> hipError_t {
    using T = decltype(t);
    auto go = [&](auto wt) -> hipError_t {
      using W = decltype(wt);
      const T *dy = static_cast<const T *>(d_out), *xs = static_cast<const T *>(x);
      W *to_w = static_cast<W *>(d_weight), *to_b = static_cast<W *>(d_bias);
      uint32_t parts = plan.parts;
      hipError_t e = hipSuccess;
      const bool held = n > 0 && grad_group(div_up(d, kVec<T>), [&](auto g) {
        using G = decltype(g);
        constexpr uint32_t waves = G::waves > kGradWaves ? G::waves : kGradWaves;
        constexpr uint32_t rows = waves * kWave / (G::lanes * G::waves);
        const uint32_t all = div_up(n, rows);
        parts = least(all, G::vecs > 2 ? least(plan.parts, kMaxParts / 2) : plan.parts);
        const bool alone = parts == 1;
        hipLaunchKernelGGL((layer_norm_grad_kernel<T, W, G::lanes, G::waves, G::vecs>),
                           dim3(parts), dim3(waves * kWave), 0, stream, dy, d_out_ld, xs, n, d,
                           x_ld, mean, rstd, static_cast<const W *>(weight), static_cast<T *>(d_x),
                           d_x_ld, sums && !alone ? part : nullptr, alone ? to_w : nullptr,
                           alone ? to_b : nullptr);
        e = hipGetLastError();
      });
      if (e != hipSuccess) return e;
      if (!held && n > 0) {
        if (sums) {  // before d_x, which may overwrite d_out or x
          hipLaunchKernelGGL((layer_norm_long_parts_kernel<T>), dim3(div_up(d, kThreads), parts),
                             dim3(kThreads), 0, stream, dy, d_out_ld, xs, n, d, x_ld, mean, rstd,
                             div_up(n, parts), part);
          if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        if (d_x != nullptr) {
          hipLaunchKernelGGL((layer_norm_long_dx_kernel<T, W>), dim3(capped(n)),
                             dim3(kLongThreads), 0, stream, dy, d_out_ld, xs, n, d, x_ld, mean,
                             rstd, static_cast<const W *>(weight), static_cast<T *>(d_x), d_x_ld);
          if ((e = hipGetLastError()) != hipSuccess) return e;
        }
      }
      if (sums && !(held && parts == 1)) {
        hipLaunchKernelGGL((layer_norm_join_kernel<W>), dim3(div_up(2 * (uint64_t)d, kWave)),
                           dim3(kJoinWaves * kWave), 0, stream, part, parts, d, to_w, to_b);
        e = hipGetLastError();
      }
      return e;
    };
    return weight_type == (uint32_t)Dtype::f32 ? go(float{}) : go(t);
  });
}

}  // namespace seacells
