// Log probabilities straight from hidden rows and a class table, and their
// gradient, on gfx950: a product of x [n, d] and table [v, d] on the matrix
// cores (mm.hpp) whose results z = x table^T + bias never reach memory as
// logits.
//
// Forward: a wave keeps of its tile's rows the maximum, sum e^(z - m) and
// sum (z - m) e^(z - m); the target's z is the one result that is written.
// A second kernel joins the slices of a row.
//
// Backward, in pieces of the classes: z again, d_z from it and the rows'
// figures, to a buffer of one piece (16 bits; f32: three bf16), then
// d_table's rows of the piece, finished, and the piece's part of d_x, kept in
// f32 between pieces. d_bias is summed from d_z before its rounding.
#include "few.hpp"
#include "mm.hpp"

namespace seacells {
namespace {

using namespace mm;

// z of a lane's results in one row: with the bias, -inf for masked classes
// (whatever their rows hold) and behind the last class. kPlain: no bias, and
// the wave's columns are all there.
template <bool kPlain, uint32_t kSub>
struct Logits {
  float bias[kPlain ? 1 : kSub][4];

  __device__ __forceinline__ void load(const float *from, uint32_t col0, uint32_t n) {
    if (kPlain) return;
#pragma unroll
    for (uint32_t j = 0; j < kSub; ++j) {
      const uint32_t col = col0 + outer_of(j, (lane_id() / 16) * 4);
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) {
        const float b = from != nullptr ? from[min(col + e, n - 1)] : 0.0f;
        bias[j][e] = col + e < n ? b : -kInf;
      }
    }
  }
  __device__ __forceinline__ float of(const Acc &acc, uint32_t j, uint32_t e) const {
    const float z = result(acc, e);
    return kPlain ? z : bias[j][e] == -kInf ? -kInf : z + bias[j][e];
  }
};

// Epilogue of the forward product. A slice is a wave's columns.
struct RowSums {
  const float *bias;
  const int32_t *targets;  // of the first row here
  float *sums;             // [slice][3][rows]
  float *at_target;        // [rows]
  uint32_t rows, n;

  template <bool kPlain, uint32_t kSub>
  __device__ __forceinline__ void go(const Acc (&acc)[kSub][kSub], uint32_t row0,
                                     uint32_t col0) const {
    const uint32_t lane = lane_id();
    Logits<kPlain, kSub> logits;
    logits.load(bias, col0, n);
    float *const out = sums + (uint64_t)(col0 / (kSub * 16)) * 3 * rows;
    uint32_t in[kSub];  // the target's place among the wave's columns
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
      const uint32_t row = row0 + outer_of(i, lane & 15);
      in[i] = targets != nullptr ? (uint32_t)targets[min(row, rows - 1)] - col0 : ~0u;
    }
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
      const uint32_t row = row0 + outer_of(i, lane & 15);
      float z[kSub][4], m = -kInf;
#pragma unroll
      for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          z[j][e] = logits.of(acc[i][j], j, e);
          m = nan_max(m, z[j][e]);
        }
      m = nan_max(m, __shfl_xor(m, 16, kWave));
      m = nan_max(m, __shfl_xor(m, 32, kWave));
      const float base = m == -kInf ? 0.0f : m;
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          // (in powers of 2; the difference first, so that any z of f32 will do)
          const float t = not_below((z[j][e] - base) * kLog2E);
          const float x = __builtin_amdgcn_exp2f(t);
          s[e] += x;
          u[e] = fmaf(t, x, u[e]);
        }
      float s1 = (s[0] + s[1]) + (s[2] + s[3]), u1 = ((u[0] + u[1]) + (u[2] + u[3])) * kLn2;
      s1 += __shfl_xor(s1, 16, kWave);
      u1 += __shfl_xor(u1, 16, kWave);
      s1 += __shfl_xor(s1, 32, kWave);
      u1 += __shfl_xor(u1, 32, kWave);
      if (lane < 16 && row < rows) {
        out[row] = m;
        out[(uint64_t)rows + row] = s1;
        out[2ull * rows + row] = u1;
      }
      if (in[i] < kSub * 16 && row < rows && col0 + in[i] < n) {
#pragma unroll
        for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e)
            if (in[i] == outer_of(j, (lane / 16) * 4) + e) at_target[row] = z[j][e];
      }
    }
  }

  template <bool kGated, uint32_t kSub>
  __device__ __forceinline__ void run(const Acc (&acc)[kSub][kSub], uint32_t row0, uint32_t col0,
                                      bool whole, uint32_t) const {
    if (whole && bias == nullptr) go<true>(acc, row0, col0);
    else go<false>(acc, row0, col0);
  }
};

// Rows' slices joined, kLanes threads a row; the last block reports targets past
// the classes. Where rows are few the slices of one want a whole block (4 rows
// of 1024 slices 50 us with 16 threads a row, 5 with 256; 8192 rows 40 us and
// 16 threads read whole lines of 16 rows).
template <uint32_t kLanes>
__global__ __launch_bounds__(kThreads) void join_rows(const float *__restrict__ sums,
                                                      const float *__restrict__ at_target,
                                                      uint32_t slices, uint32_t rows, uint32_t v,
                                                      const int32_t *__restrict__ targets,
                                                      float *__restrict__ logp,
                                                      float *__restrict__ entropy,
                                                      float *__restrict__ stats,
                                                      const int32_t *__restrict__ all_targets,
                                                      uint32_t all, uint32_t *__restrict__ status) {
  if (blockIdx.x == gridDim.x - 1) {
    if (status != nullptr) report_ids<kThreads>(all_targets, all, v, status);
    return;
  }
  constexpr uint32_t kRows = kThreads / kLanes;
  __shared__ Sums part[kLanes][kRows + (kRows > 1)];
  const uint32_t in = threadIdx.x % kRows, lane = threadIdx.x / kRows;
  const uint32_t row = blockIdx.x * kRows + in;
  Sums a = {-kInf, 0.0f, 0.0f};
  if (row < rows)
    for (uint32_t k = lane; k < slices; k += kLanes) {
      const float *const p = sums + (uint64_t)k * 3 * rows + row;
      a = joined(a, Sums{p[0], p[rows], p[2ull * rows]});
    }
#pragma unroll
  for (uint32_t half = kLanes / 2; half > 0; half /= 2) {
    if (lane < 2 * half) part[lane][in] = a;
    __syncthreads();
    if (lane < half) a = joined(a, part[lane + half][in]);
    __syncthreads();
  }
  if (lane > 0 || row >= rows) return;
  const bool none = a.m == -kInf;
  // NaN: a row that holds NaN or +inf has no distribution
  const float m = a.m == kInf ? __builtin_nanf("") : a.m;
  const float ls = none ? 0.0f : logf(a.s) + (m - m);
  if (stats != nullptr) {
    stats[2ull * row] = m;
    stats[2ull * row + 1] = ls;
  }
  if (entropy != nullptr) entropy[row] = none ? 0.0f : ls - a.u / a.s;
  if (logp != nullptr) {
    const int32_t t = targets[row];
    const bool known = t >= 0 && (uint32_t)t < v;
    logp[row] = !known ? 0.0f : none ? -kInf : at_target[row] - m - ls;
  }
}

// --- backward ------------------------------------------------------------------

// Targets past the classes, by one block, where the first product's first block
// does not look for them beside its other work.
constexpr uint32_t kPrepare = 1024;
__global__ __launch_bounds__(kPrepare) void report_targets(const int32_t *__restrict__ targets,
                                                           uint32_t n, uint32_t v,
                                                           uint32_t *__restrict__ status) {
  if (targets != nullptr) report_ids<kPrepare>(targets, n, v, status);
  else if (threadIdx.x == 0) *status = 0u;
}

// f16 holds 2^-24 to 2^15; d_z of a mean over rows is far below that. It is
// kept times a power of two that takes its bound, max |d_logp| + 17 |d_entropy|
// (p |log p + H| <= 0.4 + log v), to below 2^15. Values that d_z does not
// depend on choose nothing: d_logp of ignored targets, both of rows with nothing
// left or without a distribution. Targets past the classes are reported in the
// same pass. The maximum is of 1/32 of the bound, so that it is finite for any
// finite gradients. One block up to kOneBlock rows, more blocks in two launches
// (gradient of 64 x 1300, us in one and two: 3001 rows 45.2 and 46.4, 8192 rows
// 57.2 and 54.4, 131072 rows 498 and 387).
constexpr uint32_t kOneBlock = 4096, kScaleBlocks = 128;
struct Looked {
  float most;
  uint32_t bad;
};

// By one thread, from the maximum over all rows.
__device__ __forceinline__ void put_scale(Looked all, Scale *__restrict__ scale,
                                          uint32_t *__restrict__ status) {
  *status = all.bad ? kFlagBadIndex : 0u;
  // 32 most < 2^(e + 1), e <= 132; powers from 2^-118 to 2^100 keep both factors normal
  int e = (int)((__float_as_uint(all.most) >> 23) & 255u) - 122;
  e = all.most > 0.0f ? min(14 - e, 100) : 0;
  scale->by = __uint_as_float((uint32_t)(e + 127) << 23);
  scale->back = __uint_as_float((uint32_t)(127 - e) << 23);
}

__global__ __launch_bounds__(kPrepare) void scale_rows(const int32_t *__restrict__ targets,
                                                       const float *__restrict__ stats,
                                                       const float *__restrict__ d_logp,
                                                       const float *__restrict__ d_entropy,
                                                       uint32_t n, uint32_t v,
                                                       Looked *__restrict__ parts,
                                                       Scale *__restrict__ scale,
                                                       uint32_t *__restrict__ status) {
  float most = 0.0f;
  bool bad = false;
#pragma unroll 4
  for (uint64_t i = blockIdx.x * kPrepare + threadIdx.x; i < n; i += gridDim.x * kPrepare) {
    const bool left = stats[2 * i] > -kInf;  // (false for NaN)
    const int32_t target = targets != nullptr ? targets[i] : -1;
    const float g = d_logp != nullptr ? fabsf(d_logp[i]) / 32.0f : 0.0f;
    const float h = d_entropy != nullptr ? fabsf(d_entropy[i]) * (17.0f / 32.0f) : 0.0f;
    const float x = ((uint32_t)target < v ? g : 0.0f) + h;
    most = left && x < kInf ? fmaxf(most, x) : most;
    bad |= target >= (int32_t)v;
  }
  most = group_max<kWave>(most);
  __shared__ float wave_most[kPrepare / kWave];
  if (lane_id() == 0) wave_most[threadIdx.x / kWave] = most;
  const bool any = __syncthreads_or(bad);
  if (threadIdx.x != 0) return;
  for (uint32_t w = 1; w < kPrepare / kWave; ++w) most = fmaxf(most, wave_most[w]);
  if (gridDim.x > 1) parts[blockIdx.x] = Looked{most, any};
  else put_scale(Looked{most, any}, scale, status);
}

__global__ __launch_bounds__(kWave) void join_scale(const Looked *__restrict__ parts, uint32_t count,
                                                    Scale *__restrict__ scale,
                                                    uint32_t *__restrict__ status) {
  float most = 0.0f;
  bool bad = false;
  for (uint32_t i = threadIdx.x; i < count; i += kWave) {
    most = fmaxf(most, parts[i].most);
    bad |= parts[i].bad != 0;
  }
  most = group_max<kWave>(most);
  const bool any = __any(bad);
  if (threadIdx.x == 0) put_scale(Looked{most, any}, scale, status);
}

hipError_t launch_scale(const LossGradCall &c, Looked *parts, Scale *scale, uint32_t *status,
                        hipStream_t stream) {
  const uint32_t blocks = c.n <= kOneBlock ? 1 : min(div_up(c.n, kPrepare), kScaleBlocks);
  scale_rows<<<blocks, kPrepare, 0, stream>>>(c.targets, c.stats, c.d_logp, c.d_entropy, c.n, c.v, parts,
                                              scale, status);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1) return e;
  join_scale<<<1, kWave, 0, stream>>>(parts, blocks, scale, status);
  return hipGetLastError();
}

// Epilogue of the backward's first product: d_z of a piece of the classes.
// With lp = log p: d_z = g [target] - p (g + h H + h lp).
constexpr float kLarge = 0x1p120f;
template <class O>
struct PutDz {
  const float *bias;  // of the piece
  const int32_t *targets;
  const float *stats, *entropy, *d_logp, *d_entropy;
  const Scale *scale;  // or nullptr
  uint16_t *dz;
  uint64_t ld, plane;
  float *column_sums;  // [half tiles of rows][ld], or nullptr
  uint32_t rows, n, first, classes;
  uint32_t *status;  // or nullptr: not reported here

  template <bool kPlain, uint32_t kSub>
  __device__ __forceinline__ void go(const Acc (&acc)[kSub][kSub], uint32_t row0,
                                     uint32_t col0) const {
    const uint32_t lane = lane_id();
    Logits<kPlain, kSub> logits;
    logits.load(bias, col0, n);
    float sum[kSub][4];
#pragma unroll
    for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) sum[j][e] = 0.0f;
    const float by = scale != nullptr ? scale->by : 1.0f;
    // the rows' figures, all in flight together
    float m[kSub], ls[kSub], g[kSub], h[kSub], gh[kSub];
    uint32_t hit[kSub];
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
      const uint32_t r = min(row0 + outer_of(i, lane & 15), rows - 1);
      m[i] = stats[2ull * r];
      ls[i] = stats[2ull * r + 1];
      hit[i] = targets != nullptr ? (uint32_t)targets[r] : ~0u;
      g[i] = d_logp != nullptr ? d_logp[r] : 0.0f;
      h[i] = d_entropy != nullptr ? d_entropy[r] : 0.0f;
      gh[i] = d_entropy != nullptr ? entropy[r] : 0.0f;
    }
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
      g[i] = hit[i] < classes ? g[i] : 0.0f;
      if (m[i] == -kInf) g[i] = h[i] = 0.0f;  // nothing left: 0, whatever they hold
      gh[i] = m[i] == m[i] ? fmaf(h[i], gh[i], g[i]) : m[i];  // no distribution: NaN
      ls[i] *= kLog2E;  // (log p in powers of 2)
      h[i] *= kLn2;
      hit[i] -= first;
      if (bias != nullptr && hit[i] < n && bias[hit[i]] == -kInf) hit[i] = ~0u;  // masked
      hit[i] = hit[i] < n ? hit[i] - col0 : ~0u;
    }
#pragma unroll
    for (uint32_t i = 0; i < kSub; ++i) {
      const uint32_t row = row0 + outer_of(i, lane & 15);
      const bool in_row = row < rows;
      float d[kSub][4];
#pragma unroll
      for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const float lp = not_below(fmaf(logits.of(acc[i][j], j, e) - m[i], kLog2E, -ls[i]));
          d[j][e] = -__builtin_amdgcn_exp2f(lp) * fmaf(h[i], lp, gh[i]);
        }
      if (hit[i] < kSub * 16) {
#pragma unroll
        for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e)
            if (hit[i] == outer_of(j, (lane / 16) * 4) + e) d[j][e] += g[i];
      }
      // 0 times what is not finite (200 |h| may be past f32): masked classes stay at 0
      if (!kPlain && __any(!(fabsf(gh[i]) < kLarge && fabsf(h[i]) < kLarge))) {
#pragma unroll
        for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e)
            if (logits.bias[j][e] == -kInf && m[i] == m[i]) d[j][e] = 0.0f;
      }
      if (column_sums != nullptr && in_row) {
#pragma unroll
        for (uint32_t j = 0; j < kSub; ++j)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) sum[j][e] += d[j][e];
      }
#pragma unroll
      for (uint32_t j = 0; j < kSub; j += 2) {
        const uint32_t col = col0 + outer_of(j, (lane / 16) * 4);
        Row8 v;
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e) v[e] = d[j + e / 4][e & 3] * by;
        if (in_row && (kPlain || col < n)) put_operand<O>(dz + row * ld + col, plane, v);
      }
    }
    if (column_sums == nullptr) return;
    float *const to = column_sums + (uint64_t)(row0 / (kSub * 16)) * ld;
#pragma unroll
    for (uint32_t j = 0; j < kSub; ++j) {
      Acc s;
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) s[e] = group_sum<16>(sum[j][e]);
      const uint32_t col = col0 + outer_of(j, (lane / 16) * 4);
      if ((lane & 15) == 0 && col < n) *reinterpret_cast<Acc *>(to + col) = s;
    }
  }

  template <bool kGated, uint32_t kSub>
  __device__ __forceinline__ void run(const Acc (&acc)[kSub][kSub], uint32_t row0, uint32_t col0,
                                      bool whole, uint32_t) const {
    if (whole && bias == nullptr) go<true>(acc, row0, col0);
    else go<false>(acc, row0, col0);
    if (status != nullptr && blockIdx.x == 0) report_ids<kThreads>(targets, rows, classes, status);
  }
};

// d_bias of a piece: the tiles' column sums, 16 columns and 16 parts of the
// tiles a block, then the parts in order.
__global__ __launch_bounds__(kThreads) void join_columns(const float *__restrict__ sums,
                                                         uint32_t slices, uint64_t ld, uint32_t n,
                                                         float *__restrict__ out) {
  __shared__ float part[16][17];
  const uint32_t in = threadIdx.x & 15, lane = threadIdx.x / 16, col = blockIdx.x * 16 + in;
  const uint32_t each = (slices + 15) / 16;
  float a = 0.0f;
  if (col < n) {
#pragma unroll 4
    for (uint32_t k = lane * each; k < min(slices, (lane + 1) * each); ++k) a += sums[k * ld + col];
  }
  part[lane][in] = a;
  __syncthreads();
  if (lane > 0 || col >= n) return;
  for (uint32_t k = 1; k < 16; ++k) a += part[k][in];
  out[col] = a;
}

template <class O>
__global__ __launch_bounds__(kThreads) void zero_table(O *out, uint64_t ld, uint32_t v, uint32_t d,
                                                       float *bias) {
  for (uint64_t id = (uint64_t)blockIdx.x * kThreads + threadIdx.x; id < (uint64_t)v * d;
       id += (uint64_t)gridDim.x * kThreads) {
    const uint64_t row = id / d;
    if (out != nullptr) out[row * ld + (id - row * d)] = (O)0.0f;
    if (bias != nullptr && id - row * d == 0) bias[row] = 0.0f;
  }
}

// Rows of one launch of the forward product: its slices' sums stay below this, or
// are those of 4096 rows where that is more (above 700k classes; 3.2 GB at 2^23).
constexpr uint64_t kSumsBytes = 512ull << 20;

struct LossRoom {
  Matrix x, table;
  float *sums, *at_target;
  PackList list = {};
  Shape shape;
  uint32_t rows;  // of a launch
  size_t bytes;
};

bool few(const LossCall &c) { return few_rows(c.dtype, c.n, (uint64_t)c.d * c.v, false); }

LossRoom lay_out(const LossCall &c, bool x_stays, bool table_stays, void *ws) {
  LossRoom r;
  Room room{static_cast<char *>(ws)};
  if (few(c)) {
    r.rows = c.n;
    r.sums = static_cast<float *>(room.take((size_t)c.n * 12 * few_slices(c.v)));
    r.at_target = static_cast<float *>(room.take((size_t)c.n * 4));
    r.bytes = room.used;
    return r;
  }
  r.x = operand(c.x, c.dtype, c.x_ld, c.n, c.d, x_stays, room, r.list);
  r.table = operand(c.table, c.dtype, c.table_ld, c.v, c.d, table_stays, room, r.list);
  const uint64_t a_row = 3ull * 4 * 2 * div_up(c.v, 128);  // (of the most slices)
  uint64_t rows = kSumsBytes / a_row / 256 * 256;
  if (rows < 4096) rows = 4096;
  r.rows = rows < c.n ? (uint32_t)rows : c.n;
  r.shape = plan_shape(r.rows, c.v, tiles_of(c.dtype, 1, up8(c.d)), true);
  r.sums = static_cast<float *>(
      room.take((size_t)r.rows * 12 * 2 * div_up(c.v, r.shape.tile)));
  r.at_target = static_cast<float *>(room.take((size_t)r.rows * 4));
  r.bytes = room.used;
  return r;
}

// Classes of a piece: d_z of one stays below this, or has 256 classes where that
// is more (from 2^19 16-bit rows on, a third of that in f32).
constexpr uint64_t kPieceBytes = 256ull << 20;

struct LossGradRoom {
  Matrix x, table;
  uint16_t *dz;
  uint64_t dz_ld;
  float *parts, *columns;
  Scale *scale;  // (f16)
  Looked *looked;
  PackList list = {};
  Shape z, dx, dt;
  uint32_t piece;  // classes
  size_t bytes;
};

LossGradRoom lay_out_grad(const LossGradCall &c, bool x_stays, bool table_stays, bool d_x, bool d_bias,
                          void *ws) {
  LossGradRoom r;
  Room room{static_cast<char *>(ws)};
  r.x = operand(c.x, c.dtype, c.x_ld, c.n, c.d, x_stays, room, r.list);
  r.table = operand(c.table, c.dtype, c.table_ld, c.v, c.d, table_stays, room, r.list);
  uint64_t piece = kPieceBytes / ((uint64_t)c.n * 2 * planes_of(c.dtype)) / 256 * 256;
  if (piece < 256) piece = 256;
  const uint32_t count = div_up(c.v, piece);
  // pieces of equal size
  piece = (div_up(c.v, count) + 255) / 256 * 256;
  r.piece = piece < c.v ? (uint32_t)piece : c.v;
  r.dz_ld = apart64(r.piece);
  r.dz = static_cast<uint16_t *>(room.take(matrix_bytes(c.dtype, c.n, r.piece)));
  const uint32_t tiles = tiles_of(c.dtype, 1, up8(c.d));
  r.z = plan_shape(c.n, r.piece, tiles, true);
  r.dx = plan_shape(c.n, c.d, tiles_of(c.dtype, 1, up8(r.piece)));
  r.dt = plan_shape(r.piece, c.d, tiles_of(c.dtype, 1, c.n));
  const size_t a = d_x ? (size_t)r.dx.parts * c.n * up8(c.d) * 4 : 0;
  const size_t b = parts_bytes(r.dt, r.piece, up8(c.d));
  r.parts = static_cast<float *>(room.take(a));
  r.columns = static_cast<float *>(room.take(b));
  const size_t s = d_bias ? (size_t)div_up(c.n, r.z.tile) * 2 * r.dz_ld * 4 : 0;
  // (the table's parts and the bias' sums are not there at the same time)
  if (s > b) {
    room.used -= align_up(b, 256);
    r.columns = static_cast<float *>(room.take(s));
  }
  r.scale = static_cast<Scale *>(room.take(sizeof(Scale)));
  r.looked = static_cast<Looked *>(
      room.take(is_f16(c.dtype) ? kScaleBlocks * sizeof(Looked) : 0));
  r.bytes = room.used;
  return r;
}

}  // namespace

size_t loss_workspace(const LossCall &c, bool aligned) {
  if (c.n == 0) return 0;
  const bool s = aligned && c.dtype != 0u && c.d % 8 == 0;
  return lay_out(c, s, s, nullptr).bytes;
}

size_t loss_need(const LossCall &c) {
  if (c.n == 0) return 0;
  return lay_out(c, in_place(c.x, c.dtype, c.x_ld, c.d), in_place(c.table, c.dtype, c.table_ld, c.d),
                 nullptr)
      .bytes;
}

hipError_t launch_loss(const LossCall &c, float *logp, float *entropy, float *stats, void *ws,
                       uint32_t *status, hipStream_t stream) {
  const LossRoom r =
      c.n == 0 ? LossRoom{}
               : lay_out(c, in_place(c.x, c.dtype, c.x_ld, c.d),
                         in_place(c.table, c.dtype, c.table_ld, c.d), ws);
  hipError_t e = launch_pack(r.list, c.dtype, stream);
  const uint32_t d8 = up8(c.d);
  for (uint64_t i = 0; e == hipSuccess && (i < c.n || i == 0); i += r.rows) {
    const uint32_t rows = (uint32_t)(c.n - i < r.rows ? c.n - i : r.rows);
    const uint32_t slices = few(c) ? few_slices(c.v) : 2 * div_up(c.v, r.shape.tile);
    const int32_t *const targets = c.targets == nullptr ? nullptr : c.targets + i;
    if (few(c) && rows > 0) {
      const FewSums sums = {c.x, c.table, c.bias, targets, r.sums, r.at_target, c.x_ld, c.table_ld,
                            rows, c.d, c.v};
      if ((e = launch_few_sums(sums, c.dtype, stream)) != hipSuccess) break;
    } else if (rows > 0) {
      const uint64_t a_base[1] = {i * r.x.ld};
      const Args g = make_args(c.dtype, r.x, r.table, rows, c.v, d8, d8, 1, a_base, nullptr, r.shape, c.v);
      const RowSums sums = {c.bias, targets, r.sums, r.at_target, rows, c.v};
      e = with_types(c.dtype, [&](auto, auto t) {
        return launch_tiles<decltype(t), kAlongK, kAlongK, false>(g, r.shape, sums, stream);
      });
      if (e != hipSuccess) break;
    }
    const auto join = rows < 4096 ? join_rows<256> : join_rows<16>;
    join<<<div_up(rows, rows < 4096 ? 1 : 16) + 1, kThreads, 0, stream>>>(
        r.sums, r.at_target, slices, rows, c.v, targets, logp == nullptr ? nullptr : logp + i,
        entropy == nullptr ? nullptr : entropy + i, stats == nullptr ? nullptr : stats + 2 * i,
        c.targets, c.targets == nullptr ? 0 : c.n, i == 0 ? status : nullptr);
    e = hipGetLastError();
    if (c.n == 0) break;
  }
  return e;
}

size_t loss_grad_workspace(const LossGradCall &c, bool aligned) {
  if (c.n == 0) return 0;
  const bool s = aligned && c.dtype != 0u && c.d % 8 == 0;
  return lay_out_grad(c, s, s, true, true, nullptr).bytes;
}

size_t loss_grad_need(const LossGradCall &c, bool d_x, bool d_bias) {
  if (c.n == 0) return 0;
  return lay_out_grad(c, in_place(c.x, c.dtype, c.x_ld, c.d),
                      in_place(c.table, c.dtype, c.table_ld, c.d), d_x, d_bias, nullptr)
      .bytes;
}

hipError_t launch_loss_grad(const LossGradCall &c, void *d_x, uint64_t d_x_ld, void *d_table,
                            uint64_t d_table_ld, float *d_bias, void *ws, uint32_t *status,
                            hipStream_t stream) {
  if (c.n == 0)
    return with_type(c.dtype, [&](auto o) {
      typedef decltype(o) O;
      report_targets<<<1, kPrepare, 0, stream>>>(nullptr, 0, c.v, status);
      if (d_table != nullptr || d_bias != nullptr)
        zero_table<O><<<1024, kThreads, 0, stream>>>(static_cast<O *>(d_table), d_table_ld, c.v, c.d,
                                                     d_bias);
      return hipGetLastError();
    });
  const LossGradRoom r = lay_out_grad(c, in_place(c.x, c.dtype, c.x_ld, c.d),
                                      in_place(c.table, c.dtype, c.table_ld, c.d), d_x != nullptr,
                                      d_bias != nullptr, ws);
  hipError_t e = launch_pack(r.list, c.dtype, stream);
  if (e != hipSuccess) return e;
  const bool scaled = is_f16(c.dtype);
  Scale *const scale = scaled ? r.scale : nullptr;
  const bool apart = scaled || c.targets == nullptr || c.n > 32768;
  if (scaled) {
    e = launch_scale(c, r.looked, scale, status, stream);
  } else if (apart) {
    report_targets<<<1, kPrepare, 0, stream>>>(c.targets, c.n, c.v, status);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  const uint64_t plane = (uint64_t)c.n * r.dz_ld;
  const Matrix dz = {r.dz, r.dz_ld, plane};
  const uint32_t d8 = up8(c.d);
  return with_types(c.dtype, [&](auto o, auto t) {
    typedef decltype(o) O;
    typedef decltype(t) T;
    hipError_t rc = hipSuccess;
    for (uint32_t first = 0; rc == hipSuccess && first < c.v; first += r.piece) {
      const uint32_t n = c.v - first < r.piece ? c.v - first : r.piece;
      const uint32_t n8 = up8(n);
      const uint64_t t_base[1] = {first * r.table.ld};
      {
        const Args g = make_args(c.dtype, r.x, r.table, c.n, n, d8, d8, 1, nullptr, t_base, r.z, n);
        const PutDz<O> put = {c.bias == nullptr ? nullptr : c.bias + first,
                              c.targets,
                              c.stats,
                              c.entropy,
                              c.d_logp,
                              c.d_entropy,
                              scale,
                              r.dz,
                              r.dz_ld,
                              plane,
                              d_bias == nullptr ? nullptr : r.columns,
                              c.n,
                              n,
                              first,
                              c.v,
                              apart || first > 0 ? nullptr : status};
        rc = launch_tiles<T, kAlongK, kAlongK, false>(g, r.z, put, stream);
        if (rc != hipSuccess) break;
        if (d_bias != nullptr) {
          const uint32_t slices = 2 * div_up(c.n, r.z.tile);
          join_columns<<<div_up(n, 16), kThreads, 0, stream>>>(r.columns, slices, r.dz_ld, n,
                                                                     d_bias + first);
          if ((rc = hipGetLastError()) != hipSuccess) break;
        }
      }
      if (d_x != nullptr) {
        Shape s = r.dx;
        const uint32_t tiles = tiles_of(c.dtype, 1, n8);
        s.per_part = (tiles + s.parts - 1) / s.parts;
        s.per_part += s.per_part & 1;
        s.parts = (tiles + s.per_part - 1) / s.per_part;
        const Args g = make_args(c.dtype, dz, r.table, c.n, c.d, n8, n, 1, nullptr, t_base, s, c.d);
        const ToScaledRows<O> to = {static_cast<O *>(d_x), d_x_ld, c.d, scale};
        if (r.piece >= c.v && r.dx.parts == 1) {
          rc = launch_tiles<T, kAlongK, kAcrossK, false>(g, s, Each<ToScaledRows<O>>{to, c.n, c.d},
                                                         stream);
        } else {
          rc = launch_tiles<T, kAlongK, kAcrossK, false>(
              g, s, Parts{r.parts, c.n, c.d, d8, first > 0}, stream);
          if (rc == hipSuccess && first + n == c.v)
            rc = launch_join<false>(r.parts, r.dx.parts, c.n, c.d, d8, to, stream);
        }
        if (rc != hipSuccess) break;
      }
      if (d_table != nullptr) {
        Shape s = r.dt;
        const Args g = make_args(c.dtype, dz, r.x, n, c.d, c.n, c.n, 1, nullptr, nullptr, s, c.d);
        rc = launch_product<T, kAcrossK, kAcrossK, false>(
            g, s,
            ToScaledRows<O>{static_cast<O *>(d_table) + first * d_table_ld, d_table_ld, c.d, scale},
            r.columns, stream);
      }
    }
    return rc;
  });
}

}  // namespace seacells
