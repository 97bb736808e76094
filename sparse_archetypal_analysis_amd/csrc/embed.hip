// Embedding lookup with scaling, and its table gradient by sorted tokens.
//
//   y[i] = scale * table[token[i]]
//   d_table[t] = add_to[t] + scale * sum of d_y[i] over token[i] = t
//
// Both are bound by memory: the lookup reads and writes each element once, the
// gradient reads d_y once and writes the whole table once.
//
// The gradient sorts the token positions by id first, so each table row is
// summed by one owner in a fixed order: no floating-point atomics, no zero
// fill of the table in a pass of its own, one rounding.
#include "token.hpp"

namespace seacells {

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kMaxBlocks = 1u << 20;

// --- lookup -----------------------------------------------------------------

template <class T>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(const T *__restrict__ table, uint32_t v, uint32_t d, uint64_t table_ld,
                 const int32_t *__restrict__ tokens, uint32_t n, float scale, T *__restrict__ out,
                 uint64_t out_ld, uint32_t *__restrict__ status) {
  const uint32_t lane = lane_id();
  const uint32_t waves = gridDim.x * (kThreads / kWave);
  for (uint64_t i = blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave; i < n; i += waves) {
    const int32_t t = tokens[i];
    const bool bad = t >= 0 && (uint32_t)t >= v;
    if (bad && lane == 0) atomicOr(status, kFlagBadIndex);
    const bool have = t >= 0 && !bad;
    const T *row = table + (have ? (uint64_t)t * table_ld : 0);
    T *to = out + i * out_ld;
    for (uint32_t c = lane * kVec<T>; c < d; c += kWave * kVec<T>) {
      Vec<T> y = {};
      if (have) {
        const Vec<T> x = load_vec_tail(row, c, d, (T)0.0f);
#pragma unroll
        for (uint32_t j = 0; j < kVec<T>; ++j) y[j] = (T)((float)x[j] * scale);
      }
      store_vec_tail(to, c, d, y);
    }
  }
}

// --- token sort -------------------------------------------------------------

constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / kWave;
constexpr uint32_t kSortMaxIds = 1024;  // 64 KB of counters
constexpr uint32_t kSortUnroll = 8;

// Positions 0..n-1 ordered by token id, equal ids by position: perm, and
// start[t] = the first place of id t (start[v] = tokens kept). Block b owns
// the ids [b * ids, b * ids + ids) and reads every token twice (they stay in
// L2): once to count its own ids and the tokens below them, which is where
// its part of perm begins, so no block waits for another and the whole sort
// is one launch. Each wave owns one stretch of the positions and its own
// counters; cursors follow the order (id, wave), and a wave places equal ids
// of one step by lane, so the order does not depend on timing.
__global__ void __launch_bounds__(kSortThreads)
    token_sort_kernel(const int32_t *__restrict__ tokens, uint32_t n, uint32_t v, uint32_t ids,
                      uint32_t *__restrict__ perm, uint32_t *__restrict__ start,
                      uint32_t *__restrict__ status) {
  extern __shared__ uint32_t counts[];  // [kSortWaves][ids]
  __shared__ uint32_t wave_part[kSortWaves];
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
  const uint32_t lo = blockIdx.x * ids;
  const uint32_t mine = min(ids, v - lo);
  uint32_t *cnt = counts + wave * ids;
  for (uint32_t i = threadIdx.x; i < kSortWaves * ids; i += kSortThreads) counts[i] = 0u;
  __syncthreads();

  const uint32_t steps = (uint32_t)(((uint64_t)n + kSortThreads - 1) / kSortThreads);
  const uint64_t first = (uint64_t)wave * steps * kWave;  // this wave's positions
  uint32_t below = 0;
  bool bad = false;
  for (uint32_t s = 0; s < steps; s += kSortUnroll) {
    int32_t t[kSortUnroll];
#pragma unroll
    for (uint32_t u = 0; u < kSortUnroll; ++u) {
      const uint64_t i = first + (uint64_t)(s + u) * kWave + lane;
      t[u] = s + u < steps && i < n ? tokens[i] : -1;
    }
#pragma unroll
    for (uint32_t u = 0; u < kSortUnroll; ++u) {
      if (t[u] < 0) continue;
      const uint32_t id = (uint32_t)t[u];
      bad |= id >= v;
      below += id < lo ? 1u : 0u;
      if (id - lo < mine) atomicAdd(&cnt[id - lo], 1u);
    }
  }
  // every block has seen every token; the first one reports
  const bool any_bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = any_bad ? kFlagBadIndex : 0u;

  // tokens below the block's ids
  for (uint32_t off = 32; off >= 1; off >>= 1) below += __shfl_xor(below, off, kWave);
  if (lane == 0) wave_part[wave] = below;
  __syncthreads();
  uint32_t base = 0;
  for (uint32_t w = 0; w < kSortWaves; ++w) base += wave_part[w];
  __syncthreads();

  // one thread per id: counts into cursors (ids <= kSortThreads)
  uint32_t total = 0;
  if (threadIdx.x < mine)
    for (uint32_t w = 0; w < kSortWaves; ++w) total += counts[w * ids + threadIdx.x];
  uint32_t incl = total;
  for (uint32_t off = 1; off < kWave; off <<= 1) {
    const uint32_t x = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += x;
  }
  if (lane == kWave - 1) wave_part[wave] = incl;
  __syncthreads();
  for (uint32_t w = 0; w < wave; ++w) base += wave_part[w];
  if (threadIdx.x < mine) {
    uint32_t at = base + incl - total;
    start[lo + threadIdx.x] = at;
    if (lo + threadIdx.x + 1 == v) start[v] = at + total;
    for (uint32_t w = 0; w < kSortWaves; ++w) {
      const uint32_t c = counts[w * ids + threadIdx.x];
      counts[w * ids + threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();

  for (uint32_t s = 0; s < steps; s += kSortUnroll) {
    int32_t t[kSortUnroll];
#pragma unroll
    for (uint32_t u = 0; u < kSortUnroll; ++u) {
      const uint64_t i = first + (uint64_t)(s + u) * kWave + lane;
      t[u] = s + u < steps && i < n ? tokens[i] : -1;
    }
#pragma unroll
    for (uint32_t u = 0; u < kSortUnroll; ++u) {
      const uint32_t id = (uint32_t)t[u];
      const bool hit = t[u] >= 0 && id - lo < mine;
      uint64_t left = __ballot(hit);
      while (left != 0) {
        const uint32_t cur = readlane_u32(id, (uint32_t)__builtin_ctzll(left));
        const bool same_id = hit && id == cur;
        const uint64_t same = __ballot(same_id);
        const uint32_t at = cnt[cur - lo];
        if (same_id) {
          const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
          perm[at + rank] = (uint32_t)(first + (uint64_t)(s + u) * kWave + lane);
        }
        wave_lds_sync();
        if (lane == 0) cnt[cur - lo] = at + (uint32_t)__popcll(same);
        wave_lds_sync();
        left &= ~same;
      }
    }
  }
}

// --- table gradient ---------------------------------------------------------

// Ids with more tokens than this ("heavy") are summed in parts, one part per
// window of kHeavy sorted positions, so that a token that fills a third of
// the batch does not leave its row to one wave.
constexpr uint32_t kHeavy = 32;
constexpr uint32_t kRowUnroll = 8;  // rows of d_y in flight per lane

// How the lanes cover the columns: `lanes` (a power of two, at most a wave)
// side by side with `chunks` vectors each, then further slabs (grid y).
struct Cover {
  uint32_t lanes, chunks, slabs;
};

template <uint32_t kV>
Cover cover(uint32_t d) {
  Cover c{};
  const uint32_t vecs = div_up(d, kV);
  c.lanes = 1;
  while (c.lanes < kWave && c.lanes < vecs) c.lanes *= 2;
  const uint32_t per = div_up(vecs, c.lanes);
  c.chunks = per <= 1 ? 1 : per <= 2 ? 2 : 4;
  c.slabs = div_up(vecs, c.lanes * c.chunks);
  return c;
}

// acc += the rows perm[p0 .. p1) of d_y in order, columns c0 + chunk * step.
template <class T, uint32_t kC>
__device__ __forceinline__ void sum_rows(const uint32_t *__restrict__ perm, uint32_t p0, uint32_t p1,
                                         const T *__restrict__ d_out, uint64_t ld, uint32_t c0,
                                         uint32_t step, uint32_t d, float (&acc)[kC][kVec<T>]) {
  constexpr uint32_t kU = kRowUnroll / kC > 1 ? kRowUnroll / kC : 2;
  for (uint32_t p = p0; p < p1; p += kU) {
    Vec<T> x[kU][kC];
#pragma unroll
    for (uint32_t u = 0; u < kU; ++u) {
      const T *row = d_out + (uint64_t)perm[p + u < p1 ? p + u : p] * ld;
#pragma unroll
      for (uint32_t k = 0; k < kC; ++k) {
        const uint32_t c = c0 + k * step;
        x[u][k] = p + u < p1 && c < d ? load_vec_tail(row, c, d, (T)0.0f) : Vec<T>{};
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < kU; ++u)
#pragma unroll
      for (uint32_t k = 0; k < kC; ++k)
#pragma unroll
        for (uint32_t j = 0; j < kVec<T>; ++j) acc[k][j] += (float)x[u][k][j];
  }
}

// d_table[t, c ..] = so_far + scale * acc
template <class O, uint32_t kV>
__device__ __forceinline__ void write_row(const O *so_far, O *to, uint32_t c, uint32_t d,
                                          float scale, const float (&acc)[kV]) {
  if (c + kV <= d) {
    Pack<O, kV> y;
    if (so_far != nullptr) {
      const Pack<O, kV> a = *reinterpret_cast<const Pack<O, kV> *>(so_far + c);
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) y[j] = (O)((float)a[j] + scale * acc[j]);
    } else {
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) y[j] = (O)(scale * acc[j]);
    }
    *reinterpret_cast<Pack<O, kV> *>(to + c) = y;
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < kV; ++j)
    if (c + j < d) to[c + j] = (O)((so_far != nullptr ? (float)so_far[c + j] : 0.0f) + scale * acc[j]);
}

// One group of lanes per unit: first the windows of sorted positions (parts
// of heavy ids), then the table rows. A window meets at most two heavy ids,
// one at each end; part[2 w] holds the sum of the one that covers its first
// position, part[2 w + 1] of one that starts inside it.
template <class T, class O, uint32_t kC>
__global__ void __launch_bounds__(kThreads)
    embed_grad_rows_kernel(const uint32_t *__restrict__ perm, const uint32_t *__restrict__ start,
                           const int32_t *__restrict__ tokens, uint32_t windows, uint32_t lanes,
                           const T *__restrict__ d_out, uint64_t d_out_ld, uint32_t v, uint32_t d,
                           float scale, const O *add_to, O *d_table, uint64_t d_table_ld,
                           float *__restrict__ part) {
  constexpr uint32_t kV = kVec<T>;
  const uint32_t step = lanes * kV;
  const uint32_t c0 = blockIdx.y * step * kC + (threadIdx.x & (lanes - 1)) * kV;
  const uint32_t per_block = kThreads / lanes;
  const uint64_t units = (uint64_t)windows + v;
  for (uint64_t unit = (uint64_t)blockIdx.x * per_block + threadIdx.x / lanes; unit < units;
       unit += (uint64_t)gridDim.x * per_block) {
    if (unit < windows) {
      const uint32_t a = (uint32_t)unit * kHeavy;
      const uint32_t kept = start[v];
      if (a >= kept) continue;
      const uint32_t b = a + kHeavy < kept ? a + kHeavy : kept;
      const uint32_t first = (uint32_t)tokens[perm[a]], last = (uint32_t)tokens[perm[b - 1]];
      for (uint32_t k = 0; k < 2; ++k) {
        const uint32_t id = k == 0 ? first : last;
        if (k == 1 && last == first) break;
        const uint32_t s0 = start[id], s1 = start[id + 1];
        if (s1 - s0 <= kHeavy) continue;
        float acc[kC][kV] = {};
        sum_rows<T, kC>(perm, s0 > a ? s0 : a, s1 < b ? s1 : b, d_out, d_out_ld, c0, step, d, acc);
        float *to = part + (2 * unit + (s0 > a ? 1 : 0)) * d;
#pragma unroll
        for (uint32_t q = 0; q < kC; ++q) {
          const uint32_t c = c0 + q * step;
          if (c < d) write_row<float, kV>(nullptr, to, c, d, 1.0f, acc[q]);
        }
      }
      continue;
    }
    const uint64_t t = unit - windows;
    const uint32_t p0 = start[t], p1 = start[t + 1];
    if (p1 - p0 > kHeavy || (p0 == p1 && add_to == d_table)) continue;
    float acc[kC][kV] = {};
    sum_rows<T, kC>(perm, p0, p1, d_out, d_out_ld, c0, step, d, acc);
#pragma unroll
    for (uint32_t q = 0; q < kC; ++q) {
      const uint32_t c = c0 + q * step;
      if (c < d)
        write_row<O, kV>(add_to != nullptr ? add_to + t * d_table_ld : nullptr,
                         d_table + t * d_table_ld, c, d, scale, acc[q]);
    }
  }
}

// Joins the parts of the heavy id that starts in the block's window, if one
// does (it then covers the window's last position, and no other heavy id
// starts there): the waves take equal runs of its windows, then their sums
// are added in order.
constexpr uint32_t kJoinThreads = 1024;
constexpr uint32_t kJoinWaves = kJoinThreads / kWave;

template <class O>
__global__ void __launch_bounds__(kJoinThreads)
    embed_grad_join_kernel(const uint32_t *__restrict__ perm, const uint32_t *__restrict__ start,
                           const int32_t *__restrict__ tokens, uint32_t windows, uint32_t v,
                           uint32_t d, float scale, const O *add_to, O *d_table,
                           uint64_t d_table_ld, const float *__restrict__ part) {
  constexpr uint32_t kV = 4;
  __shared__ float sums[kJoinWaves][kWave * kV];
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
  const uint32_t c = (blockIdx.y * kWave + lane) * kV;
  const uint32_t kept = start[v];
  for (uint32_t w = blockIdx.x; w < windows; w += gridDim.x) {
    const uint32_t a = w * kHeavy;
    if (a + kHeavy >= kept) return;  // a heavy id that starts here ends past the window
    const uint32_t id = (uint32_t)tokens[perm[a + kHeavy - 1]];
    const uint32_t s0 = start[id], s1 = start[id + 1];
    if (s0 < a || s1 - s0 <= kHeavy) continue;
    const uint32_t count = (s1 - 1) / kHeavy - w + 1;  // windows it meets
    const uint32_t run = (count + kJoinWaves - 1) / kJoinWaves;
    const uint32_t k0 = wave * run, k1 = k0 + run < count ? k0 + run : count;
    float acc[kV] = {};
    if (c < d) {
      for (uint32_t k = k0; k < k1; k += kRowUnroll) {
        Vec<float> x[kRowUnroll];
#pragma unroll
        for (uint32_t u = 0; u < kRowUnroll; ++u) {
          const uint64_t slot = 2 * ((uint64_t)w + k + u) + (k + u == 0 && s0 > a ? 1 : 0);
          x[u] = k + u < k1 ? load_vec_tail(part + slot * d, c, d, 0.0f) : Vec<float>{};
        }
#pragma unroll
        for (uint32_t u = 0; u < kRowUnroll; ++u)
#pragma unroll
          for (uint32_t j = 0; j < kV; ++j) acc[j] += x[u][j];
      }
    }
    __syncthreads();  // the sums of an earlier id have been read
#pragma unroll
    for (uint32_t j = 0; j < kV; ++j) sums[wave][lane * kV + j] = acc[j];
    __syncthreads();
    if (wave != 0 || c >= d) continue;
    for (uint32_t q = 1; q < kJoinWaves; ++q)
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) acc[j] += sums[q][lane * kV + j];
    write_row<O, kV>(add_to != nullptr ? add_to + (uint64_t)id * d_table_ld : nullptr,
                     d_table + (uint64_t)id * d_table_ld, c, d, scale, acc);
  }
}

uint32_t wave_blocks(uint64_t waves) {
  const uint64_t b = (waves + kThreads / kWave - 1) / (kThreads / kWave);
  return (uint32_t)(b < kMaxBlocks ? b : kMaxBlocks);
}

}  // namespace

hipError_t launch_embed(const void *table, uint32_t dtype, uint32_t v, uint32_t d, uint64_t table_ld,
                        const int32_t *tokens, uint32_t n, float scale, void *out, uint64_t out_ld,
                        uint32_t *status, hipStream_t stream) {
  hipError_t e = launch_status_clear(status, stream);
  if (e != hipSuccess || n == 0) return e;
  return with_type(dtype, [&](auto x) {
    using T = decltype(x);
    hipLaunchKernelGGL((embed_kernel<T>), dim3(wave_blocks(n)), dim3(kThreads), 0, stream,
                       static_cast<const T *>(table), v, d, table_ld, tokens, n, scale,
                       static_cast<T *>(out), out_ld, status);
    return hipGetLastError();
  });
}

EmbedGradPlan plan_embed_grad(uint32_t n, uint32_t v, uint32_t d) {
  EmbedGradPlan p{};
  // blocks for every compute unit where the ids allow it
  uint32_t ids = div_up(v, 256);
  ids = ids < kSortMaxIds ? ids : kSortMaxIds;
  p.ids = ids > 0 ? ids : 1;
  p.blocks = div_up(v, p.ids);
  p.windows = n > kHeavy ? div_up(n, kHeavy) : 0;  // heavy ids are possible
  p.off_perm = 0;
  p.off_start = align_up((size_t)n * sizeof(uint32_t), 256);
  p.off_part = p.off_start + align_up(((size_t)v + 1) * sizeof(uint32_t), 256);
  p.ws_bytes = p.off_part + (size_t)p.windows * 2 * d * sizeof(float);
  return p;
}

hipError_t launch_embed_grad(const EmbedGradPlan &plan, const int32_t *tokens, uint32_t n,
                             const void *d_out, uint32_t d_out_type, uint64_t d_out_ld, uint32_t v,
                             uint32_t d, float scale, const void *add_to, void *d_table,
                             uint32_t d_table_type, uint64_t d_table_ld, void *ws, uint32_t *status,
                             hipStream_t stream) {
  char *base = static_cast<char *>(ws);
  uint32_t *perm = reinterpret_cast<uint32_t *>(base + plan.off_perm);
  uint32_t *start = reinterpret_cast<uint32_t *>(base + plan.off_start);
  hipLaunchKernelGGL(token_sort_kernel, dim3(plan.blocks), dim3(kSortThreads),
                     kSortWaves * plan.ids * sizeof(uint32_t), stream, tokens, n, v, plan.ids, perm,
                     start, status);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float *part = reinterpret_cast<float *>(base + plan.off_part);
  return with_type(d_out_type, [&](auto x) {
    using T = decltype(x);
    const Cover cv = cover<kVec<T>>(d);
    const uint64_t groups = kThreads / cv.lanes;
    const uint64_t want = ((uint64_t)plan.windows + v + groups - 1) / groups;
    const dim3 grid((uint32_t)(want < kMaxBlocks ? want : kMaxBlocks), cv.slabs);
    auto go = [&](auto y) {
      using O = decltype(y);
      const O *add = static_cast<const O *>(add_to);
      O *to = static_cast<O *>(d_table);
      auto rows = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, perm, start, tokens,
                           plan.windows, cv.lanes, static_cast<const T *>(d_out), d_out_ld, v, d,
                           scale, add, to, d_table_ld, part);
      };
      if (cv.chunks == 1) rows(embed_grad_rows_kernel<T, O, 1>);
      else if (cv.chunks == 2) rows(embed_grad_rows_kernel<T, O, 2>);
      else rows(embed_grad_rows_kernel<T, O, 4>);
      hipError_t err = hipGetLastError();
      if (err != hipSuccess || plan.windows == 0) return err;
      hipLaunchKernelGGL((embed_grad_join_kernel<O>), dim3(plan.windows < kMaxBlocks ? plan.windows : kMaxBlocks,
                              div_up(d, kWave * 4)),
                         dim3(kJoinThreads), 0, stream, perm, start, tokens, plan.windows, v, d, scale, add, to,
                         d_table_ld, part);
      return hipGetLastError();
    };
    return d_table_type == (uint32_t)Dtype::f32 ? go(float{}) : go(x);
  });
}

}  // namespace seacells
