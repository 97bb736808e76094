// Embedding lookup with scaling, and its table gradient by sorted tokens.
//
//   y[i] = scale * table[token[i]]
//   d_table[t] = add_to[t] + scale * sum of d_y[i] over token[i] = t
//
// Both are bound by memory: the lookup reads and writes each element once, the
// gradient reads d_y once and writes the whole table once.
//
// The gradient sorts the token positions by id first and sums windows of the
// sorted positions, so the order of every sum is fixed: no floating-point
// atomics, no zero fill of the table in a pass of its own, one rounding.
#include "token.hpp"

namespace seacells {

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kMaxBlocks = 1u << 20;

// How the lanes cover the columns: `lanes` (a power of two, at most a wave)
// side by side with a vector each, then further slabs.
struct Cover {
  uint32_t lanes, slabs;
};

template <uint32_t kV>
Cover cover(uint32_t d) {
  Cover c{};
  const uint32_t vecs = div_up(d, kV);
  c.lanes = 1;
  while (c.lanes < kWave && c.lanes < vecs) c.lanes *= 2;
  c.slabs = div_up(vecs, c.lanes);
  return c;
}

// --- lookup -----------------------------------------------------------------

constexpr uint32_t kRows = 4;  // rows in flight per lane group

// A vector of kRows rows per lane. A row's broken last vector is pulled back
// to end with the row (its first columns are written twice, the same), and
// where there is nothing to look up row 0 is loaded: no load has a branch, so
// they are all in flight together. kWhole: a group is a wave, whose tokens the
// scalar unit reads.
template <class T, bool kWhole>
__global__ void __launch_bounds__(kThreads)
    embed_kernel(const T *__restrict__ table, uint32_t v, uint32_t d, uint64_t table_ld,
                 const int32_t *__restrict__ tokens, uint32_t n, float scale, T *__restrict__ out,
                 uint64_t out_ld, uint32_t lanes_, uint32_t slabs, uint32_t *__restrict__ status,
                 bool check) {
  constexpr uint32_t kV = kVec<T>;
  const uint32_t lanes = kWhole ? kWave : lanes_;
  const uint32_t groups = kThreads / lanes;
  const uint32_t group =
      kWhole ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave))
             : threadIdx.x / lanes;
  const uint32_t lane = threadIdx.x & (lanes - 1);
  const uint32_t slab = blockIdx.x % slabs;
  const uint32_t col = (slab * lanes + lane) * kV;
  const uint32_t at = d < kV ? 0u : col < d - kV ? col : d - kV;
  const uint64_t step = (uint64_t)(gridDim.x / slabs) * groups * kRows;
  for (uint64_t i0 = (uint64_t)(blockIdx.x / slabs) * groups * kRows + group; i0 < n; i0 += step) {
    int32_t t[kRows];
    bool have[kRows];
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u)
      t[u] = i0 + u * groups < n ? tokens[i0 + u * groups] : -1;
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      have[u] = t[u] >= 0 && t[u] < (int32_t)v;
      if (check && t[u] >= (int32_t)v && lane == 0) atomicOr(status, kFlagBadIndex);
    }
    Vec<T> x[kRows];
    if (d >= kV) {
#pragma unroll
      for (uint32_t u = 0; u < kRows; ++u)
        x[u] = load_vec(table + (have[u] ? (uint64_t)t[u] * table_ld : 0) + at);
    } else {
#pragma unroll
      for (uint32_t u = 0; u < kRows; ++u)
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j)
          x[u][j] = table[(have[u] ? (uint64_t)t[u] * table_ld : 0) + (j < d ? j : 0u)];
    }
#pragma unroll
    for (uint32_t u = 0; u < kRows; ++u) {
      if (i0 + u * groups >= n || col >= d) break;
      T *to = out + (i0 + u * groups) * out_ld + at;
      Vec<T> y = {};
      if (have[u])
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j) y[j] = (T)((float)x[u][j] * scale);
      if (d >= kV) store_stream(to, y);
      else store_vec_tail(to, 0u, d, y);
    }
  }
  // after the rows: the other blocks' work hides it
  if (!check && blockIdx.x == 0) report_ids<kThreads>(tokens, n, v, status);
}

// --- token sort -------------------------------------------------------------
//
// Positions 0..n-1 ordered by token id, equal ids by position: perm, their ids
// (sorted), and start[t] = the first place of id t (start[v] = tokens kept).
// The ids are cut into buckets of 2^shift. Chunks of tokens are first ordered
// by bucket, each on its own; then a block per bucket collects its pieces of
// the chunks, orders them by id and writes its part of perm, which begins at
// the sum of the places where its pieces begin in their chunks: no block waits
// for another, and no atomic's order shows. (A block per bucket that reads all
// tokens costs buckets x n: 79 us for 131072 tokens and 262144 rows against 26
// in two launches; up to kDirect of them it saves the chunks' launch: 3500
// tokens and 20000 ids of 64 columns 20.8 us against 25.8.)

constexpr uint32_t kChunkThreads = 256;
constexpr uint32_t kChunkWaves = kChunkThreads / kWave;
constexpr uint32_t kMaxBuckets = 1024;  // with that of the frequent id (there or not)

constexpr uint32_t kSortThreads = 512;
constexpr uint32_t kSortWaves = kSortThreads / kWave;
constexpr uint32_t kSortIds = 512;    // ids ordered at once, a thread each
constexpr uint32_t kDirect = 4096;
constexpr uint32_t kSortUnroll = 4;   // of a wave's loads
constexpr uint32_t kSortBlocks = 128;

// Exclusive prefix of x over the block's kWaves waves, and the sum in *total.
template <uint32_t kWaves>
__device__ __forceinline__ uint32_t block_prefix(uint32_t x, uint32_t *lds, uint32_t *total) {
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
  uint32_t incl = x;
#pragma unroll
  for (uint32_t off = 1; off < kWave; off <<= 1) {
    const uint32_t y = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += y;
  }
  __syncthreads();
  if (lane == kWave - 1) lds[wave] = incl;
  __syncthreads();
  uint32_t before = 0, sum = 0;
#pragma unroll
  for (uint32_t w = 0; w < kWaves; ++w) {
    const uint32_t y = lds[w];
    before += w < wave ? y : 0u;
    sum += y;
  }
  *total = sum;
  return before + incl - x;
}

// The id that most lanes hold in t (a wave takes 64 tokens at even distances),
// kNoId if none is there kOften times. A bucket with such an id (padding, a frequent
// word) would keep its one block busy long after the others, so the id has a
// bucket of its own, after the ids' own, that several blocks share: 50000 tokens
// of one id of 100000, 100 columns, 111 us without and 34 with it, 131072 of
// 20000 ids, 4 columns, 233 and 30, with frequencies as 1 / rank 47 and 42, all
// even 28.9 and 30.1. Fewer tokens than kOwnFrom do without.
constexpr uint32_t kNoId = 0xffffffffu;
constexpr uint32_t kOften = 4;
constexpr uint32_t kOwnFrom = 16384;

__device__ __forceinline__ uint32_t frequent_id(int32_t t, uint32_t v) {
  const bool has = t >= 0 && t < (int32_t)v;
  uint64_t same = __ballot(has);
  for (uint32_t bit = 1; bit != 0 && bit < v; bit <<= 1) {
    const uint64_t set = __ballot(((uint32_t)t & bit) != 0);
    same &= ((uint32_t)t & bit) != 0 ? set : ~set;
  }
  const uint32_t times = has ? (uint32_t)__popcll(same) : 0u;
  uint64_t more = __ballot(times >= kOften);
  uint32_t id = kNoId;
  while (more != 0) {
    const uint32_t from = (uint32_t)__builtin_ctzll(more);
    id = readlane_u32((uint32_t)t, from);
    more = __ballot(times > readlane_u32(times, from));
  }
  return id;
}

// A chunk of kPer * 256 tokens, ordered by bucket: entry_id, entry_pos, and
// cuts[chunk][k] = the first place of bucket k in the chunk, the last bucket
// that of the frequent id (if `own`, else empty: buckets < kMaxBuckets, so a
// thread writes it), then the tokens kept, then whether an id was v or more.
template <uint32_t kPer>
__global__ void __launch_bounds__(kChunkThreads)
    token_chunk_kernel(const int32_t *__restrict__ tokens, uint32_t n, uint32_t v, uint32_t shift,
                       uint32_t buckets, bool own, uint32_t *__restrict__ entry_id,
                       uint32_t *__restrict__ entry_pos, uint32_t *__restrict__ cuts,
                       uint32_t *__restrict__ frequent) {
  __shared__ uint32_t cnt[kChunkWaves][kMaxBuckets];
  __shared__ uint32_t part[kChunkWaves];
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
  const uint64_t lower = (1ull << lane) - 1ull;
  const uint64_t chunk = (uint64_t)blockIdx.x * kPer * kChunkThreads;
  const uint64_t first = chunk + wave * kPer * kWave + lane;
  int32_t t[kPer];
#pragma unroll
  for (uint32_t u = 0; u < kPer; ++u)
    t[u] = first + u * kWave < n ? tokens[first + u * kWave] : -1;
  const int32_t sample = own ? tokens[(uint64_t)lane * n / kWave] : -1;
  for (uint32_t i = threadIdx.x; i < kMaxBuckets; i += kChunkThreads)
#pragma unroll
    for (uint32_t w = 0; w < kChunkWaves; ++w) cnt[w][i] = 0u;
  const uint32_t often = own ? frequent_id(sample, v) : kNoId;
  if (blockIdx.x == 0 && threadIdx.x == 0) *frequent = often;
  auto bucket_of = [&](int32_t id) {
    return (uint32_t)id == often ? buckets : (uint32_t)id >> shift;
  };
  __syncthreads();

  uint32_t place[kPer];
  bool bad = false;
#pragma unroll
  for (uint32_t u = 0; u < kPer; ++u) {
    bad |= t[u] >= (int32_t)v;
    const bool has = t[u] >= 0 && t[u] < (int32_t)v;
    const uint32_t k = has ? bucket_of(t[u]) : 0u;
    uint64_t same = __ballot(has);  // the lanes with this one's bucket
    for (uint32_t bit = 1; bit <= buckets; bit <<= 1) {
      const uint64_t set = __ballot((k & bit) != 0);
      same &= (k & bit) != 0 ? set : ~set;
    }
    const uint32_t rank = (uint32_t)__popcll(same & lower);
    const uint32_t at = cnt[wave][k];
    place[u] = at + rank;
    wave_lds_sync();
    if (has && rank == 0) cnt[wave][k] = at + (uint32_t)__popcll(same);
    wave_lds_sync();
  }
  const bool any_bad = __syncthreads_or(bad);
  // four neighbouring buckets per thread
  constexpr uint32_t kMine = kMaxBuckets / kChunkThreads;
  uint32_t c[kMine][kChunkWaves], sum = 0, total;
#pragma unroll
  for (uint32_t m = 0; m < kMine; ++m)
#pragma unroll
    for (uint32_t w = 0; w < kChunkWaves; ++w) {
      c[m][w] = cnt[w][threadIdx.x * kMine + m];
      sum += c[m][w];
    }
  uint32_t at = block_prefix<kChunkWaves>(sum, part, &total);
  uint32_t *row = cuts + (uint64_t)blockIdx.x * (buckets + 3);
#pragma unroll
  for (uint32_t m = 0; m < kMine; ++m) {
    const uint32_t k = threadIdx.x * kMine + m;
    if (k <= buckets) row[k] = at;
#pragma unroll
    for (uint32_t w = 0; w < kChunkWaves; ++w) {
      cnt[w][k] = at;
      at += c[m][w];
    }
  }
  if (threadIdx.x == 0) {
    row[buckets + 1] = total;
    row[buckets + 2] = any_bad ? 1u : 0u;
  }
  __syncthreads();
#pragma unroll
  for (uint32_t u = 0; u < kPer; ++u) {
    if (t[u] < 0 || t[u] >= (int32_t)v) continue;
    const uint64_t to = chunk + cnt[wave][bucket_of(t[u])] + place[u];
    entry_id[to] = (uint32_t)t[u];
    entry_pos[to] = (uint32_t)(first + u * kWave);
  }
}

// Orders a bucket's tokens by id. They come from the chunks (cuts) or, few of
// them (kFew), from the tokens themselves. Each wave takes an equal run of
// them, in the order of their positions, counts it by counters of its own and
// then places it: cursors follow the order (id, wave). A bucket of one id is in
// order as it comes, and several blocks (grid y) may share it. The blocks from
// `buckets` on share the frequent id's tokens: these stand among its bucket's,
// after those of the ids before it, which they count first.
template <bool kFew>
__global__ void __launch_bounds__(kSortThreads)
    token_sort_kernel(const int32_t *__restrict__ tokens, uint32_t n, uint32_t v, uint32_t shift,
                      uint32_t buckets, const uint32_t *__restrict__ cuts, uint32_t chunks,
                      uint32_t chunk_len, const uint32_t *__restrict__ entry_id,
                      const uint32_t *__restrict__ entry_pos,
                      const uint32_t *__restrict__ frequent, uint32_t *__restrict__ perm,
                      uint32_t *__restrict__ sorted, uint32_t *__restrict__ start,
                      uint32_t *__restrict__ status) {
  extern __shared__ uint32_t counts[];  // [kSortWaves][ids at once]
  __shared__ uint32_t first[kSortThreads], begin[kSortThreads];  // of the chunks at hand
  __shared__ uint32_t lds[kSortWaves];
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
  const uint64_t lower = (1ull << lane) - 1ull;
  uint32_t bucket = blockIdx.x;
  const bool sharing = !kFew && blockIdx.x >= buckets;
  if (sharing) {
    if (*frequent == kNoId) return;
    bucket = *frequent >> shift;
  }
  const uint32_t lo = bucket << shift;
  const uint32_t mine = min(1u << shift, v - lo);
  const uint32_t at_once = min(1u << shift, kSortIds);

  // the chunks from c0 on: where the bucket begins in each, and how many of
  // its tokens the chunks before hold; returns the tokens in all of them
  auto load_cuts = [&](uint32_t c0) {
    const uint32_t c = c0 + threadIdx.x;
    const uint32_t *cut = cuts + (uint64_t)(c < chunks ? c : 0u) * (buckets + 3) + bucket;
    const uint32_t e0 = cut[0], e1 = c < chunks ? cut[1] : e0;
    uint32_t all;
    const uint32_t before = block_prefix<kSortWaves>(e1 - e0, lds, &all);
    first[threadIdx.x] = before;
    begin[threadIdx.x] = e0;
    __syncthreads();
    return all;
  };

  // a batch of the wave's tokens: id, position, and whether there is one
  uint32_t id[kSortUnroll], pos[kSortUnroll];
  bool has[kSortUnroll];
  constexpr uint32_t kBatch = kWave * kSortUnroll;
  auto read_tokens = [&](uint32_t i, uint32_t i1) {
#pragma unroll
    for (uint32_t u = 0; u < kSortUnroll; ++u) {
      pos[u] = i + u * kWave + lane;
      id[u] = pos[u] < i1 ? (uint32_t)tokens[pos[u]] : ~0u;
      has[u] = id[u] - lo < mine;  // (a negative token is no id below 2^31)
    }
  };
  // the bucket's tokens from e on, of those before e1, in the chunks from c0
  // on, before which there are `done`
  auto read_chunks = [&](uint32_t e, uint32_t e1, uint32_t c0, uint32_t done) {
#pragma unroll
    for (uint32_t u = 0; u < kSortUnroll; ++u) {
      const uint32_t q = e + u * kWave + lane;
      const uint32_t r = (q < e1 ? q : e) - done;
      uint32_t c = 0;  // the last chunk that begins at or before it
#pragma unroll
      for (uint32_t half = kSortThreads / 2; half >= 1; half /= 2)
        c = first[c + half] <= r ? c + half : c;
      const uint64_t from = (uint64_t)(c0 + c) * chunk_len + begin[c] + (r - first[c]);
      has[u] = q < e1;
      id[u] = entry_id[from];
      pos[u] = entry_pos[from];
    }
  };

  uint32_t base = 0, have = 0;  // where the bucket begins in perm, and its tokens
  bool bad = false;
  uint32_t below = 0, of_often = 0;
  if constexpr (kFew) {
    for (uint32_t i = threadIdx.x; i < n; i += kSortThreads) {
      const int32_t t = tokens[i];
      bad |= t >= (int32_t)v;
      below += (uint32_t)t < lo ? 1u : 0u;
    }
  } else {
    for (uint32_t c0 = 0; c0 < chunks; c0 += kSortThreads) {
      have += load_cuts(c0);
      if (c0 + threadIdx.x < chunks) {
        const uint32_t *last = cuts + (uint64_t)(c0 + threadIdx.x) * (buckets + 3) + buckets;
        below += begin[threadIdx.x];
        of_often += last[1] - last[0];
        bad |= last[2] != 0;
      }
    }
    if (chunks > kSortThreads) load_cuts(0);
  }
  block_prefix<kSortWaves>(below, lds, &base);
  const bool any_bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = any_bad ? kFlagBadIndex : 0u;

  // the frequent id's tokens, where they stand in this bucket or before
  const uint32_t often = kFew ? kNoId : *frequent;
  if (often != kNoId && bucket >= often >> shift) {
    uint32_t all;
    block_prefix<kSortWaves>(of_often, lds, &all);
    of_often = all;
    if (bucket > often >> shift) base += all;
  }

  uint32_t w0, w1;  // the wave's run
  auto share = [&](uint32_t part, uint32_t parts) {
    part = part * kSortWaves + wave;
    parts *= kSortWaves;
    w0 = (uint32_t)((uint64_t)have * part / parts);
    w1 = (uint32_t)((uint64_t)have * (part + 1) / parts);
  };
  share(blockIdx.y, gridDim.y);
  // a run of one batch from the chunks stays in registers (28509 tokens 29.6 us
  // against 31.1; of tokens read directly it cost 1.3 at 200)
  bool once = !kFew && chunks <= kSortThreads && w0 < w1 && w1 - w0 <= kBatch;
  if (once) read_chunks(w0, w1, 0, 0);

  // f(has, id, position, place among the bucket's tokens (from chunks)) for
  // the wave's tokens in order, a wave's worth at a time
  auto every = [&](auto f) {
    auto each = [&](uint32_t e) {
#pragma unroll
      for (uint32_t u = 0; u < kSortUnroll; ++u) f(has[u], id[u], pos[u], e + u * kWave + lane);
    };
    if (once) {
      each(w0);
      return;
    }
    if constexpr (kFew) {
      const uint32_t i0 = n * wave / kSortWaves, i1 = n * (wave + 1) / kSortWaves;
      for (uint32_t i = i0; i < i1; i += kBatch) {
        read_tokens(i, i1);
        each(0);
      }
      return;
    }
    uint32_t done = 0;
    for (uint32_t c0 = 0; c0 < chunks; c0 += kSortThreads) {
      uint32_t end = have;
      if (chunks > kSortThreads) {
        __syncthreads();
        end = done + load_cuts(c0);
      }
      const uint32_t e0 = max(w0, done), e1 = min(w1, end);
      for (uint32_t e = e0; e < e1; e += kBatch) {
        read_chunks(e, e1, c0, done);
        each(e);
      }
      done = end;
    }
  };

  if (shift == 0 && !kFew) {
    if (threadIdx.x == 0 && blockIdx.y == 0) {
      start[lo] = base;
      if (lo + 1 == v) start[v] = base + have;
    }
    every([&](bool has, uint32_t, uint32_t pos, uint32_t at) {
      if (has) {
        perm[base + at] = pos;
        sorted[base + at] = lo;
      }
    });
    return;
  }

  if (!kFew && sharing) {
    uint32_t x = 0, before;
    every([&](bool has, uint32_t id, uint32_t, uint32_t) { x += has && id < often ? 1u : 0u; });
    block_prefix<kSortWaves>(x, lds, &before);
    base += before;
    bucket = buckets;
    have = of_often;
    once = false;
    share(blockIdx.x - buckets, gridDim.x - buckets);
    if (chunks <= kSortThreads) load_cuts(0);
    every([&](bool has, uint32_t, uint32_t pos, uint32_t at) {
      if (has) {
        perm[base + at] = pos;
        sorted[base + at] = often;
      }
    });
    return;
  }

  uint32_t *cnt = counts + wave * at_once;
  for (uint32_t s0 = 0; s0 < mine; s0 += at_once) {
    const uint32_t ids = min(at_once, mine - s0), from = lo + s0;
    for (uint32_t i = threadIdx.x; i < kSortWaves * at_once; i += kSortThreads) counts[i] = 0u;
    __syncthreads();
    every([&](bool has, uint32_t id, uint32_t, uint32_t) {
      id -= from;
      const bool hit = has && id < ids;
      const uint64_t hits = __ballot(hit);
      if (hits == 0) return;
      // one addition for all lanes that share the first one's id: an id that
      // fills the batch would be counted lane by lane
      const uint32_t lead = (uint32_t)__builtin_ctzll(hits);
      const bool same = hit && id == readlane_u32(id, lead);
      const uint32_t all = lanes_of(same);
      if (hit && (!same || lane == lead)) atomicAdd(&cnt[id], same ? all : 1u);
    });
    __syncthreads();

    // one thread per id: counts into cursors
    uint32_t total = 0, sum;
    if (threadIdx.x < ids) {
#pragma unroll
      for (uint32_t w = 0; w < kSortWaves; ++w) total += counts[w * at_once + threadIdx.x];
      // (the blocks that share them place them)
      if (from + threadIdx.x == often) total = of_often;
    }
    uint32_t at = base + block_prefix<kSortWaves>(total, lds, &sum);
    if (threadIdx.x < ids) {
      start[from + threadIdx.x] = at;
      if (from + threadIdx.x + 1 == v) start[v] = at + total;
#pragma unroll
      for (uint32_t w = 0; w < kSortWaves; ++w) {
        const uint32_t c = counts[w * at_once + threadIdx.x];
        counts[w * at_once + threadIdx.x] = at;
        at += c;
      }
    }
    base += sum;
    __syncthreads();

    every([&](bool has, uint32_t id, uint32_t pos, uint32_t) {
      id -= from;
      const bool hit = has && id < ids;
      uint32_t rank = 0, all = 0;
      uint64_t left = __ballot(hit);
      while (left != 0) {
        const bool same = hit && id == readlane_u32(id, (uint32_t)__builtin_ctzll(left));
        const uint64_t those = __ballot(same);
        rank = same ? (uint32_t)__popcll(those & lower) : rank;
        all = same ? (uint32_t)__popcll(those) : all;
        left &= ~those;
      }
      uint32_t to = 0;
      if (hit) {
        to = cnt[id];
        perm[to + rank] = pos;
        sorted[to + rank] = from + id;
      }
      wave_lds_sync();
      if (hit && rank == 0) cnt[id] = to + all;
      wave_lds_sync();
    });

    __syncthreads();  // the next ids reuse the counters
  }
}

// --- table gradient ---------------------------------------------------------

// to[at + j] = so_far + scale * acc[j] for the columns at + j in [c, c + kV)
// and below d (at < c in a row's last vector, where it is pulled back).
template <class O, uint32_t kV>
__device__ __forceinline__ void write_row(const O *so_far, O *to, uint32_t at, uint32_t c,
                                          uint32_t d, float scale, const float (&acc)[kV]) {
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
    store_stream(to + c, y);
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < kV; ++j)
    if (at + j >= c && at + j < d)
      to[at + j] = (O)((so_far != nullptr ? (float)so_far[at + j] : 0.0f) + scale * acc[j]);
}

constexpr uint32_t kSumThreads = 512;
constexpr uint32_t kSumGroups = 64;  // lane groups per block at most (their pieces are joined one by one)
constexpr uint32_t kRun = 8;         // sorted positions per lane group and round: rows in flight
constexpr uint32_t kSumWaves = 4096;
constexpr uint32_t kNone = 0xffffffffu;

__host__ __device__ constexpr uint32_t sum_threads(uint32_t lanes) {
  return kSumGroups * lanes < kSumThreads ? kSumGroups * lanes : kSumThreads;
}

// Sorted positions per block and round.
__host__ __device__ constexpr uint32_t window_of(uint32_t lanes) {
  return sum_threads(lanes) / lanes * kRun;
}

// What a window's last id leaves to later windows: the id, and how many
// windows it meets in all (0: it ends in this one).
struct Open {
  uint32_t id, windows;
};

// The table rows [r0, r1) that have no token: zeros, or add_to's row.
template <class O>
__device__ __forceinline__ void fill_rows(const uint32_t *__restrict__ start, uint32_t r0,
                                          uint32_t r1, uint32_t lanes, uint32_t d, const O *add_to,
                                          O *d_table, uint64_t ld) {
  constexpr uint32_t kU = 4;  // rows in flight
  const uint32_t groups = blockDim.x / lanes, c0 = (threadIdx.x & (lanes - 1)) * kVec<O>;
  for (uint32_t r = r0 + threadIdx.x / lanes; r < r1; r += groups * kU) {
    bool empty[kU];
#pragma unroll
    for (uint32_t u = 0; u < kU; ++u) {
      const uint32_t q = r + u * groups < r1 ? r + u * groups : r;
      empty[u] = start[q] == start[q + 1] && r + u * groups < r1;
    }
    if (add_to == nullptr) {
#pragma unroll
      for (uint32_t u = 0; u < kU; ++u)
        if (empty[u])
          for (uint32_t c = c0; c < d; c += lanes * kVec<O>)
            store_vec_tail<O, true>(d_table + (uint64_t)(r + u * groups) * ld, c, d, Vec<O>{});
      continue;
    }
    for (uint32_t c = c0; c < d; c += lanes * kVec<O>) {
      Vec<O> y[kU];
#pragma unroll
      for (uint32_t u = 0; u < kU; ++u)
        if (empty[u])
          y[u] = load_vec_tail(add_to + (uint64_t)(r + u * groups) * ld, c, d, (O)0.0f);
#pragma unroll
      for (uint32_t u = 0; u < kU; ++u)
        if (empty[u])
          store_vec_tail<O, true>(d_table + (uint64_t)(r + u * groups) * ld, c, d, y[u]);
    }
  }
}

// The sums of d_y's rows by id, over windows of sorted positions, so that the
// work goes by tokens however they are spread over the ids. Each lane group
// takes `rounds` times kRun positions, kRun rows in flight at once. An id that
// begins and ends among them is written; one that goes on from the group
// before leaves its piece in LDS, and the group where it began adds the pieces
// up in order. An id that crosses windows leaves a sum per window: part[2 w]
// of what came from the window before, part[2 w + 1] of what began in this one.
//
// A row's broken last vector is pulled back to end with the row (its first
// columns are summed twice and written once), and a lane past the row or a
// position past the end loads something that exists: no load has a branch, so
// they are all in flight together. kWhole: a group is a wave, whose positions
// and rows the scalar unit follows.
//
// The blocks after windows * slabs write the rows without a token, whose
// stores fill the time that the sums' loads take (32768 x 1024 bf16 into 65536
// f32 rows: 67 us for 332 MB, 5 TB/s; in a launch of their own 30 + 42).
template <class T, class O, bool kWhole>
__global__ void __launch_bounds__(kSumThreads)
    embed_grad_sum_kernel(const uint32_t *__restrict__ perm, const uint32_t *__restrict__ sorted,
                          const uint32_t *__restrict__ start, uint32_t windows, uint32_t slabs,
                          uint32_t lanes_, uint32_t rounds, const T *__restrict__ d_out,
                          uint64_t d_out_ld, uint32_t v, uint32_t d, float scale, const O *add_to,
                          O *d_table, uint64_t d_table_ld, float *__restrict__ part,
                          Open *__restrict__ open, uint32_t fill_lanes, uint32_t fill) {
  constexpr uint32_t kV = kVec<T>;
  __shared__ float carry[kV][kSumThreads];
  __shared__ uint8_t goes_on[kSumGroups];  // the group's piece from before fills it and goes on
  const uint32_t w = blockIdx.x % max(windows, 1u), slab = blockIdx.x / max(windows, 1u);
  if (blockIdx.x >= windows * slabs) {
    const uint64_t r0 = (uint64_t)(blockIdx.x - windows * slabs) * fill;
    fill_rows<O>(start, (uint32_t)r0, r0 + fill < v ? (uint32_t)r0 + fill : v, fill_lanes, d,
                 add_to, d_table, d_table_ld);
    return;
  }
  const uint32_t lanes = kWhole ? kWave : lanes_;
  const uint32_t groups = blockDim.x / lanes;
  const uint32_t group =
      kWhole ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave))
             : threadIdx.x / lanes;
  const uint32_t lane = threadIdx.x & (lanes - 1);
  const uint32_t kept = start[v];
  const uint32_t run = rounds * kRun, window = groups * run;
  const uint32_t w0 = w * window;
  if (w0 >= kept) {
    if (threadIdx.x == 0 && slab == 0) open[w] = Open{0, 0};
    return;
  }
  const uint32_t col = (slab * lanes + lane) * kV;
  const uint32_t at = d < kV ? 0u : col < d - kV ? col : d - kV;
  float acc[kV] = {};
  auto finish = [&](uint32_t t) {
    if (col < d)
      write_row<O, kV>(add_to != nullptr ? add_to + (uint64_t)t * d_table_ld : nullptr,
                       d_table + (uint64_t)t * d_table_ld, at, col, d, scale, acc);
  };
  auto leave = [&]() {
#pragma unroll
    for (uint32_t j = 0; j < kV; ++j) carry[j][threadIdx.x] = acc[j];
  };
  const uint32_t p0 = w0 + group * run, p1 = p0 + run < kept ? p0 + run : kept;
  const uint32_t before = p0 > 0 && p0 < kept ? sorted[p0 - 1] : kNone;
  const bool came = before != kNone && sorted[p0] == before;
  bool joined = came;  // the piece at hand goes on from before
  uint32_t last = kNone, after = kNone;
  for (uint32_t p = p0; p < p1; p += kRun) {
    uint32_t id[kRun];
    const T *row[kRun];
#pragma unroll
    for (uint32_t u = 0; u < kRun; ++u) {
      const uint32_t q = p + u < p1 ? p + u : p;
      id[u] = p + u < p1 ? sorted[q] : kNone;
      row[u] = d_out + (uint64_t)perm[q] * d_out_ld;
    }
    after = p + kRun < kept ? sorted[p + kRun] : kNone;
    Vec<T> x[kRun];
    if (d >= kV) {
#pragma unroll
      for (uint32_t u = 0; u < kRun; ++u) x[u] = load_vec(row[u] + at);
    } else {
#pragma unroll
      for (uint32_t u = 0; u < kRun; ++u)
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j) x[u][j] = row[u][j < d ? j : 0u];
    }
#pragma unroll
    for (uint32_t u = 0; u < kRun; ++u) {
      if (id[u] == kNone) break;
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) acc[j] += (float)x[u][j];
      const uint32_t next = u + 1 < kRun ? id[u + 1 < kRun ? u + 1 : u] : after;
      if (next == id[u]) continue;
      if (joined) leave();
      else finish(id[u]);
      joined = false;
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) acc[j] = 0.0f;
    }
    last = id[kRun - 1];
  }
  // what is left at the end goes on in the next group
  const bool more = last != kNone && last == after;
  if (more && joined) leave();
  if (lane == 0) goes_on[group] = more && joined ? 1 : 0;
  __syncthreads();

  const bool owner = more && !joined;
  bool past = false;
  if (owner) {
    uint32_t g = group;  // the last group whose piece is in acc
    do {
      ++g;
      if (g == groups) {
        past = true;
        break;
      }
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) acc[j] += carry[j][g * lanes + lane];
    } while (goes_on[g]);
    if (past) {
      if (col < d)
        write_row<float, kV>(nullptr, part + (2 * (uint64_t)w + 1) * d, at, col, d, 1.0f, acc);
      if (slab == 0 && lane == 0) open[w] = Open{last, (start[last + 1] - 1) / window - w + 1};
    } else {
      finish(last);
    }
  }
  if (group == 0 && came) {  // the id of the window before: its pieces from here on
    float sum[kV];
#pragma unroll
    for (uint32_t j = 0; j < kV; ++j) sum[j] = carry[j][lane];
    for (uint32_t h = 0; goes_on[h] && h + 1 < groups; ++h)
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) sum[j] += carry[j][(h + 1) * lanes + lane];
    if (col < d) write_row<float, kV>(nullptr, part + 2 * (uint64_t)w * d, at, col, d, 1.0f, sum);
  }
  const bool any = __syncthreads_or(past);
  if (!any && threadIdx.x == 0 && slab == 0) open[w] = Open{0, 0};
}

// Joins the parts of the ids that cross windows. A wave per window and 256
// columns adds up to kWaveParts of them; an id with more is left to the whole
// block (it crosses more windows than the block has, so there is one at most):
// its waves take equal runs of the parts, then their sums are added in order.
constexpr uint32_t kJoinThreads = 1024;
constexpr uint32_t kJoinWaves = kJoinThreads / kWave;
constexpr uint32_t kWaveParts = 2 * kJoinWaves;
constexpr uint32_t kPartUnroll = 8;

// acc += the parts [k0, k1) of the id that begins in window w.
__device__ __forceinline__ void sum_parts(const float *__restrict__ part, uint64_t w, uint32_t k0,
                                          uint32_t k1, uint32_t c, uint32_t d, float (&acc)[4]) {
  for (uint32_t k = k0; k < k1; k += kPartUnroll) {
    Vec<float> x[kPartUnroll];
#pragma unroll
    for (uint32_t u = 0; u < kPartUnroll; ++u) {
      const uint64_t slot = 2 * (w + k + u) + (k + u == 0 ? 1 : 0);
      x[u] = Vec<float>{};
      if (k + u < k1) x[u] = load_vec_tail(part + slot * d, c, d, 0.0f);
    }
#pragma unroll
    for (uint32_t u = 0; u < kPartUnroll; ++u)
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) acc[j] += x[u][j];
  }
}

template <class O>
__global__ void __launch_bounds__(kJoinThreads)
    embed_grad_join_kernel(const Open *__restrict__ open, uint32_t windows, uint32_t d, float scale,
                           const O *add_to, O *d_table, uint64_t d_table_ld,
                           const float *__restrict__ part) {
  __shared__ float sums[kJoinWaves][kWave * 4];
  __shared__ uint32_t many;
  const uint32_t lane = lane_id(), wave = threadIdx.x / kWave;
  const uint32_t c = (blockIdx.y * kWave + lane) * 4;
  if (threadIdx.x == 0) many = kNone;
  __syncthreads();
  const uint32_t w = blockIdx.x * kJoinWaves + wave;
  const Open mine = w < windows ? open[w] : Open{0, 0};
  float acc[4] = {};
  auto finish = [&](uint32_t id) {
    write_row<O, 4>(add_to != nullptr ? add_to + (uint64_t)id * d_table_ld : nullptr,
                    d_table + (uint64_t)id * d_table_ld, c, c, d, scale, acc);
  };
  if (mine.windows > kWaveParts) {
    if (lane == 0) many = w;
  } else if (mine.windows > 0 && c < d) {
    sum_parts(part, w, 0, mine.windows, c, d, acc);
    finish(mine.id);
  }
  __syncthreads();
  if (many == kNone) return;
  const Open all = open[many];
  const uint32_t run = (all.windows + kJoinWaves - 1) / kJoinWaves;
  const uint32_t k0 = min(wave * run, all.windows), k1 = min(k0 + run, all.windows);
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) acc[j] = 0.0f;
  if (c < d) sum_parts(part, many, k0, k1, c, d, acc);
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) sums[wave][lane * 4 + j] = acc[j];
  __syncthreads();
  if (wave != 0 || c >= d) return;
  for (uint32_t q = 1; q < kJoinWaves; ++q)
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) acc[j] += sums[q][lane * 4 + j];
  finish(all.id);
}

// Few tokens: the whole gradient in one launch. A block has `rows` table rows
// (and a slab of columns); it looks at all tokens, a thread each, orders those
// of its rows by (id, position) in LDS, and sums each id's rows of d_y: a lane
// group an id, or, where an id has more than kGroupRows of them, all groups in
// equal runs whose pieces are then added in order. 256 tokens of 20000 ids of 64
// columns 8.2 us against 11.9 in the launches above, of 262144 of one column 8.1
// and 15.9, of 40 of 300 7.8 and 13.2; all of one id 17 and 13, 512 of 20000 10.9
// and 12.4: hence the limits.
constexpr uint32_t kFewThreads = 512;
constexpr uint32_t kFewWaves = kFewThreads / kWave;
constexpr uint32_t kFewRows = 4096;
constexpr uint32_t kFewTokens = 256;
constexpr uint32_t kFewTimes = 16;  // tokens per id, on average
constexpr uint32_t kFewBlocks = 1024;
constexpr uint32_t kFewBytes = 8192;  // of table rows per block
constexpr uint32_t kGroupRows = 4 * kRun;

template <class T, class O>
__global__ void __launch_bounds__(kFewThreads)
    embed_grad_few_kernel(const int32_t *__restrict__ tokens, uint32_t n, uint32_t v, uint32_t rows,
                          uint32_t slabs, uint32_t lanes, const T *__restrict__ d_out,
                          uint64_t d_out_ld, uint32_t d, float scale, const O *add_to, O *d_table,
                          uint64_t d_table_ld, uint32_t *__restrict__ status) {
  constexpr uint32_t kV = kVec<T>;
  __shared__ uint32_t lds[kFewWaves], used[kFewRows / 32];
  __shared__ alignas(16) uint32_t ids[kFewTokens];
  __shared__ uint32_t perm[kFewTokens], from[kFewTokens];
  __shared__ uint32_t head[kFewTokens], begin[kFewTokens + 1];
  __shared__ float piece[kV][kFewThreads];
  const uint32_t slab = blockIdx.x % slabs, lo = blockIdx.x / slabs * rows;
  const uint32_t mine = min(rows, v - lo);
  const int32_t t = threadIdx.x < n ? tokens[threadIdx.x] : -1;
  const bool bad = t >= (int32_t)v;
  const bool hit = t >= 0 && (uint32_t)t - lo < mine;
  for (uint32_t i = threadIdx.x; i < (mine + 31) / 32; i += kFewThreads) used[i] = 0u;
  if (threadIdx.x < kFewTokens) ids[threadIdx.x] = kNone;
  uint32_t hits, heads, all;
  const uint32_t place = block_prefix<kFewWaves>(hit ? 1u : 0u, lds, &hits);
  if (hit) {
    const uint32_t id = (uint32_t)t - lo;
    ids[place] = id;
    atomicOr(&used[id / 32], 1u << (id % 32));
  }
  const bool any_bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = any_bad ? kFlagBadIndex : 0u;

  const uint32_t lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes;
  const uint32_t groups = kFewThreads / lanes;
  if (add_to != d_table) {  // rows without a token: zeros, or add_to's
    const uint32_t c1 = min((slab + 1) * lanes * kV, d);
    constexpr uint32_t kU = 4;  // rows in flight
    for (uint32_t r = group; r < mine; r += groups * kU) {
      bool empty[kU];
#pragma unroll
      for (uint32_t u = 0; u < kU; ++u) {
        const uint32_t q = r + u * groups < mine ? r + u * groups : r;
        empty[u] = (used[q / 32] >> (q % 32) & 1u) == 0 && r + u * groups < mine;
      }
      for (uint32_t c = slab * lanes * kV + lane * kVec<O>; c < c1; c += lanes * kVec<O>) {
        Vec<O> y[kU] = {};
        if (add_to != nullptr)
#pragma unroll
          for (uint32_t u = 0; u < kU; ++u)
            if (empty[u])
              y[u] = load_vec_tail(add_to + (uint64_t)(lo + r + u * groups) * d_table_ld, c, c1,
                                   (O)0.0f);
#pragma unroll
        for (uint32_t u = 0; u < kU; ++u)
          if (empty[u])
            store_vec_tail<O, true>(d_table + (uint64_t)(lo + r + u * groups) * d_table_ld, c, c1,
                                    y[u]);
      }
    }
  }
  if (hits == 0) return;

  // each hit's place: after the ids that come up before its own, and after the
  // hits of its id before it
  const uint32_t id = threadIdx.x < hits ? ids[threadIdx.x] : kNone;
  constexpr uint32_t kAtOnce = 16;  // (past the hits: kNone)
  uint32_t first = kNone, before = 0, times = 0;
  if (threadIdx.x < hits)
    for (uint32_t e = 0; e < hits; e += kAtOnce) {
      uint32_t other[kAtOnce];
#pragma unroll
      for (uint32_t u = 0; u < kAtOnce; ++u) other[u] = ids[e + u];
#pragma unroll
      for (uint32_t u = 0; u < kAtOnce; ++u) {
        const bool same = other[u] == id;
        first = same && first == kNone ? e + u : first;
        before += same && e + u < threadIdx.x ? 1u : 0u;
        times += same ? 1u : 0u;
      }
    }
  const bool leads = threadIdx.x < hits && before == 0;
  const uint32_t h = block_prefix<kFewWaves>(leads ? 1u : 0u, lds, &heads);
  const uint32_t at_first = block_prefix<kFewWaves>(leads ? times : 0u, lds, &all);
  if (leads) {
    from[threadIdx.x] = at_first;
    head[h] = id;
    begin[h] = at_first;
  }
  if (threadIdx.x == 0) begin[heads] = hits;
  __syncthreads();
  // (the hit's position is its thread's in the tokens, not in the list)
  if (threadIdx.x < hits) ids[threadIdx.x] = from[first] + before;
  __syncthreads();
  if (hit) perm[ids[place]] = threadIdx.x;
  __syncthreads();

  const uint32_t col = (slab * lanes + lane) * kV;
  const uint32_t at = d < kV ? 0u : col < d - kV ? col : d - kV;
  float acc[kV];
  auto add = [&](uint32_t p0, uint32_t p1) {
#pragma unroll
    for (uint32_t j = 0; j < kV; ++j) acc[j] = 0.0f;
    for (uint32_t p = p0; p < p1; p += kRun) {
      Vec<T> x[kRun];
#pragma unroll
      for (uint32_t u = 0; u < kRun; ++u) {
        const T *row = d_out + (uint64_t)perm[p + u < p1 ? p + u : p] * d_out_ld;
        if (d >= kV) x[u] = load_vec(row + at);
        else
#pragma unroll
          for (uint32_t j = 0; j < kV; ++j) x[u][j] = row[j < d ? j : 0u];
      }
#pragma unroll
      for (uint32_t u = 0; u < kRun; ++u)
        if (p + u < p1)
#pragma unroll
          for (uint32_t j = 0; j < kV; ++j) acc[j] += (float)x[u][j];
    }
  };
  auto finish = [&](uint32_t r) {
    const uint64_t row = (uint64_t)(lo + r) * d_table_ld;
    if (col < d)
      write_row<O, kV>(add_to != nullptr ? add_to + row : nullptr, d_table + row, at, col, d, scale,
                       acc);
  };
  for (uint32_t q = group; q < heads; q += groups) {
    if (begin[q + 1] - begin[q] > kGroupRows) continue;
    add(begin[q], begin[q + 1]);
    finish(head[q]);
  }
  const uint32_t parts = min(groups, kSumGroups);
  for (uint32_t q = 0; q < heads; ++q) {
    const uint32_t p = begin[q], len = begin[q + 1] - p;
    if (len <= kGroupRows) continue;
    if (group < parts) {
      add(p + len * group / parts, p + len * (group + 1) / parts);
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) piece[j][threadIdx.x] = acc[j];
    }
    __syncthreads();
    if (group == 0) {
      for (uint32_t g = 1; g < parts; ++g)
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j) acc[j] += piece[j][g * lanes + lane];
      finish(head[q]);
    }
    __syncthreads();  // the next id reuses the pieces
  }
}

}  // namespace

hipError_t launch_embed(const void *table, uint32_t dtype, uint32_t v, uint32_t d, uint64_t table_ld,
                        const int32_t *tokens, uint32_t n, float scale, void *out, uint64_t out_ld,
                        uint32_t *status, hipStream_t stream) {
  const bool one = one_block_reports(n, d, dtype_size(dtype));
  if (!one) {
    const hipError_t e = launch_status_clear(status, stream);
    if (e != hipSuccess || n == 0) return e;
  }
  return with_type(dtype, [&](auto x) {
    using T = decltype(x);
    const Cover cv = cover<kVec<T>>(d);
    const uint32_t tiles = div_up(n, kThreads / cv.lanes * kRows), most = kMaxBlocks / cv.slabs;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((tiles < most ? tiles : most) * cv.slabs), dim3(kThreads), 0, stream,
                         static_cast<const T *>(table), v, d, table_ld, tokens, n, scale,
                         static_cast<T *>(out), out_ld, cv.lanes, cv.slabs, status, !one);
    };
    if (cv.lanes < kWave) go(embed_kernel<T, false>);
    else go(embed_kernel<T, true>);
    return hipGetLastError();
  });
}

EmbedGradPlan plan_embed_grad(uint32_t n, uint32_t v, uint32_t d) {
  EmbedGradPlan p{};
  // buckets for every compute unit where the ids allow it, and fewer than the
  // chunks' counters: the cut after the last bucket needs one too, with or
  // without a frequent id
  while ((2u << p.shift) <= v / 256u && (1u << p.shift) < kSortIds) ++p.shift;
  p.own = n >= kOwnFrom && p.shift != 0;
  while (((uint64_t)(kMaxBuckets - 1) << p.shift) < v) ++p.shift;
  p.buckets = (uint32_t)(((uint64_t)v + (1u << p.shift) - 1) >> p.shift);
  p.counters = kMaxBuckets;
  p.per = n <= 32768 ? 1 : n <= 262144 ? 2 : 4;  // chunks grow with the tokens
  p.chunk_len = p.per * kChunkThreads;
  p.chunks = n <= kDirect ? 0 : div_up(n, p.chunk_len);
  // an f32 row takes more lanes, so its windows are smaller (one size covers
  // every type)
  const uint32_t windows = div_up(n, window_of(cover<kVec<float>>(d).lanes));
  size_t at = 0;
  auto take = [&](size_t words) {
    const size_t here = at;
    at += align_up(words * sizeof(uint32_t), 256);
    return here;
  };
  p.off_perm = take(n);
  p.off_sorted = take(n);
  p.off_start = take((size_t)v + 1);
  p.off_open = take(2 * (size_t)windows);
  p.off_entry_id = take(p.chunks != 0 ? n : 0);
  p.off_entry_pos = take(p.chunks != 0 ? n : 0);
  p.off_cuts = take((size_t)p.chunks * (p.buckets + 3));
  p.off_frequent = take(p.chunks != 0 ? 1 : 0);
  p.off_part = take((size_t)windows * 2 * d);
  p.ws_bytes = at;
  return p;
}

hipError_t launch_embed_grad(const EmbedGradPlan &plan, const int32_t *tokens, uint32_t n,
                             const void *d_out, uint32_t d_out_type, uint64_t d_out_ld, uint32_t v,
                             uint32_t d, float scale, const void *add_to, void *d_table,
                             uint32_t d_table_type, uint64_t d_table_ld, void *ws, uint32_t *status,
                             hipStream_t stream) {
  char *base = static_cast<char *>(ws);
  auto words = [&](size_t off) { return reinterpret_cast<uint32_t *>(base + off); };
  uint32_t *perm = words(plan.off_perm), *sorted = words(plan.off_sorted);
  uint32_t *start = words(plan.off_start), *cuts = words(plan.off_cuts);
  uint32_t *frequent = words(plan.off_frequent);
  uint32_t *entry_id = words(plan.off_entry_id), *entry_pos = words(plan.off_entry_pos);
  Open *open = reinterpret_cast<Open *>(base + plan.off_open);
  float *part = reinterpret_cast<float *>(base + plan.off_part);
  if (n <= kFewTokens && n <= (uint64_t)kFewTimes * v) {
    const hipError_t e = with_type(d_out_type, [&](auto x) {
      using T = decltype(x);
      auto go = [&](auto y) {
        using O = decltype(y);
        const Cover cv = cover<kVec<T>>(d);
        // 8 KB of the table per block, but about eight tokens at most, and no
        // more blocks than start in one go
        const uint32_t bytes = kFewBytes / (cv.lanes * kVec<T> * (uint32_t)sizeof(O));
        const uint32_t eight = (uint32_t)((uint64_t)v * 8 / max(n, 8u));
        const uint32_t rows =
            max(div_up(v, div_up(kFewBlocks, cv.slabs)), max(min(bytes, eight), 1u));
        if (rows > kFewRows) return hipErrorNotSupported;
        hipLaunchKernelGGL((embed_grad_few_kernel<T, O>), dim3(div_up(v, rows) * cv.slabs),
                           dim3(kFewThreads), 0, stream, tokens, n, v, rows, cv.slabs, cv.lanes,
                           static_cast<const T *>(d_out), d_out_ld, d, scale,
                           static_cast<const O *>(add_to), static_cast<O *>(d_table), d_table_ld,
                           status);
        return hipGetLastError();
      };
      return d_table_type == (uint32_t)Dtype::f32 ? go(float{}) : go(x);
    });
    if (e != hipErrorNotSupported) return e;
  }
  if (plan.chunks != 0) {
    auto cut = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(plan.chunks), dim3(kChunkThreads), 0, stream, tokens, n, v,
                         plan.shift, plan.buckets, plan.own, entry_id, entry_pos, cuts,
                         frequent);
    };
    if (plan.per == 1) cut(token_chunk_kernel<1>);
    else if (plan.per == 2) cut(token_chunk_kernel<2>);
    else cut(token_chunk_kernel<4>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const uint32_t at_once = (1u << plan.shift) < kSortIds ? 1u << plan.shift : kSortIds;
  // few ids: their buckets hold many tokens each (131072 of one id: one block
  // 93 us, shared 6)
  const uint32_t share =
      plan.shift == 0 && plan.chunks != 0 ? div_up(kSortBlocks, plan.buckets) : 1u;
  // a batch for each wave of the blocks that share the frequent id
  const uint32_t helpers = plan.own ? min(kSortBlocks, div_up(n, 2048)) : 0u;
  auto sort = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(plan.buckets + helpers, share), dim3(kSortThreads),
                       kSortWaves * at_once * sizeof(uint32_t), stream, tokens, n, v, plan.shift,
                       plan.buckets, cuts, plan.chunks, plan.chunk_len, entry_id,
                       entry_pos, frequent, perm, sorted, start, status);
  };
  if (plan.chunks != 0) sort(token_sort_kernel<false>);
  else sort(token_sort_kernel<true>);
  const hipError_t sorting = hipGetLastError();
  if (sorting != hipSuccess) return sorting;
  return with_type(d_out_type, [&](auto x) {
    using T = decltype(x);
    auto go = [&](auto y) {
      using O = decltype(y);
      const O *add = static_cast<const O *>(add_to);
      O *to = static_cast<O *>(d_table);
      const Cover cv = cover<kVec<T>>(d);
      const uint32_t threads = sum_threads(cv.lanes);
      // as many rounds as still fill the card: fewer windows for the ids that
      // fill many of them
      const uint64_t waves =
          (uint64_t)div_up(n, window_of(cv.lanes)) * cv.slabs * (threads / kWave);
      const uint32_t rounds = waves > kSumWaves ? (uint32_t)(waves / kSumWaves) : 1u;
      const uint32_t windows = div_up(n, (uint64_t)window_of(cv.lanes) * rounds);
      // rows without a token: 8 KB per wave, four rows per lane group at least
      const uint32_t fill_lanes = cover<kVec<O>>(d).lanes;
      const uint32_t most = threads / kWave * (8192 / sizeof(O)) / d;
      const uint32_t least = threads / fill_lanes * 4;
      const uint32_t fill = most > least ? most : least;
      const uint32_t fill_blocks = add == to ? 0 : div_up(v, fill);
      const uint32_t blocks = windows * cv.slabs + fill_blocks;
      if (blocks == 0) return hipSuccess;
      auto sum = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(blocks), dim3(threads), 0, stream, perm, sorted, start,
                           windows, cv.slabs, cv.lanes, rounds, static_cast<const T *>(d_out),
                           d_out_ld, v, d, scale, add, to, d_table_ld, part, open, fill_lanes,
                           fill);
      };
      if (cv.lanes < kWave) sum(embed_grad_sum_kernel<T, O, false>);
      else sum(embed_grad_sum_kernel<T, O, true>);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess || windows <= 1) return e;
      hipLaunchKernelGGL((embed_grad_join_kernel<O>),
                         dim3(div_up(windows, kJoinWaves), div_up(d, kWave * 4)),
                         dim3(kJoinThreads), 0, stream, open, windows, d, scale, add, to,
                         d_table_ld, part);
      return hipGetLastError();
    };
    return d_table_type == (uint32_t)Dtype::f32 ? go(float{}) : go(x);
  });
}

}  // namespace seacells
