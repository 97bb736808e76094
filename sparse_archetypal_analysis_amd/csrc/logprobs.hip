// Log probabilities of given classes, entropy and top alternatives of rows of
// logits, and their gradient.
//
//   m = max x, s = log sum exp(x - m)
//   log p_c = x_c - m - s      entropy H = s - sum p_c (x_c - m)
//   d_x = d_logp (1[c = target] - p_c) - d_entropy p_c (log p_c + H)
//
// -inf logits are masked: their p is an exact 0 and the product with their
// logarithm is taken as 0. NaN and +inf leave a row without a distribution.
//
// Both directions are bound by memory: forward reads the logits once, with a
// running (maximum, sum exp, sum t exp) that is rescaled once per 64 bytes; the
// gradient reads and writes each element once.
//
// Alternatives cost no second pass: every lane (or thread) already has the
// maximum of its own elements, the top_k-th largest of those maxima bounds the
// top_k-th largest element from below, and only the few lanes whose maximum
// reaches that bound look for the elements that do. Those candidates - hardly
// more than top_k - are ordered by counting, with (value, lowest column first)
// as one 64-bit key.
#include "token.hpp"

namespace seacells {

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = kThreads / kWave;
constexpr uint32_t kMaxBlocks = 1u << 20;
constexpr uint32_t kMaxParts = kWave;  // a lane of the join per part
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLowest = -3.4028234663852886e38f;
// exp of anything below is 0 in f32 (log of the least denormal: -103.3);
// products with a probability of 0 stay finite
constexpr float kFloor = -200.0f;

__device__ __forceinline__ uint64_t u64max(uint64_t x, uint64_t y) { return x > y ? x : y; }

// Descending (value, lowest column first) as one ascending number; never 0.
__device__ __forceinline__ uint64_t top_key(float x, uint32_t c) {
  return ((uint64_t)f32_order(x) << 32) | (0xffffffffu - c);
}

// The sums of a set of logits against its maximum: s = sum e^t, u = sum t e^t,
// t = x - max(best, lowest finite). The lowest finite value stands in for the
// maximum of nothing, so masked entries get t = -inf and add an exact 0; a
// NaN or +inf makes s NaN. s = 0 says that nothing is left.
struct Sums {
  float best, s, u;
};

__device__ __forceinline__ float reference(float best) { return fmaxf(best, kLowest); }

// a's sums against the maximum `best` of a larger set.
__device__ __forceinline__ void rescale(Sums &a, float best) {
  const float t = nan_max(reference(a.best) - reference(best), kFloor);
  const float e = exp_neg(t);
  a.u = e * (a.u + t * a.s);
  a.s *= e;
  a.best = best;
}

template <uint32_t kLanes>
__device__ __forceinline__ void join_lanes(Sums &a) {
  rescale(a, group_max<kLanes>(a.best));
  a.s = group_sum<kLanes>(a.s);
  a.u = group_sum<kLanes>(a.u);
}

// Keeps the compiler from carrying what it computed of a vector past here.
template <class V>
__device__ __forceinline__ void hide(V &x) {
  typedef uint32_t Raw __attribute__((ext_vector_type(4)));
  Raw r = __builtin_bit_cast(Raw, x);
  asm volatile("" : "+v"(r));
  x = __builtin_bit_cast(V, r);
}

// Adds kN vectors (entries that are not there hold -inf).
template <class T, uint32_t kN>
__device__ __forceinline__ void add_vectors(Sums &a, Vec<T> (&x)[kN]) {
  float best = a.best;
#pragma unroll
  for (uint32_t k = 0; k < kN; ++k)
#pragma unroll
    for (uint32_t j = 0; j < kVec<T>; ++j) best = fmaxf(best, (float)x[k][j]);
  rescale(a, best);
  const float m = reference(best);
#pragma unroll
  for (uint32_t k = 0; k < kN; ++k) {
    if (sizeof(T) == 2 && kN > 1) hide(x[k]);  // unpacked again rather than held as f32
#pragma unroll
    for (uint32_t j = 0; j < kVec<T>; ++j) {
      const float t = nan_max((float)x[k][j] - m, kFloor);
      const float e = exp_neg(t);
      a.s += e;
      a.u += t * e;
    }
  }
}

// What a row's sums say: the logarithm of its sum, and whether it has a
// distribution at all.
struct Row {
  float m, log_sum;
  bool none, empty;
  __device__ __forceinline__ explicit Row(const Sums &a) {
    none = a.s != a.s;
    empty = a.s == 0.0f;
    m = a.best;
    log_sum = none ? a.s : empty ? 0.0f : logf(a.s);
  }
  __device__ __forceinline__ float log_p(float x) const {
    return none ? log_sum : x > kNegInf ? (x - m) - log_sum : kNegInf;
  }
};

struct Outputs {
  const int32_t *targets;
  float *logp, *entropy, *stats;
  int32_t *top_idx;
  float *top_logp;
  uint32_t top_k;
  uint32_t *status;
  bool check;  // flag targets past the row here (else one block looks at all)
};

// A row's target and its logit: two dependent loads, each started early enough
// not to be waited for.
template <class T>
struct Target {
  int32_t id;
  bool bad;
  T x;
  __device__ __forceinline__ Target(const Outputs &o, uint64_t i, uint32_t v) {
    id = o.targets != nullptr ? o.targets[i] : -1;
    bad = id >= 0 && (uint32_t)id >= v;
  }
  __device__ __forceinline__ void fetch(const Outputs &o, const T *row) {
    x = o.logp != nullptr && id >= 0 && !bad ? row[id] : (T)0.0f;
  }
};

// By one lane.
template <class T>
__device__ __forceinline__ void write_row(const Outputs &o, uint64_t i, const Target<T> &t,
                                          const Sums &a, const Row &r) {
  if (o.stats != nullptr) {
    o.stats[2 * i] = r.none ? r.log_sum : r.m;
    o.stats[2 * i + 1] = r.log_sum;
  }
  if (o.entropy != nullptr) o.entropy[i] = r.empty ? 0.0f : r.log_sum - a.u / a.s;
  if (t.bad && o.check) atomicOr(o.status, kFlagBadIndex);
  if (o.logp != nullptr) o.logp[i] = t.id < 0 || t.bad ? 0.0f : r.log_p((float)t.x);
}

__device__ __forceinline__ void write_top(const Outputs &o, uint64_t i, uint32_t place,
                                          uint64_t key, const Row &r) {
  o.top_idx[i * o.top_k + place] = key != 0 ? (int32_t)(0xffffffffu - (uint32_t)key) : -1;
  o.top_logp[i * o.top_k + place] = r.log_p(key != 0 ? f32_unorder((uint32_t)(key >> 32)) : kNegInf);
}

// The k-th largest of a wave's values, but at least the lowest finite one (what
// is below is masked), bit by bit of its order, whatever k is. reach(y) counts
// the values >= y (orders past infinity are NaN: none).
template <class F>
__device__ __forceinline__ float wave_bound(uint32_t k, F &&reach) {
  uint32_t at = 0;
  for (uint32_t bit = 1u << 31; bit != 0; bit >>= 1)
    at = reach(f32_unorder(at | bit)) >= k ? at | bit : at;
  return fmaxf(f32_unorder(at), kLowest);
}

// A bound of it from below for kN values per lane: 16 bits of its order, that is
// 7 of the mantissa (orders compared, not numbers: 5 operations a step).
template <uint32_t kN>
__device__ __forceinline__ float wave_bound_of(const float (&x)[kN], uint32_t k) {
  uint32_t key[kN];
#pragma unroll
  for (uint32_t j = 0; j < kN; ++j) key[j] = f32_order(x[j]);
  uint32_t at = 0;
#pragma unroll 4
  for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
    uint32_t reach = 0;
#pragma unroll
    for (uint32_t j = 0; j < kN; ++j) reach += lanes_of(key[j] >= (at | bit));
    at = reach >= k ? at | bit : at;
  }
  return fmaxf(f32_unorder(at), kLowest);
}

// A row of v logits over kStride lanes, kR vectors each: x[k] holds the
// elements from (k * kStride + at) * kVec<T>, -inf past the end. The row's one
// broken vector has a branch of its own (a branch in each load took up to
// twice the registers). Many vectors of halves are loaded without a branch,
// those past the end from the row's beginning, and chosen as whole words: put
// together from branches, each load was waited for before the next (100k x
// 2600 bf16 with 5 alternatives 198 us against 156; f32 and fewer vectors lose
// up to 9 % that way, 1300 f32 107 against 116).
template <class T, uint32_t kStride, uint32_t kR>
__device__ __forceinline__ void load_row(const T *row, uint32_t at, uint32_t v, bool live,
                                         Vec<T> (&x)[kR]) {
  constexpr uint32_t kV = kVec<T>;
  constexpr uint32_t kWords = kV * sizeof(T) / 4;
  typedef uint32_t Words __attribute__((ext_vector_type(kWords), aligned(sizeof(T))));
  const uint32_t last = v / kV;  // the broken vector, if there is one
  const bool broken = v % kV != 0 && live && at == last % kStride;
  if constexpr (sizeof(T) == 2 && kR > 4) {  // (rows this long have a whole vector)
    Vec<T> none;
    none = (T)kNegInf;
    const Words filled = __builtin_bit_cast(Words, none);
    Words w[kR];
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      const uint32_t c = (k * kStride + at) * kV;
      w[k] = *reinterpret_cast<const Words *>(row + (c + kV <= v ? c : 0u));
    }
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      const bool in = live && (k * kStride + at) * kV + kV <= v;
#pragma unroll
      for (uint32_t j = 0; j < kWords; ++j) w[k][j] = in ? w[k][j] : filled[j];
    }
    if (broken) {
      const Words y = __builtin_bit_cast(Words, load_vec_tail(row, last * kV, v, (T)kNegInf));
#pragma unroll
      for (uint32_t k = 0; k < kR; ++k)
        if (k == last / kStride) w[k] = y;
    }
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) x[k] = __builtin_bit_cast(Vec<T>, w[k]);
  } else {
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      const uint32_t c = (k * kStride + at) * kV;
      x[k] = (T)kNegInf;
      if (live && c + kV <= v) x[k] = load_vec(row + c);
    }
    if (broken) {
      const Vec<T> y = load_vec_tail(row, last * kV, v, (T)kNegInf);
#pragma unroll
      for (uint32_t k = 0; k < kR; ++k)
        if (k == last / kStride) x[k] = y;
    }
  }
}

// --- rows that a wave's registers hold ------------------------------------------

// Candidates that a wave orders.
constexpr uint32_t kTopRoom = 2 * kWave;

// The first top_k of `count` keys in LDS, kK of them per lane, written at
// their places: a key's place is the count of the larger ones.
template <uint32_t kK>
__device__ __forceinline__ void order_top(const Outputs &o, uint64_t i, const Row &r,
                                          const uint64_t *keys, uint32_t count) {
  const uint32_t lane = lane_id();
  uint64_t key[kK];
  uint32_t place[kK];
#pragma unroll
  for (uint32_t m = 0; m < kK; ++m) {
    key[m] = m * kWave + lane < count ? keys[m * kWave + lane] : 0ull;
    place[m] = 0;
  }
#pragma unroll
  for (uint32_t m = 0; m < kK; ++m) {
    const uint32_t hi = (uint32_t)(key[m] >> 32), lo = (uint32_t)key[m];
    const uint32_t here = min(count - min(count, m * kWave), kWave);
    for (uint32_t p = 0; p < here; ++p) {
      const uint64_t other = ((uint64_t)readlane_u32(hi, p) << 32) | readlane_u32(lo, p);
#pragma unroll
      for (uint32_t l = 0; l < kK; ++l) place[l] += other > key[l] ? 1u : 0u;
    }
  }
#pragma unroll
  for (uint32_t m = 0; m < kK; ++m) {
    const uint32_t q = m * kWave + lane < count ? place[m] : m * kWave + lane;
    if (q < o.top_k) write_top(o, i, q, key[m], r);
  }
}

// The alternatives of a row that a wave holds. A lane's largest element (mine)
// stands for its others: the bound that top_k of those reach, or of up to 8
// from each lane where the lanes are too few, leaves hardly more than top_k
// elements, which go to LDS and are ordered by counting. Should more than
// kTopRoom be left (many equals, or a bound too coarse), the
// top_k-th largest element itself is looked for, and of those that equal it
// the first columns are taken.
template <class T, uint32_t kR>
__device__ __forceinline__ void wave_top(const Outputs &o, uint64_t i, uint32_t v, Vec<T> (&x)[kR],
                                         float mine, const Row &r, uint64_t *keys) {
  constexpr uint32_t kV = kVec<T>;
  constexpr uint32_t kE = kR * kV;
  const uint32_t lane = lane_id(), top_k = o.top_k;
  if (r.none) {
    if (lane < top_k) write_top(o, i, lane, 0ull, r);
    return;
  }
  // (what was computed of the elements before is not carried this far: it
  // would take up to 220 registers, 2 waves per SIMD)
#pragma unroll
  for (uint32_t k = 0; k < kR; ++k) hide(x[k]);
  float least;
  if (2 * top_k <= min((v + kV - 1) / kV, kWave)) {
    const float sets[1] = {mine};
    least = wave_bound_of<1>(sets, top_k);
  } else {
    constexpr uint32_t kSets = kE < 8 ? kE : 8;
    float sets[kSets];
#pragma unroll
    for (uint32_t e = 0; e < kE; ++e)
      sets[e % kSets] = e < kSets ? (float)x[e / kV][e % kV]
                                  : fmaxf(sets[e % kSets], (float)x[e / kV][e % kV]);
    least = wave_bound_of<kSets>(sets, top_k);
  }
  uint32_t first = lane * kV;      // the lane's first column
  asm volatile("" : "+v"(first));  // (not one register per element's)
#pragma unroll
  for (uint32_t k = 0; k < kR; ++k) hide(x[k]);
  const uint64_t lower = (1ull << lane) - 1ull;
  uint32_t count = 0;
#pragma unroll
  for (uint32_t k = 0; k < kR; ++k)
#pragma unroll
    for (uint32_t j = 0; j < kV; ++j) {
      const float y = (float)x[k][j];
      const bool hit = y >= least;
      const uint64_t hits = __ballot(hit);
      if (hits == 0) continue;
      const uint32_t place = count + (uint32_t)__popcll(hits & lower);
      if (hit && place < kTopRoom) keys[place] = top_key(y, first + k * kWave * kV + j);
      count += (uint32_t)__popcll(hits);
    }
  if (count > kTopRoom) {
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) hide(x[k]);
    const float kth = wave_bound(top_k, [&](float y) {
      uint32_t c = 0;
#pragma unroll
      for (uint32_t k = 0; k < kR; ++k) hide(x[k]);
#pragma unroll
      for (uint32_t e = 0; e < kE; ++e) c += lanes_of((float)x[e / kV][e % kV] >= y);
      return c;
    });
    count = 0;
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) hide(x[k]);
#pragma unroll
    for (uint32_t e = 0; e < kE; ++e) count += lanes_of((float)x[e / kV][e % kV] > kth);
    uint32_t above = 0, equal = count;  // places of the larger ones, then of the equal ones
    // vectors in the order of their columns: by k, then lane, then element
#pragma unroll
    for (uint32_t k = 0; k < kR; ++k) {
      hide(x[k]);
      uint32_t mine_equal = equal, all_equal = 0;
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) {
        const uint64_t same = __ballot((float)x[k][j] == kth);
        mine_equal += (uint32_t)__popcll(same & lower);
        all_equal += (uint32_t)__popcll(same);
      }
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) {
        const float y = (float)x[k][j];
        const uint64_t hits = __ballot(y > kth);
        const uint32_t place = y == kth ? mine_equal : above + (uint32_t)__popcll(hits & lower);
        if (y >= kth && place < kWave) keys[place] = top_key(y, first + k * kWave * kV + j);
        mine_equal += y == kth ? 1u : 0u;
        above += (uint32_t)__popcll(hits);
      }
      equal += all_equal;
    }
    count = equal < kWave ? equal : kWave;
  }
  wave_lds_sync();
  if (count <= kWave) order_top<1>(o, i, r, keys, count);
  else order_top<kTopRoom / kWave>(o, i, r, keys, count);
  wave_lds_sync();
}

// A row per kLanes lanes, kR vectors per lane.
template <class T, uint32_t kLanes, uint32_t kR>
__global__ void __launch_bounds__(kThreads)
    logprobs_held_kernel(const T *__restrict__ logits, uint32_t n, uint32_t v, uint64_t ld,
                         Outputs o) {
  constexpr uint32_t kV = kVec<T>;
  constexpr uint32_t kGroups = kThreads / kLanes;
  constexpr bool kWhole = kLanes == kWave;
  __shared__ uint64_t room[kWhole ? kWaves : 1][kWhole ? kTopRoom : 1];
  const uint32_t at = threadIdx.x % kLanes;
  // (a wave's row is the same in all its lanes, which the compiler cannot see)
  const uint32_t group = kWhole ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave))
                                : threadIdx.x / kLanes;
  const uint64_t step = (uint64_t)gridDim.x * kGroups;
  for (uint64_t i0 = (uint64_t)blockIdx.x * kGroups; i0 < n; i0 += step) {
    const uint64_t i = i0 + group;
    const bool live = i < n;
    const T *row = logits + (live ? i : 0) * ld;
    Vec<T> x[kR];
    load_row<T, kLanes, kR>(row, at, v, live, x);
    Target<T> target(o, live ? i : 0, v);
    target.fetch(o, row);
    Sums a{kNegInf, 0.0f, 0.0f};
    add_vectors<T, kR>(a, x);
    const float mine = a.best;
    join_lanes<kLanes>(a);
    const Row r(a);
    if (live && at == 0) write_row(o, i, target, a, r);
    if (o.top_k == 0) continue;

    if constexpr (kWhole) {
      if (live) wave_top<T, kR>(o, i, v, x, mine, r, room[group]);
    } else {
      // one alternative per round, kept by the lane of its place until all
      // lanes have one, which they write side by side (131072 x 60 f32 with 8:
      // written one by one 37 us, so 35; x 250 bf16 with 16, the elements held as
      // f32 and by the rule below 174 and 125)
      uint64_t kept = 0;
      constexpr uint32_t kE = kR * kV;
      float y[kE];
#pragma unroll
      for (uint32_t e = 0; e < kE; ++e) y[e] = (float)x[e / kV][e % kV];
      uint32_t first = at * kV;        // the lane's first column
      asm volatile("" : "+v"(first));  // (not one register per element's)
      for (uint32_t q = 0; q < o.top_k; ++q) {
        float best = kNegInf;
#pragma unroll
        for (uint32_t e = 0; e < kE; ++e) best = fmaxf(best, y[e]);
        best = r.none ? kNegInf : group_max<kLanes>(best);
        const uint32_t turn = q % kLanes;
        if (__ballot(best > kNegInf) == 0) {  // nothing left in any of the rows
          for (uint32_t p = q - turn + at; p < o.top_k; p += kLanes)
            if (live) write_top(o, i, p, p < q ? kept : 0ull, r);
          break;
        }
        // the lowest column that holds it, as an offset from the lane's first
        uint32_t c = 0xffffffffu;
#pragma unroll
        for (uint32_t e = kE; e-- > 0;)
          c = y[e] == best ? e / kV * kLanes * kV + e % kV : c;
        const uint32_t mine = c;
        c = group_min_u32<kLanes>(c != 0xffffffffu ? first + c : c);
        const uint32_t gone = first + mine == c ? mine : 0xffffffffu;
#pragma unroll
        for (uint32_t e = 0; e < kE; ++e)
          y[e] = gone == e / kV * kLanes * kV + e % kV ? kNegInf : y[e];
        if (at == turn) kept = best > kNegInf ? top_key(best, c) : 0ull;
        if (turn + 1 == kLanes || q + 1 == o.top_k)
          if (live && at <= turn) write_top(o, i, q - turn + at, kept, r);
      }
    }
  }
  // after the rows: the other blocks' work hides it
  if (blockIdx.x == 0 && !o.check)
    report_ids<kThreads>(o.targets, o.targets != nullptr ? n : 0u, v, o.status);
}

// --- rows that are streamed -------------------------------------------------------

constexpr uint32_t kUnroll = 4;   // vectors in flight per thread
constexpr uint32_t kRoom = 1024;  // candidates in LDS

struct Stream {
  float best[kThreads];
  Sums wave[kWaves];
  uint32_t holders, count;
  uint16_t holder[kThreads];
  uint64_t keys[kRoom];
  uint64_t wave_key[kWaves];
};

// The candidates of columns [q0, q1) (in vectors) go to sh.keys, best first at
// their place; f(place, key) is called by the thread that holds it, for the
// places below top_k, key 0 where nothing is left. `mine` is the maximum of
// the thread's own columns, every kThreads-th vector from q0 + its place. The
// columns of the threads whose maxima reach the bound ("holders", hardly more
// than top_k) are read again, by all threads: one latency, not a column's
// length of them (4096 x 50001 bf16 with 8: 5 of 87 us, else 29 of 111).
template <class T, class F>
__device__ __forceinline__ void block_top(Stream &sh, const T *row, uint32_t q0, uint32_t q1,
                                          uint32_t v, uint32_t top_k, float mine, F &&f) {
  constexpr uint32_t kV = kVec<T>;
  sh.best[threadIdx.x] = mine;
  if (threadIdx.x == 0) sh.holders = sh.count = 0;
  __syncthreads();
  float sets[kWaves];
#pragma unroll
  for (uint32_t k = 0; k < kWaves; ++k) sets[k] = sh.best[k * kWave + lane_id()];
  const float least = wave_bound_of<kWaves>(sets, top_k);
  if (mine >= least) sh.holder[atomicAdd(&sh.holders, 1u)] = (uint16_t)threadIdx.x;
  __syncthreads();
  const uint32_t holders = sh.holders;
  const uint32_t total = holders * ((q1 - q0 + kThreads - 1) / kThreads);
  constexpr uint32_t kAgain = 2;  // (4: 69 registers against 64, 1 to 5 % slower)
  for (uint32_t w = threadIdx.x; w < total; w += kThreads * kAgain) {
    Vec<T> x[kAgain];
    uint32_t at[kAgain];
#pragma unroll
    for (uint32_t u = 0; u < kAgain; ++u) {
      const uint32_t z = w + u * kThreads, turn = z / holders;
      const uint32_t q = z < total ? q0 + turn * kThreads + sh.holder[z - turn * holders] : q1;
      at[u] = q * kV;
      if (q < q1) x[u] = load_vec_tail(row, q * kV, v, (T)kNegInf);
      else x[u] = (T)kNegInf;
    }
#pragma unroll
    for (uint32_t u = 0; u < kAgain; ++u)
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) {
        const float y = (float)x[u][j];
        if (y >= least) {
          const uint32_t place = atomicAdd(&sh.count, 1u);
          if (place < kRoom) sh.keys[place] = top_key(y, at[u] + j);
        }
      }
  }
  __syncthreads();
  const uint32_t count = sh.count;
  if (count <= kRoom) {
    for (uint32_t q = threadIdx.x; q < (count > top_k ? count : top_k); q += kThreads) {
      const uint64_t key = q < count ? sh.keys[q] : 0ull;
      uint32_t place = 0;
#pragma unroll 8
      for (uint32_t p = 0; p < count; ++p) place += sh.keys[p] > key ? 1u : 0u;
      place = q < count ? place : q;
      if (place < top_k) f(place, key);
    }
    __syncthreads();
    return;
  }
  // many equals: one alternative per pass over the row
  uint64_t last = ~0ull;
  for (uint32_t k = 0; k < top_k; ++k) {
    uint64_t key = 0;
    for (uint32_t q = q0 + threadIdx.x; q < q1; q += kThreads) {
      const Vec<T> x = load_vec_tail(row, q * kV, v, (T)kNegInf);
#pragma unroll
      for (uint32_t j = 0; j < kV; ++j) {
        const uint64_t y = top_key((float)x[j], q * kV + j);
        if ((float)x[j] > kNegInf && y < last) key = u64max(key, y);
      }
    }
    for (int off = 32; off >= 1; off >>= 1)
      key = u64max(key, (uint64_t)__shfl_xor((unsigned long long)key, off, kWave));
    __syncthreads();
    if (lane_id() == 0) sh.wave_key[threadIdx.x / kWave] = key;
    __syncthreads();
    last = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) last = u64max(last, sh.wave_key[w]);
    if (threadIdx.x == 0) f(k, last);
  }
  __syncthreads();
}

// A block per part of a row (grid x: rows, y: parts). One part writes the
// row's outputs, several leave their sums and their candidates for the join.
template <class T>
__global__ void __launch_bounds__(kThreads)
    logprobs_stream_kernel(const T *__restrict__ logits, uint32_t n, uint32_t v, uint64_t ld,
                           Outputs o, Sums *__restrict__ part_sums, uint64_t *__restrict__ part_keys) {
  constexpr uint32_t kV = kVec<T>;
  __shared__ Stream sh;
  const uint32_t parts = gridDim.y, part = blockIdx.y;
  const uint32_t vecs = (v + kV - 1) / kV;
  const uint32_t q0 = (uint32_t)((uint64_t)vecs * part / parts);
  const uint32_t q1 = (uint32_t)((uint64_t)vecs * (part + 1) / parts);
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T *row = logits + i * ld;
    Target<T> target(o, i, v);
    Sums a{kNegInf, 0.0f, 0.0f};
    for (uint32_t q = q0; q < q1; q += kThreads * kUnroll) {
      Vec<T> x[kUnroll];
      if ((uint64_t)(q + kThreads * kUnroll) * kV <= v && q + kThreads * kUnroll <= q1) {
#pragma unroll
        for (uint32_t u = 0; u < kUnroll; ++u)
          x[u] = load_vec(row + (size_t)(q + u * kThreads + threadIdx.x) * kV);
      } else {
#pragma unroll
        for (uint32_t u = 0; u < kUnroll; ++u) {
          const uint32_t p = q + u * kThreads + threadIdx.x;
          if (p < q1) x[u] = load_vec_tail(row, p * kV, v, (T)kNegInf);
          else x[u] = (T)kNegInf;
        }
      }
      add_vectors<T, kUnroll>(a, x);
    }
    target.fetch(o, row);
    const float mine = a.best;
    join_lanes<kWave>(a);
    if (lane_id() == 0) sh.wave[threadIdx.x / kWave] = a;
    __syncthreads();
    float best = kNegInf;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) best = fmaxf(best, sh.wave[w].best);
    a = Sums{best, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
      Sums b = sh.wave[w];
      rescale(b, best);
      a.s += b.s;
      a.u += b.u;
    }
    __syncthreads();
    if (parts == 1) {
      const Row r(a);
      if (threadIdx.x == 0) write_row(o, i, target, a, r);
      if (o.top_k == 0) continue;
      if (r.none) {
        if (threadIdx.x < o.top_k) write_top(o, i, threadIdx.x, 0ull, r);
        continue;
      }
      block_top<T>(sh, row, q0, q1, v, o.top_k, mine,
                   [&](uint32_t place, uint64_t key) { write_top(o, i, place, key, r); });
    } else {
      if (threadIdx.x == 0) part_sums[i * parts + part] = a;
      if (o.top_k == 0) continue;
      uint64_t *to = part_keys + (i * parts + part) * o.top_k;
      block_top<T>(sh, row, q0, q1, v, o.top_k, mine,
                   [&](uint32_t place, uint64_t key) { to[place] = key; });
    }
  }
  // after the rows: the other blocks' work hides it
  if (blockIdx.x == 0 && part == 0 && !o.check)
    report_ids<kThreads>(o.targets, o.targets != nullptr ? n : 0u, v, o.status);
}

// The parts of a row, one per lane, in one wave: their sums joined, their
// ordered candidates merged from LDS, lane q keeping the q-th.
template <class T>
__global__ void __launch_bounds__(kWave)
    logprobs_join_kernel(const T *__restrict__ logits, uint32_t n, uint32_t v, uint64_t ld,
                         uint32_t parts, Outputs o, const Sums *__restrict__ part_sums,
                         const uint64_t *__restrict__ part_keys) {
  extern __shared__ uint64_t lists[];  // [parts][top_k]
  const uint32_t lane = lane_id(), top_k = o.top_k;
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const uint64_t *keys = part_keys + i * parts * top_k;
#pragma unroll 8
    for (uint32_t q = lane; q < parts * top_k; q += kWave) lists[q] = keys[q];
    Target<T> target(o, i, v);
    target.fetch(o, logits + i * ld);
    Sums a{kNegInf, 0.0f, 0.0f};
    if (lane < parts) a = part_sums[i * parts + lane];
    join_lanes<kWave>(a);
    const Row r(a);
    if (lane == 0) write_row(o, i, target, a, r);
    if (top_k == 0) continue;
    wave_lds_sync();
    uint32_t next = lane * top_k;
    uint64_t head = lane < parts && !r.none ? lists[next] : 0ull, mine = 0;
    for (uint32_t q = 0; q < top_k; ++q) {
      const uint32_t hi = ~wave_min_u32(~(uint32_t)(head >> 32));
      const uint32_t lo = ~wave_min_u32((uint32_t)(head >> 32) == hi ? ~(uint32_t)head : ~0u);
      const uint64_t key = ((uint64_t)hi << 32) | lo;
      if (lane == q) mine = key;
      if (key != 0 && head == key) head = ++next < (lane + 1) * top_k ? lists[next] : 0ull;
    }
    if (lane < top_k) write_top(o, i, lane, mine, r);
    wave_lds_sync();
  }
}

// --- gradient -----------------------------------------------------------------

constexpr uint32_t kGradUnroll = 4;  // vectors in flight per lane

// A row per `lanes` lanes (a power of two), or, few rows, a part of a row per
// block (grid y). Nothing is exchanged between lanes: an element's gradient
// needs the row's five numbers and itself, so a lane loads up to 4 vectors,
// then stores over them (d_logits may be logits; stores that the L2 gives up
// first gain 2 % here and lose 5 where rows are not aligned). Bound by memory: 8192 x
// 32768 bf16 204 us (5.3 TB/s; an element per lane and load: 406 us).
template <class T>
__global__ void __launch_bounds__(kThreads)
    logprobs_grad_kernel(const T *logits, uint32_t n, uint32_t v, uint64_t ld, uint32_t lanes,
                         const int32_t *__restrict__ targets, const float *__restrict__ stats,
                         const float *__restrict__ entropy, const float *__restrict__ d_logp,
                         const float *__restrict__ d_entropy, T *d_logits, uint64_t d_ld,
                         uint32_t *__restrict__ status, bool check) {
  constexpr uint32_t kV = kVec<T>;
  const uint32_t groups = kThreads / lanes;
  const uint32_t at = threadIdx.x & (lanes - 1);
  const uint32_t vecs = (v + kV - 1) / kV;
  const uint32_t q0 = (uint32_t)((uint64_t)vecs * blockIdx.y / gridDim.y);
  const uint32_t q1 = (uint32_t)((uint64_t)vecs * (blockIdx.y + 1) / gridDim.y);
  for (uint64_t i = (uint64_t)blockIdx.x * groups + threadIdx.x / lanes; i < n;
       i += (uint64_t)gridDim.x * groups) {
    const T *row = logits + i * ld;
    T *to = d_logits + i * d_ld;
    const int32_t t = targets != nullptr ? targets[i] : -1;
    const bool bad = t >= 0 && (uint32_t)t >= v;
    if (check && bad && at == 0) atomicOr(status, kFlagBadIndex);
    const bool has = t >= 0 && !bad;
    const float g = has && d_logp != nullptr ? d_logp[i] : 0.0f;
    const float h = d_entropy != nullptr ? d_entropy[i] : 0.0f;
    const float H = d_entropy != nullptr ? entropy[i] : 0.0f;
    float m = stats[2 * i];
    const float ls = stats[2 * i + 1];
    const bool none = m != m;     // no distribution: NaN throughout
    if (m == kNegInf) m = 0.0f;   // nothing left: every entry is masked
    const uint32_t hit = has ? (uint32_t)t : 0xffffffffu;
    for (uint32_t q = q0 + at; q < q1; q += lanes * kGradUnroll) {
      Vec<T> x[kGradUnroll];
#pragma unroll
      for (uint32_t u = 0; u < kGradUnroll; ++u) {
        const uint32_t p = q + u * lanes;
        if (p < q1) x[u] = load_vec_tail(row, p * kV, v, (T)kNegInf);
      }
#pragma unroll
      for (uint32_t u = 0; u < kGradUnroll; ++u) {
        const uint32_t p = q + u * lanes;
        if (p >= q1) break;
        Vec<T> y;
#pragma unroll
        for (uint32_t j = 0; j < kV; ++j) {
          const float z = (float)x[u][j];
          const float lp = nan_max(z - m - ls, kFloor);
          float d = -exp_neg(lp) * (g + h * (lp + H));
          d = hit == p * kV + j ? d + g : d;
          // masked entries get 0, whatever the row's d_logp and d_entropy are
          y[j] = (T)(z == kNegInf && !none ? 0.0f : d);
        }
        store_vec_tail(to, p * kV, v, y);
      }
    }
  }
  // after the rows: the other blocks' work hides it
  if (blockIdx.x == 0 && blockIdx.y == 0 && !check)
    report_ids<kThreads>(targets, targets != nullptr ? n : 0u, v, status);
}

uint32_t capped(uint64_t blocks) { return (uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks); }

// How a row that a wave's registers hold is spread over lanes.
template <uint32_t kLanes_, uint32_t kR_>
struct Group {
  static constexpr uint32_t lanes = kLanes_, vecs = kR_;
};

constexpr uint32_t kFewRows = 4096;  // four per SIMD

// f(Group) for rows of `vecs` vectors of kV logits, false where a wave's
// registers do not hold them. Rows this short are bound by the instructions of
// a wave, so the group with the fewest per row is taken, counted roughly: 10
// per element and 150 for the sums and the outputs of all rows of the wave;
// per alternative a round over the elements (few lanes), or a search and the
// candidates' order (a wave). 60000 rows, a wave per row against what is taken:
// 200 f32 26 and 15 us, with 8 alternatives 43 and 36, with 16 a wave; 500 bf16
// 36 and 25, with 4 50 and 43; 1000 bf16 41 and 32, with 1 51 and 42. Few rows
// leave units idle, and get a wave each (rows of up to 8 vectors 8 lanes).
template <uint32_t kV, class F>
bool held_group(uint32_t n, uint32_t vecs, uint32_t top_k, F &&f) {
  if (vecs > 512) return false;
  const uint32_t wide = vecs <= 64 ? 1 : vecs <= 128 ? 2 : vecs <= 192 ? 3 : vecs <= 256 ? 4
                      : vecs <= 384 ? 6 : 8;
  uint32_t least = 10 * kV * wide + 150 + (top_k != 0 ? 120 + 6 * top_k : 0u);
  uint32_t lanes = kWave, per = wide;
  if (n <= kFewRows) {
    if (vecs <= 8) lanes = 8;
  } else {
    for (uint32_t l = 8; l < kWave; l *= 2)
      for (uint32_t r = 1; r <= 4; r *= 2) {
        const uint32_t e = kV * r;
        const uint32_t cost = (10 * e + 150 + top_k * (5 * e + 40)) * l / kWave;
        if (l * r >= vecs && cost < least) {
          least = cost;
          lanes = l;
          per = r;
        }
      }
  }
  if (lanes == 8) {
    if (per == 1) f(Group<8, 1>{});
    else if (per == 2) f(Group<8, 2>{});
    else f(Group<8, 4>{});
  } else if (lanes == 16) {
    if (per == 1) f(Group<16, 1>{});
    else if (per == 2) f(Group<16, 2>{});
    else f(Group<16, 4>{});
  } else if (lanes == 32) {
    if (per == 1) f(Group<32, 1>{});
    else if (per == 2) f(Group<32, 2>{});
    else f(Group<32, 4>{});
  } else if (per == 1) {
    f(Group<64, 1>{});
  } else if (per == 2) {
    f(Group<64, 2>{});
  } else if (per == 3) {
    f(Group<64, 3>{});
  } else if (per == 4) {
    f(Group<64, 4>{});
  } else if (per == 6) {
    f(Group<64, 6>{});
  } else {
    f(Group<64, 8>{});
  }
  return true;
}

constexpr uint32_t kHeldVecs = 512;
constexpr uint32_t kFillBlocks = 512;               // two blocks per compute unit
constexpr uint32_t kGradBlocks = 4096;  // (600 x 30000 f32: 512 36 us, 2048 33, 4096 32.6)
constexpr uint32_t kPartVecs = kThreads * kUnroll;  // least part of a row

}  // namespace

LogprobsPlan plan_logprobs(uint32_t dtype, uint32_t n, uint32_t v, uint32_t top_k) {
  LogprobsPlan p{};
  const uint32_t vecs = div_up(v, kVecBytes / dtype_size(dtype));
  p.parts = 1;
  if (vecs > kHeldVecs && n > 0 && n < kFillBlocks / 2) {
    const uint32_t fill = kFillBlocks / n, most = div_up(vecs, kPartVecs);
    p.parts = fill < most ? fill : most;
    p.parts = p.parts < kMaxParts ? p.parts : kMaxParts;
  }
  if (p.parts > 1) {
    p.off_keys = align_up((size_t)n * p.parts * sizeof(Sums), 256);
    p.ws_bytes = p.off_keys + (size_t)n * p.parts * top_k * sizeof(uint64_t);
  }
  return p;
}

hipError_t launch_logprobs(const LogprobsPlan &plan, const void *logits, uint32_t dtype, uint32_t n,
                           uint32_t v, uint64_t ld, const int32_t *targets, uint32_t top_k,
                           float *logp, float *entropy, float *stats, int32_t *top_idx,
                           float *top_logp, void *ws, uint32_t *status, hipStream_t stream) {
  // one block looks at all targets, or the status is cleared first
  const bool one = one_block_reports(targets != nullptr ? n : n != 0, v, dtype_size(dtype));
  if (!one) {
    const hipError_t e = launch_status_clear(status, stream);
    if (e != hipSuccess || n == 0) return e;
  }
  const Outputs o{targets, logp, entropy, stats, top_idx, top_logp, top_k, status, !one};
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const T *x = static_cast<const T *>(logits);
    const bool held = held_group<kVec<T>>(n, div_up(v, kVec<T>), top_k, [&](auto g) {
      using G = decltype(g);
      hipLaunchKernelGGL((logprobs_held_kernel<T, G::lanes, G::vecs>),
                         dim3(capped(div_up(n, kThreads / G::lanes))), dim3(kThreads), 0, stream, x,
                         n, v, ld, o);
    });
    if (held) return hipGetLastError();
    Sums *sums = static_cast<Sums *>(ws);
    uint64_t *keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + plan.off_keys);
    hipLaunchKernelGGL((logprobs_stream_kernel<T>), dim3(capped(n), plan.parts), dim3(kThreads), 0,
                       stream, x, n, v, ld, o, sums, keys);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || plan.parts == 1) return e;
    hipLaunchKernelGGL((logprobs_join_kernel<T>), dim3(n), dim3(kWave),
                       plan.parts * top_k * sizeof(uint64_t), stream, x, n, v, ld, plan.parts, o,
                       sums, keys);
    return hipGetLastError();
  });
}

hipError_t launch_logprobs_grad(const void *logits, uint32_t dtype, uint32_t n, uint32_t v,
                                uint64_t ld, const int32_t *targets, const float *stats,
                                const float *entropy, const float *d_logp, const float *d_entropy,
                                void *d_logits, uint64_t d_logits_ld, uint32_t *status,
                                hipStream_t stream) {
  const bool one = one_block_reports(targets != nullptr ? n : n != 0, v, dtype_size(dtype));
  if (!one) {
    const hipError_t e = launch_status_clear(status, stream);
    if (e != hipSuccess || n == 0) return e;
  }
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const uint32_t vecs = div_up(v, kVec<T>);
    // as few lanes as hold the row in one round of loads (100k x 130 f32: a wave
    // per row 57 us, 16 lanes 29 us), more where the rows leave lanes idle
    uint32_t lanes = 8;
    while (lanes < kThreads && (lanes * kGradUnroll < vecs ||
                                (lanes < vecs && div_up(n, kThreads / lanes) < kFillBlocks)))
      lanes *= 2;
    const uint64_t blocks = div_up(n, kThreads / lanes);
    // few rows: parts of a row until the card is full, a vector per lane at least
    const uint32_t most = div_up(vecs, kThreads);
    const uint32_t fill = blocks < kGradBlocks ? (uint32_t)(kGradBlocks / blocks) : 1u;
    const uint32_t parts = lanes < kThreads ? 1u : fill < most ? fill : most;
    hipLaunchKernelGGL((logprobs_grad_kernel<T>), dim3(capped(blocks), parts), dim3(kThreads), 0,
                       stream, static_cast<const T *>(logits), n, v, ld, lanes, targets, stats,
                       entropy, d_logp, d_entropy, static_cast<T *>(d_logits), d_logits_ld, status,
                       !one);
    return hipGetLastError();
  });
}

}  // namespace seacells
