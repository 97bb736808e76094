// Element access and reductions shared by the token operators (embedding,
// layer norm, log probabilities), and their internal host interface. Nothing
// here is exported.
#pragma once

#include "common.hpp"

namespace seacells {

// Device-side element types, same values as SEACELLS_F32 / F16 / BF16.
enum class Dtype : uint32_t { f32 = 0, f16 = 1, bf16 = 2 };

constexpr uint32_t kVecBytes = 16;  // one lane's load or store
template <class T>
constexpr uint32_t kVec = kVecBytes / sizeof(T);

// 16 bytes of elements at any element-aligned address: the global memory path
// takes dwordx4 accesses at any byte address, so odd widths, strides and
// offsets need no variant of their own (a row that starts inside a 64-byte
// line costs the wave one more line, not a narrower access).
template <class T>
using Vec = T __attribute__((ext_vector_type(kVec<T>), aligned(sizeof(T))));

template <class T>
__device__ __forceinline__ Vec<T> load_vec(const T *p) {
  return *reinterpret_cast<const Vec<T> *>(p);
}

template <class T>
__device__ __forceinline__ void store_vec(T *p, Vec<T> v) {
  *reinterpret_cast<Vec<T> *>(p) = v;
}

// A store whose lines the L2 gives up first: an output that is written once
// leaves the L2 to the inputs that are read again (lookup of 32768 rows of
// 2048 bf16 45 -> 40 us, 12000 of 8000 62 -> 46; layer norm 60499 x 940 f16
// 74 -> 66; a table's gradient 88 -> 83).
template <class V, class T>
__device__ __forceinline__ void store_stream(T *p, V v) {
  __builtin_nontemporal_store(v, reinterpret_cast<V *>(p));
}

// The elements of [at, end) that a lane's vector at `at` covers, at < end;
// those past the end read as `fill`. The last vector's elements are loaded at
// clamped places without a branch, so that the loads do not wait for each
// other (a branch per element took 8 memory latencies: 10 of 107 us for 4096
// rows of 50001 bf16).
template <class T>
__device__ __forceinline__ Vec<T> load_vec_tail(const T *row, uint32_t at, uint32_t end, T fill) {
  if (at + kVec<T> <= end) return load_vec(row + at);
  Vec<T> v;
#pragma unroll
  for (uint32_t j = 0; j < kVec<T>; ++j) v[j] = row[at + j < end ? at + j : end - 1];
#pragma unroll
  for (uint32_t j = 0; j < kVec<T>; ++j) v[j] = at + j < end ? v[j] : fill;
  return v;
}

template <class T, bool kStream = false>
__device__ __forceinline__ void store_vec_tail(T *row, uint32_t at, uint32_t end, Vec<T> v) {
  if (at + kVec<T> <= end) {
    if (kStream) store_stream(row + at, v);
    else store_vec(row + at, v);
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < kVec<T>; ++j)
    if (at + j < end) row[at + j] = v[j];
}

// kN elements of any type at any element-aligned address (dwordx4 accesses,
// as many as they need).
template <class T, uint32_t kN>
using Pack = T __attribute__((ext_vector_type(kN), aligned(sizeof(T))));

template <class T, uint32_t kN>
__device__ __forceinline__ void store_pack_tail(T *row, uint32_t at, uint32_t end, Pack<T, kN> v) {
  if (at + kN <= end) {
    *reinterpret_cast<Pack<T, kN> *>(row + at) = v;
    return;
  }
#pragma unroll
  for (uint32_t j = 0; j < kN; ++j)
    if (at + j < end) row[at + j] = v[j];
}

// One DPP step: the value of another lane (0 where it has none or its row is
// masked off).
template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ float dpp_f32(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      0, (int)__float_as_uint(x), kCtrl, kRows, 0xF, false));
}

// As dpp_f32, but the lane's own value where it has none.
template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ float dpp_same_f32(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
      (int)__float_as_uint(x), (int)__float_as_uint(x), kCtrl, kRows, 0xF, false));
}

// How many lanes of the wave say yes.
__device__ __forceinline__ uint32_t lanes_of(bool x) { return (uint32_t)__popcll(__ballot(x)); }

// Sum over each group of kLanes neighbouring lanes (8, 16, 32 or 64) in a
// fixed order, the result in every lane of the group. Called with every lane
// active. quad_perm, half-row and row mirrors as in wave_min_u32; over the
// whole wave two row broadcasts and a lane read replace the last exchanges.
template <uint32_t kLanes>
__device__ __forceinline__ float group_sum(float x) {
  static_assert(kLanes == 8 || kLanes == 16 || kLanes == 32 || kLanes == 64, "group size");
  x += dpp_f32<0xB1>(x);
  x += dpp_f32<0x4E>(x);
  x += dpp_f32<0x141>(x);
  if (kLanes >= 16) x += dpp_f32<0x140>(x);
  if (kLanes == 32) x += __shfl_xor(x, 16, kWave);
  if (kLanes == 64) {
    x += dpp_f32<0x142, 0xA>(x);
    x += dpp_f32<0x143, 0xC>(x);
    x = readlane_f32(x, 63);
  }
  return x;
}

// Maximum over each group of kLanes neighbouring lanes, in every lane of the
// group. Called with every lane active; NaN loses against any number.
template <uint32_t kLanes>
__device__ __forceinline__ float group_max(float x) {
  x = fmaxf(x, dpp_same_f32<0xB1>(x));
  x = fmaxf(x, dpp_same_f32<0x4E>(x));
  x = fmaxf(x, dpp_same_f32<0x141>(x));
  if (kLanes >= 16) x = fmaxf(x, dpp_same_f32<0x140>(x));
  if (kLanes == 32) x = fmaxf(x, __shfl_xor(x, 16, kWave));
  if (kLanes == 64) {
    x = fmaxf(x, dpp_same_f32<0x142, 0xA>(x));
    x = fmaxf(x, dpp_same_f32<0x143, 0xC>(x));
    x = readlane_f32(x, 63);
  }
  return x;
}

// One DPP step of a minimum: the lane's own value where it has no partner.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_min_u32(uint32_t x) {
  return min(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, kCtrl, 0xF, 0xF, false));
}

template <uint32_t kLanes>
__device__ __forceinline__ uint32_t group_min_u32(uint32_t x) {
  if constexpr (kLanes == kWave) return wave_min_u32(x);
  x = dpp_min_u32<0xB1>(x);
  x = dpp_min_u32<0x4E>(x);
  x = dpp_min_u32<0x141>(x);
  if (kLanes >= 16) x = dpp_min_u32<0x140>(x);
  if (kLanes == 32) x = min(x, (uint32_t)__shfl_xor((int)x, 16, kWave));
  return x;
}

// Whether one block looks over all n ids (tokens, targets) beside the launch's
// work on rows of d elements of `size` bytes; otherwise each row's own lanes
// do, and the status word is cleared by a launch before (2 us). Lookup of 32768
// x 64 bf16 6.2 us by one block and 8.7 cleared, 131072 x 64 11.7 and 8.5, x 128
// 13.5 and 10.6, x 512 29.1 and 30.6; log probabilities 131072 x 250 f32 35.2 and
// 37.2, their gradient x 128 31.7 and 28.6, x 200 41.3 and 42.1.
inline bool one_block_reports(uint32_t n, uint32_t d, uint32_t size) {
  return n > 0 && (n <= 32768 || (uint64_t)d * size >= 600);
}

// *status = BAD_INDEX if any id is v or more, else 0; by one whole block.
template <uint32_t kBlock>
__device__ __forceinline__ void report_ids(const int32_t *__restrict__ ids, uint32_t n, uint32_t v,
                                           uint32_t *__restrict__ status) {
  typedef int32_t Four __attribute__((ext_vector_type(4), aligned(4)));
  bool bad = false;
  const uint32_t fours = n / 4;
#pragma unroll 8
  for (uint32_t i = threadIdx.x; i < fours; i += kBlock) {
    const Four t = *reinterpret_cast<const Four *>(ids + 4 * i);
    bad |= max(max(t.x, t.y), max(t.z, t.w)) >= (int32_t)v;
  }
  if (threadIdx.x < n % 4) bad |= ids[4 * fours + threadIdx.x] >= (int32_t)v;
  const bool any = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = any ? kFlagBadIndex : 0u;
}

// IEEE maximum: NaN if either side is (v_maximum3_f32 on gfx950).
__device__ __forceinline__ float nan_max(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}

// e^x for x <= 0 in one instruction beside the scaling (v_exp_f32, 1 ulp; the
// product's rounding adds |x| 2^-24 relative).
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

inline bool dtype_known(uint32_t t) { return t <= 2u; }
inline uint32_t dtype_size(uint32_t t) { return t == 0u ? 4u : 2u; }
inline uint32_t div_up(uint64_t a, uint64_t b) { return (uint32_t)((a + b - 1) / b); }

// Calls f(T{}) with the element type of a dtype code.
template <class F>
hipError_t with_type(uint32_t t, F &&f) {
  switch (static_cast<Dtype>(t)) {
    case Dtype::f32:
      return f(float{});
    case Dtype::f16:
      return f(_Float16{});
    default:
      return f(__bf16{});
  }
}

// --- host interface ---------------------------------------------------------

hipError_t launch_embed(const void *table, uint32_t dtype, uint32_t v, uint32_t d, uint64_t table_ld,
                        const int32_t *tokens, uint32_t n, float scale, void *out, uint64_t out_ld,
                        uint32_t *status, hipStream_t stream);

struct EmbedGradPlan {
  uint32_t shift;    // table rows per bucket of the token sort: 2^shift
  uint32_t buckets;
  uint32_t counters;  // of a chunk: the buckets' and the frequent id's fit
  uint32_t per;       // tokens of a chunk per thread
  uint32_t chunk_len;
  uint32_t chunks;   // 0: the buckets read the tokens themselves
  bool own;          // a frequent id has a bucket of its own
  size_t off_perm, off_sorted, off_start, off_open, off_entry_id, off_entry_pos, off_cuts, off_part,
      off_frequent;
  size_t ws_bytes;
};
EmbedGradPlan plan_embed_grad(uint32_t n, uint32_t v, uint32_t d);
hipError_t launch_embed_grad(const EmbedGradPlan &plan, const int32_t *tokens, uint32_t n,
                             const void *d_out, uint32_t d_out_type, uint64_t d_out_ld, uint32_t v,
                             uint32_t d, float scale, const void *add_to, void *d_table,
                             uint32_t d_table_type, uint64_t d_table_ld, void *ws, uint32_t *status,
                             hipStream_t stream);

hipError_t launch_layer_norm(const void *x, uint32_t dtype, uint32_t n, uint32_t d, uint64_t x_ld,
                             const void *weight, const void *bias, uint32_t weight_type, float eps,
                             void *out, uint64_t out_ld, float *mean, float *rstd,
                             hipStream_t stream);

struct NormGradPlan {
  uint32_t parts;  // row parts of the weight's and bias' sums (1: no join)
  size_t ws_bytes;
};
NormGradPlan plan_layer_norm_grad(uint32_t n, uint32_t d);
hipError_t launch_layer_norm_grad(const NormGradPlan &plan, const void *d_out, uint64_t d_out_ld,
                                  const void *x, uint32_t dtype, uint32_t n, uint32_t d,
                                  uint64_t x_ld, const float *mean, const float *rstd,
                                  const void *weight, uint32_t weight_type, void *d_x,
                                  uint64_t d_x_ld, void *d_weight, void *d_bias, void *ws,
                                  hipStream_t stream);

struct LogprobsPlan {
  uint32_t parts;  // parts of a row (1: no join)
  size_t off_keys;
  size_t ws_bytes;
};
LogprobsPlan plan_logprobs(uint32_t dtype, uint32_t n, uint32_t v, uint32_t top_k);
hipError_t launch_logprobs(const LogprobsPlan &plan, const void *logits, uint32_t dtype, uint32_t n,
                           uint32_t v, uint64_t ld, const int32_t *targets, uint32_t top_k, float *logp, float *entropy,
                           float *stats, int32_t *top_idx, float *top_logp, void *ws,
                           uint32_t *status, hipStream_t stream);
hipError_t launch_logprobs_grad(const void *logits, uint32_t dtype, uint32_t n, uint32_t v,
                                uint64_t ld, const int32_t *targets, const float *stats,
                                const float *entropy, const float *d_logp, const float *d_entropy,
                                void *d_logits, uint64_t d_logits_ld, uint32_t *status,
                                hipStream_t stream);

}  // namespace seacells
