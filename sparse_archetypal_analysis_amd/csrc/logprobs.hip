// Log probabilities of given classes, entropy and top alternatives of rows of
// logits, and their gradient.
//
//   m = max x, s = log sum exp(x - m)
//   log p_c = x_c - m - s      entropy H = s - sum p_c (x_c - m)
//   d_x = d_logp (1[c = target] - p_c) - d_entropy p_c (log p_c + H)
//
// -inf logits are masked: their p is an exact 0 and the product with their
// logarithm is taken as 0. NaN and +inf leave a row without a distribution.
// Both directions are bound by memory.
#include "token.hpp"

namespace seacells {

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = kThreads / kWave;
constexpr uint32_t kMaxBlocks = 1u << 20;
constexpr float kNegInf = -__builtin_huge_valf();
// exp of anything below is 0 in f32 (log of the least denormal: -103.3);
// products with a probability of 0 stay finite
constexpr float kFloor = -200.0f;

__device__ __forceinline__ uint64_t u64max(uint64_t x, uint64_t y) { return x > y ? x : y; }

// Descending (value, lowest column first) as one ascending number; 0 for
// masked entries (-inf orders to the least key of all values).
__device__ __forceinline__ uint64_t top_key(float x, uint32_t c) {
  return x > kNegInf ? ((uint64_t)f32_order(x) << 32) | (0xffffffffu - c) : 0ull;
}

__device__ __forceinline__ float block_max(float x, float *lds) {
  for (int off = 32; off >= 1; off >>= 1) x = nan_max(x, __shfl_xor(x, off, kWave));
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x / kWave] = x;
  __syncthreads();
  float m = lds[0];
  for (uint32_t w = 1; w < kWaves; ++w) m = nan_max(m, lds[w]);
  return m;
}

__device__ __forceinline__ float block_sum(float x, float *lds) {
  x = wave_sum_f32(x);
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x / kWave] = x;
  __syncthreads();
  float s = 0.0f;
  for (uint32_t w = 0; w < kWaves; ++w) s += lds[w];
  return s;
}

__device__ __forceinline__ uint64_t block_max_u64(uint64_t x, uint64_t *lds) {
  for (int off = 32; off >= 1; off >>= 1)
    x = u64max(x, (uint64_t)__shfl_xor((unsigned long long)x, off, kWave));
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x / kWave] = x;
  __syncthreads();
  uint64_t m = 0;
  for (uint32_t w = 0; w < kWaves; ++w) m = u64max(m, lds[w]);
  return m;
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    logprobs_kernel(const T *__restrict__ logits, uint32_t n, uint32_t v, uint64_t ld,
                    const int32_t *__restrict__ targets, uint32_t top_k, float *__restrict__ logp,
                    float *__restrict__ entropy, float *__restrict__ stats,
                    int32_t *__restrict__ top_idx, float *__restrict__ top_logp,
                    uint32_t *__restrict__ status) {
  __shared__ float lds[kWaves];
  __shared__ uint64_t lds64[kWaves];
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T *row = logits + i * ld;
    float m = kNegInf;
    for (uint32_t c = threadIdx.x; c < v; c += kThreads) m = nan_max(m, (float)row[c]);
    m = block_max(m, lds);
    float s = 0.0f, u = 0.0f;
    for (uint32_t c = threadIdx.x; c < v; c += kThreads) {
      const float t = nan_max((float)row[c] - m, kFloor);
      const float e = exp_neg(t);
      s += e;
      u += t * e;
    }
    s = block_sum(s, lds);
    u = block_sum(u, lds);
    const bool empty = m == kNegInf;
    const bool none = !(m <= 3.4028235e38f);  // NaN or +inf
    const float nan = __builtin_nanf("");
    const float ls = none ? nan : empty ? 0.0f : logf(s);
    if (threadIdx.x == 0) {
      if (stats != nullptr) {
        stats[2 * i] = none ? nan : m;
        stats[2 * i + 1] = ls;
      }
      if (entropy != nullptr) entropy[i] = none ? nan : empty ? 0.0f : ls - u / s;
      if (targets != nullptr) {
        const int32_t t = targets[i];
        const bool bad = t >= 0 && (uint32_t)t >= v;
        if (bad) atomicOr(status, kFlagBadIndex);
        if (logp != nullptr)
          logp[i] = t < 0 || bad ? 0.0f : none ? nan : empty ? kNegInf : ((float)row[t] - m) - ls;
      }
    }
    uint64_t last = ~0ull;
    for (uint32_t k = 0; k < top_k; ++k) {
      uint64_t best = 0;
      for (uint32_t c = threadIdx.x; c < v; c += kThreads) {
        const uint64_t key = none ? 0ull : top_key((float)row[c], c);
        if (key < last) best = u64max(best, key);
      }
      last = block_max_u64(best, lds64);
      if (threadIdx.x == 0) {
        top_idx[i * top_k + k] = last != 0 ? (int32_t)(0xffffffffu - (uint32_t)last) : -1;
        top_logp[i * top_k + k] =
            none ? nan : last != 0 ? (f32_unorder((uint32_t)(last >> 32)) - m) - ls : kNegInf;
      }
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    logprobs_grad_kernel(const T *logits, uint32_t n, uint32_t v, uint64_t ld,
                         const int32_t *__restrict__ targets, const float *__restrict__ stats,
                         const float *__restrict__ entropy, const float *__restrict__ d_logp,
                         const float *__restrict__ d_entropy, T *d_logits, uint64_t d_ld,
                         uint32_t *__restrict__ status) {
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T *row = logits + i * ld;
    T *to = d_logits + i * d_ld;
    const int32_t t = targets != nullptr ? targets[i] : -1;
    const bool bad = t >= 0 && (uint32_t)t >= v;
    if (bad && threadIdx.x == 0) atomicOr(status, kFlagBadIndex);
    const bool has = t >= 0 && !bad;
    const float g = has && d_logp != nullptr ? d_logp[i] : 0.0f;
    const float h = d_entropy != nullptr ? d_entropy[i] : 0.0f;
    const float H = d_entropy != nullptr ? entropy[i] : 0.0f;
    float m = stats[2 * i];
    const float ls = stats[2 * i + 1];
    if (m == kNegInf) m = 0.0f;  // nothing left: every entry is masked
    for (uint32_t c = threadIdx.x; c < v; c += kThreads) {
      const float x = (float)row[c];
      const float lp = nan_max(x - m - ls, kFloor);
      float y = -exp_neg(lp) * (g + h * (lp + H));
      if (has && c == (uint32_t)t && x > kNegInf) y += g;
      to[c] = (T)y;
    }
  }
}

uint32_t row_blocks(uint32_t n) { return n < kMaxBlocks ? n : kMaxBlocks; }

}  // namespace

size_t logprobs_workspace(uint32_t n, uint32_t v, uint32_t top_k) {
  (void)n;
  (void)v;
  (void)top_k;
  return 0;
}

hipError_t launch_logprobs(const void *logits, uint32_t dtype, uint32_t n, uint32_t v, uint64_t ld,
                           const int32_t *targets, uint32_t top_k, float *logp, float *entropy,
                           float *stats, int32_t *top_idx, float *top_logp, void *ws,
                           uint32_t *status, hipStream_t stream) {
  (void)ws;
  hipError_t e = launch_status_clear(status, stream);
  if (e != hipSuccess || n == 0) return e;
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((logprobs_kernel<T>), dim3(row_blocks(n)), dim3(kThreads), 0, stream,
                       static_cast<const T *>(logits), n, v, ld, targets, top_k, logp, entropy,
                       stats, top_idx, top_logp, status);
    return hipGetLastError();
  });
}

hipError_t launch_logprobs_grad(const void *logits, uint32_t dtype, uint32_t n, uint32_t v,
                                uint64_t ld, const int32_t *targets, const float *stats,
                                const float *entropy, const float *d_logp, const float *d_entropy,
                                void *d_logits, uint64_t d_logits_ld, uint32_t *status,
                                hipStream_t stream) {
  hipError_t e = launch_status_clear(status, stream);
  if (e != hipSuccess || n == 0) return e;
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((logprobs_grad_kernel<T>), dim3(row_blocks(n)), dim3(kThreads), 0, stream,
                       static_cast<const T *>(logits), n, v, ld, targets, stats, entropy, d_logp,
                       d_entropy, static_cast<T *>(d_logits), d_logits_ld, status);
    return hipGetLastError();
  });
}

}  // namespace seacells
