// What the kernels for many and for few rows of the model's block and head
// share: activations and the figures of a row of log probabilities; and the
// internal interface of those for few rows. Nothing here is exported.
#pragma once

#include <type_traits>

#include "token.hpp"

namespace seacells {

constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// --- activations ---------------------------------------------------------------

// 1 / (1 + e^-g): 0 and 1 at the ends, where e^-g is infinite or 0.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -kLog2E));
}

// The normal distribution's integral and density (times sqrt(2 pi)) at g:
// erfc(x) = (a1 t + ... + a5 t^5) e^(-x^2), t = 1 / (1 + p x), to 1.5e-7
// (Abramowitz and Stegun, 7.1.26), mirrored for g > 0. (act(g) in f32 is off by
// up to 2.1e-7, about twice what an erf rounded to f32 gives.)
__device__ __forceinline__ float normal(float g, float *density) {
  const float x = fabsf(g) * 0.70710678118654752440f;
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * x);
  const float e = exp_neg(-x * x);
  const float q = ((((1.061405429f * t - 1.453152027f) * t + 1.421413741f) * t - 0.284496736f) * t +
                   0.254829592f) * t * (0.5f * e);
  *density = e;
  return g >= 0.0f ? 1.0f - q : q;
}

// act(g) and act'(g). NaN stays NaN.
template <Act kAct>
__device__ __forceinline__ float act(float g) {
  if (kAct == Act::silu) return g * sigmoid(g);
  float e;
  if (kAct == Act::gelu) return g * normal(g, &e);
  return g <= 0.0f ? 0.0f : g;
}

template <Act kAct>
__device__ __forceinline__ void act_both(float g, float *a, float *da) {
  if (kAct == Act::silu) {
    const float s = sigmoid(g);
    *a = g * s;
    *da = s + *a * (1.0f - s);
  } else if (kAct == Act::gelu) {
    float e;
    const float p = normal(g, &e);
    *a = g * p;
    *da = p + g * 0.39894228040143267794f * e;
  } else {
    *a = act<Act::relu>(g);
    *da = g > 0.0f ? 1.0f : (g <= 0.0f ? 0.0f : g);
  }
}

// Calls f with the activation as a constant.
template <class F>
hipError_t with_act(Act a, F &&f) {
  switch (a) {
    case Act::silu:
      return f(std::integral_constant<Act, Act::silu>{});
    case Act::gelu:
      return f(std::integral_constant<Act, Act::gelu>{});
    default:
      return f(std::integral_constant<Act, Act::relu>{});
  }
}

// --- figures of a row of log probabilities ------------------------------------

// e^-200 (and 2^-200) is 0: a difference below that, -inf among them, is as good as that
// one, and finite. (NaN becomes that too; a row's maximum tells of NaN.)
__device__ __forceinline__ float not_below(float t) { return fmaxf(t, -200.0f); }

// What a row's figures are made of: maximum, sum e^(z - m), sum (z - m) e^(z - m).
struct Sums {
  float m, s, u;
};

// The same for the maximum m (not below own.m); nothing: (-inf, 0, 0). Classes
// of a bias at f32's low end are 1e38 below others: t s would be infinite, and e 0.
__device__ __forceinline__ void rescale(Sums &a, float m) {
  const bool none = a.m == -kInf;
  const float t = none ? 0.0f : not_below(a.m - m);
  const float e = none ? 0.0f : exp_neg(t);
  a.u = none ? 0.0f : e * (a.u + t * a.s);
  a.s *= e;
  a.m = m;
}

__device__ __forceinline__ Sums joined(Sums a, Sums b) {
  const float m = nan_max(a.m, b.m);
  rescale(a, m);
  rescale(b, m);
  return Sums{m, a.s + b.s, a.u + b.u};
}

// --- few rows ------------------------------------------------------------------

// Whether n rows against weights of `elements` elements in all go to these
// kernels (at most 64 rows). They read 16 rows of x with 16 of weights, so more
// rows cost as much as the weights; tiles cost some launches, and f32 a copy of
// the weights. Weights from memory, us here and by tiles: block of 4096 x 8192
// bf16 16 rows 54 and 66, 32 rows 65 and 67; 2048 x 16384 32 rows 87 and 67;
// 1024 x 4096 32 rows 20 and 25, 64 rows 30 and 26; f32 64 rows 57 and 70, 206
// and 445. Log probabilities of 512 x 50001 bf16 16 rows 22 and 20, 32 rows 30
// and 20; 100 x 1300 64 rows 12 and 14; f32 64 rows 81 and 96, 14 and 19. f32
// with few results and a long k, which one block walks alone, loses by the rule:
// 512 x 16384 64 rows 179, by tiles 65 rows 104.
inline bool few_rows(uint32_t dtype, uint32_t n, uint64_t elements, bool block) {
  if (n <= 16 || (n <= 64 && dtype == 0u)) return true;
  return block ? n <= 32 && elements <= (1u << 24) : n <= 64 && elements <= (1u << 18);
}

// out[n, rows] = x[n, k] w[rows, k]^T, or gated: w has 2 rows, pre [n, 2 rows]
// (or nullptr) and out = act(gate) * up.
struct FewProduct {
  const void *x, *w;
  void *out, *pre;
  uint64_t x_ld, w_ld, out_ld, pre_ld;
  uint32_t n, k, rows;
  Act act;
};
hipError_t launch_few_product(const FewProduct &g, bool gated, uint32_t dtype, hipStream_t stream);

// Sums of x[n, d] table[v, d]^T + bias per row: few_slices(v) slices of [3][n],
// and the targets' z.
struct FewSums {
  const void *x, *table;
  const float *bias;
  const int32_t *targets;
  float *sums, *at_target;
  uint64_t x_ld, table_ld;
  uint32_t n, d, v;
};
uint32_t few_slices(uint32_t v);
hipError_t launch_few_sums(const FewSums &g, uint32_t dtype, hipStream_t stream);

}  // namespace seacells
