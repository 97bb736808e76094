// Layer norm and its gradient, with the sums of the weight's and the bias'
// gradient.
//
//   h = (x - mean) rstd                    y = h weight + bias
//   g = d_y weight                         d_x = rstd (g - mean(g) - h mean(g h))
//   d_weight = sum over rows of d_y h      d_bias = sum over rows of d_y
//
// All are bound by memory: forward reads x and writes y, the gradient reads
// d_y and x and writes d_x.
#include "token.hpp"

namespace seacells {

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = kThreads / kWave;
constexpr uint32_t kMaxBlocks = 1u << 20;
constexpr uint32_t kMaxParts = 256;

// Sum over the block in a fixed order, the result in every thread.
__device__ __forceinline__ float block_sum(float x, float *lds) {
  x = wave_sum_f32(x);
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x / kWave] = x;
  __syncthreads();
  float s = 0.0f;
  for (uint32_t w = 0; w < kWaves; ++w) s += lds[w];
  return s;
}

template <class T, class W>
__global__ void __launch_bounds__(kThreads)
    layer_norm_kernel(const T *x, uint32_t n, uint32_t d, uint64_t x_ld,
                      const W *__restrict__ weight, const W *__restrict__ bias, float eps, T *out,
                      uint64_t out_ld, float *__restrict__ mean, float *__restrict__ rstd) {
  __shared__ float lds[kWaves];
  const float inv_d = 1.0f / (float)d;
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T *row = x + i * x_ld;
    float s = 0.0f;
    for (uint32_t c = threadIdx.x; c < d; c += kThreads) s += (float)row[c];
    float mu = block_sum(s, lds) * inv_d;
    // the second pass corrects the mean's own rounding
    float q = 0.0f, r = 0.0f;
    for (uint32_t c = threadIdx.x; c < d; c += kThreads) {
      const float t = (float)row[c] - mu;
      q += t * t;
      r += t;
    }
    const float shift = block_sum(r, lds) * inv_d;
    const float var = fmaxf(block_sum(q, lds) * inv_d - shift * shift, 0.0f);
    mu += shift;
    const float rs = 1.0f / sqrtf(var + eps);
    __syncthreads();  // every read of the row is done: out may be x
    for (uint32_t c = threadIdx.x; c < d; c += kThreads) {
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

template <class T, class W>
__global__ void __launch_bounds__(kThreads)
    layer_norm_dx_kernel(const T *d_out, uint64_t d_out_ld, const T *x, uint32_t n, uint32_t d,
                         uint64_t x_ld, const float *__restrict__ mean,
                         const float *__restrict__ rstd, const W *__restrict__ weight, T *d_x,
                         uint64_t d_x_ld) {
  __shared__ float lds[kWaves];
  const float inv_d = 1.0f / (float)d;
  for (uint64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const T *row = x + i * x_ld, *dy = d_out + i * d_out_ld;
    const float mu = mean[i], rs = rstd[i];
    float s = 0.0f, q = 0.0f;
    for (uint32_t c = threadIdx.x; c < d; c += kThreads) {
      const float w = weight != nullptr ? (float)weight[c] : 1.0f;
      const float g = (float)dy[c] * w, h = ((float)row[c] - mu) * rs;
      s += g;
      q += g * h;
    }
    const float a = block_sum(s, lds) * inv_d, b = block_sum(q, lds) * inv_d;
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < d; c += kThreads) {
      const float w = weight != nullptr ? (float)weight[c] : 1.0f;
      const float g = (float)dy[c] * w, h = ((float)row[c] - mu) * rs;
      d_x[i * d_x_ld + c] = (T)(rs * (g - a - h * b));
    }
  }
}

// Column sums over one part of the rows: part[p][0][c] = sum d_y h, [1][c] =
// sum d_y.
template <class T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_parts_kernel(const T *__restrict__ d_out, uint64_t d_out_ld,
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

template <class W>
__global__ void __launch_bounds__(kThreads)
    layer_norm_join_kernel(const float *__restrict__ part, uint32_t parts, uint32_t d,
                           W *__restrict__ d_weight, W *__restrict__ d_bias) {
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= d) return;
  float sw = 0.0f, sb = 0.0f;
  for (uint32_t p = 0; p < parts; ++p) {
    sw += part[((uint64_t)p * 2) * d + c];
    sb += part[((uint64_t)p * 2 + 1) * d + c];
  }
  if (d_weight != nullptr) d_weight[c] = (W)sw;
  if (d_bias != nullptr) d_bias[c] = (W)sb;
}

uint32_t row_blocks(uint32_t n) { return n < kMaxBlocks ? n : kMaxBlocks; }

}  // namespace

hipError_t launch_layer_norm(const void *x, uint32_t dtype, uint32_t n, uint32_t d, uint64_t x_ld,
                             const void *weight, const void *bias, uint32_t weight_type, float eps,
                             void *out, uint64_t out_ld, float *mean, float *rstd,
                             hipStream_t stream) {
  if (n == 0) return hipSuccess;
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto w) {
      using W = decltype(w);
      hipLaunchKernelGGL((layer_norm_kernel<T, W>), dim3(row_blocks(n)), dim3(kThreads), 0, stream,
                         static_cast<const T *>(x), n, d, x_ld, static_cast<const W *>(weight),
                         static_cast<const W *>(bias), eps, static_cast<T *>(out), out_ld, mean,
                         rstd);
      return hipGetLastError();
    };
    return weight_type == (uint32_t)Dtype::f32 ? go(float{}) : go(t);
  });
}

NormGradPlan plan_layer_norm_grad(uint32_t n, uint32_t d) {
  NormGradPlan p{};
  const uint32_t parts = div_up(n, 16);
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
  return with_type(dtype, [&](auto t) -> hipError_t {
    using T = decltype(t);
    auto go = [&](auto w) -> hipError_t {
      using W = decltype(w);
      const uint32_t cols = div_up(d, kThreads);
      hipError_t e = hipSuccess;
      if (sums && n > 0) {  // before d_x, which may overwrite d_out or x
        hipLaunchKernelGGL((layer_norm_parts_kernel<T>), dim3(cols, plan.parts), dim3(kThreads), 0,
                           stream, static_cast<const T *>(d_out), d_out_ld,
                           static_cast<const T *>(x), n, d, x_ld, mean, rstd,
                           div_up(n, plan.parts), part);
        if ((e = hipGetLastError()) != hipSuccess) return e;
      }
      if (sums) {
        hipLaunchKernelGGL((layer_norm_join_kernel<W>), dim3(cols), dim3(kThreads), 0, stream, part,
                           plan.parts, d, static_cast<W *>(d_weight), static_cast<W *>(d_bias));
        if ((e = hipGetLastError()) != hipSuccess) return e;
      }
      if (d_x != nullptr && n > 0) {
        hipLaunchKernelGGL((layer_norm_dx_kernel<T, W>), dim3(row_blocks(n)), dim3(kThreads), 0,
                           stream, static_cast<const T *>(d_out), d_out_ld,
                           static_cast<const T *>(x), n, d, x_ld, mean, rstd,
                           static_cast<const W *>(weight), static_cast<T *>(d_x), d_x_ld);
        e = hipGetLastError();
      }
      return e;
    };
    return weight_type == (uint32_t)Dtype::f32 ? go(float{}) : go(t);
  });
}

}  // namespace seacells
