// Gradient of the gated feed-forward block (ffn.hip) on gfx950. With g, u the
// halves of pre and dh = dy W_out:
//   d_pre = [dh u act'(g), dh act(g)],  dx = d_pre W_in,
//   dW_in = d_pre^T x,  dW_out = dy^T h,  h = act(g) u.
// Four products on the matrix cores (mm.hpp); the one that gives dh reads pre
// and leaves d_pre and h (ffn_d_pre.hip), in x's 16-bit type (f32: three bf16),
// one rounding of half a step beside the output's own; sums are f32. f16 holds
// numbers from 2^-14 in full: d_pre of a mean over rows is below that, and is
// held times a power of two.
#include "ffn_grad.hpp"

namespace seacells {
namespace {

using namespace mm;

// Rows of [gate columns, up columns] of d_pre (`apart` each) to W_in's rows.
template <class O>
struct ToGatedRows {
  typedef void Ahead;
  O *out;
  uint64_t ld;
  uint32_t n, f, apart;
  const Scale *scale;  // or nullptr
  template <bool kWhole>
  __device__ __forceinline__ void put(uint32_t row, uint32_t col, Row8 v) const {
    if (scale != nullptr) v *= scale->back;
    const bool up = row >= apart;
    const uint32_t in = up ? row - apart : row;
    if (in < f) put_row<kWhole>(out + (uint64_t)(up ? f + in : in) * ld, col, n, v);
  }
};

// The power of two for f16's d_pre takes the largest |d_out| to between 1 and 2,
// and is 1 for larger ones: no number is made smaller. One that would get past
// f16 by it is seen by the product that makes it, which is then done again
// without (a launch that ends at once where there is none). One block up to
// kOneBlock elements, more blocks in two launches (gradient of 64 x 128, us in one
// and two: 512 rows 33.7 and 34.2). All of it costs 64 x 128 6 us at 4 rows and 7
// at 1024, 8192 rows of 256 x 1000 8.5 of 95, 16384 of 2048 x 8192 30 of 2795.
constexpr uint32_t kLargest = 1024, kLargestBlocks = 512, kOneBlock = 1u << 15;

__device__ __forceinline__ void put_scale(float most, Scale *scale) {
  const int e = most > 0.0f ? min((int)(__float_as_uint(most) >> 23) - 127, 0) : 0;
  scale->by = __uint_as_float((uint32_t)(127 - e) << 23);
  scale->back = __uint_as_float((uint32_t)(127 + e) << 23);
  scale->past = 0u;
}

__device__ __forceinline__ float block_most(float most) {
  __shared__ float wave_most[kLargest / kWave];
  most = group_max<kWave>(most);
  if (lane_id() == 0) wave_most[threadIdx.x / kWave] = most;
  __syncthreads();
  for (uint32_t w = 0; w < kLargest / kWave; ++w) most = fmaxf(most, wave_most[w]);
  return most;
}

// The largest finite size of n rows of m, 8 elements a thread at once.
__global__ __launch_bounds__(kLargest) void largest(const _Float16 *__restrict__ from, uint64_t ld,
                                                    uint32_t n, uint32_t m,
                                                    float *__restrict__ parts, Scale *scale) {
  const uint32_t row_chunks = (m + 7) / 8;
  const uint64_t chunks = (uint64_t)n * row_chunks;
  float most = 0.0f;
#pragma unroll 4
  for (uint64_t id = (uint64_t)blockIdx.x * kLargest + threadIdx.x; id < chunks;
       id += (uint64_t)gridDim.x * kLargest) {
    const uint64_t row = id / row_chunks;
    const uint32_t col = (uint32_t)(id - row * row_chunks) * 8;
    const Vec<_Float16> v = load_vec_tail(from + row * ld, col, m, (_Float16)0.0f);
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      const float x = fabsf((float)v[e]);
      most = x <= 65504.0f ? fmaxf(most, x) : most;
    }
  }
  most = block_most(most);
  if (threadIdx.x != 0) return;
  if (gridDim.x > 1) parts[blockIdx.x] = most;
  else put_scale(most, scale);
}

__global__ __launch_bounds__(kLargest) void join_largest(const float *__restrict__ parts, uint32_t count,
                                                         Scale *scale) {
  const float most = block_most(threadIdx.x < count ? parts[threadIdx.x] : 0.0f);
  if (threadIdx.x == 0) put_scale(most, scale);
}
static_assert(kLargestBlocks <= kLargest, "one part a thread");

hipError_t launch_largest(const FfnGradCall &c, float *parts, Scale *scale, hipStream_t stream) {
  const uint64_t chunks = (uint64_t)c.n * ((c.m + 7) / 8);
  const uint32_t blocks =
      chunks <= kOneBlock / 8 ? 1 : (uint32_t)min((chunks + kLargest - 1) / kLargest, (uint64_t)kLargestBlocks);
  largest<<<blocks, kLargest, 0, stream>>>(static_cast<const _Float16 *>(c.d_out), c.d_out_ld, c.n, c.m,
                                           parts, scale);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || blocks == 1) return e;
  join_largest<<<1, kLargest, 0, stream>>>(parts, blocks, scale);
  return hipGetLastError();
}

struct GradRoom {
  Matrix x, d_out, w_in, w_out;
  uint16_t *h, *d_pre;
  float *parts, *most;
  Scale *scale;  // (f16)
  PackList list = {};
  Shape dh, dx, d_in, d_out_w;
  size_t bytes;
};

GradRoom lay_out_grad(const FfnGradCall &c, const bool stays[4], void *ws) {
  GradRoom r;
  Room room{static_cast<char *>(ws)};
  const uint32_t f8 = up8(c.f), half = up64(c.f);
  r.x = operand(c.x, c.dtype, c.x_ld, c.n, c.d, stays[0], room, r.list);
  r.d_out = operand(c.d_out, c.dtype, c.d_out_ld, c.n, c.m, stays[1], room, r.list);
  r.w_in = operand(c.w_in, c.dtype, c.w_in_ld, 2 * c.f, c.d, stays[2], room, r.list);
  r.w_out = operand(c.w_out, c.dtype, c.w_out_ld, c.m, c.f, stays[3], room, r.list);
  r.h = static_cast<uint16_t *>(room.take(matrix_bytes(c.dtype, c.n, c.f)));
  r.d_pre = static_cast<uint16_t *>(room.take(matrix_bytes(c.dtype, c.n, 2 * half)));
  r.dh = plan_shape(c.n, c.f, tiles_of(c.dtype, 1, up8(c.m)), c.n > 512);
  r.dx = plan_shape(c.n, c.d, tiles_of(c.dtype, 2, f8));
  r.d_in = plan_shape(2ull * half, c.d, tiles_of(c.dtype, 1, c.n));
  r.d_out_w = plan_shape(c.m, c.f, tiles_of(c.dtype, 1, c.n));
  size_t most = parts_bytes(r.dh, c.n, f8);
  const size_t more[3] = {parts_bytes(r.dx, c.n, up8(c.d)), parts_bytes(r.d_in, 2ull * half, up8(c.d)),
                          parts_bytes(r.d_out_w, c.m, f8)};
  for (size_t b : more) most = b > most ? b : most;
  r.parts = static_cast<float *>(room.take(most));
  r.scale = is_f16(c.dtype) ? static_cast<Scale *>(room.take(sizeof(Scale))) : nullptr;
  r.most = is_f16(c.dtype) ? static_cast<float *>(room.take(kLargestBlocks * 4)) : nullptr;
  r.bytes = room.used;
  return r;
}

// A matrix of zero rows by d: what a weight's gradient is without rows.
template <class O>
__global__ __launch_bounds__(kThreads) void zero_rows(O *out, uint64_t ld, uint64_t rows, uint32_t d) {
  for (uint64_t id = (uint64_t)blockIdx.x * kThreads + threadIdx.x; id < rows * d;
       id += (uint64_t)gridDim.x * kThreads) {
    const uint64_t row = id / d;
    out[row * ld + (id - row * d)] = (O)0.0f;
  }
}

}  // namespace

size_t ffn_grad_workspace(const FfnGradCall &c, bool aligned) {
  if (c.n == 0) return 0;
  const bool s = aligned && c.dtype != 0u;
  const bool stays[4] = {s && c.d % 8 == 0, s && c.m % 8 == 0, s && c.d % 8 == 0, s && c.f % 8 == 0};
  return lay_out_grad(c, stays, nullptr).bytes;
}

static void stay(const FfnGradCall &c, bool stays[4]) {
  stays[0] = in_place(c.x, c.dtype, c.x_ld, c.d);
  stays[1] = in_place(c.d_out, c.dtype, c.d_out_ld, c.m);
  stays[2] = in_place(c.w_in, c.dtype, c.w_in_ld, c.d, c.f);
  stays[3] = in_place(c.w_out, c.dtype, c.w_out_ld, c.f);
}

size_t ffn_grad_need(const FfnGradCall &c) {
  if (c.n == 0) return 0;
  bool stays[4];
  stay(c, stays);
  return lay_out_grad(c, stays, nullptr).bytes;
}

hipError_t launch_ffn_grad(const FfnGradCall &c, void *d_x, uint64_t d_x_ld, void *d_w_in,
                           uint64_t d_w_in_ld, void *d_w_out, uint64_t d_w_out_ld, void *ws,
                           hipStream_t stream) {
  const uint32_t f8 = up8(c.f), m8 = up8(c.m), half = up64(c.f);
  const uint32_t h_ld = apart64(c.f), d_ld = apart64(2 * half);
  if (c.n == 0)
    return with_type(c.dtype, [&](auto o) {
      typedef decltype(o) O;
      if (d_w_in != nullptr)
        zero_rows<O><<<1024, kThreads, 0, stream>>>(static_cast<O *>(d_w_in), d_w_in_ld, 2ull * c.f, c.d);
      if (d_w_out != nullptr)
        zero_rows<O><<<1024, kThreads, 0, stream>>>(static_cast<O *>(d_w_out), d_w_out_ld, c.m, c.f);
      return hipGetLastError();
    });
  bool stays[4];
  stay(c, stays);
  const GradRoom r = lay_out_grad(c, stays, ws);
  hipError_t e = launch_pack(r.list, c.dtype, stream);
  if (e != hipSuccess) return e;
  Scale *const scale = d_x != nullptr || d_w_in != nullptr ? r.scale : nullptr;  // (d_pre's readers)
  if (scale != nullptr && (e = launch_largest(c, r.most, scale, stream)) != hipSuccess) return e;
  const uint64_t h_plane = (uint64_t)c.n * h_ld, d_plane = (uint64_t)c.n * d_ld;
  const Matrix h = {r.h, h_ld, h_plane}, d_pre = {r.d_pre, d_ld, d_plane};
  const DPre d = {c.dtype, c.act, make_args(c.dtype, r.d_out, r.w_out, c.n, c.f, m8, c.m, 1, nullptr, nullptr,
                                            r.dh, c.f),
                  r.dh, c.pre, c.pre_ld, r.d_pre, r.h, d_ld, h_ld, d_plane, h_plane, c.f, half, r.parts,
                  scale};
  if ((e = launch_d_pre(d, stream)) != hipSuccess) return e;
  return with_types(c.dtype, [&](auto o, auto t) {
    typedef decltype(o) O;
    typedef decltype(t) T;
    hipError_t rc = hipSuccess;
    if (rc == hipSuccess && d_x != nullptr) {
      const uint64_t a_base[2] = {0, half}, b_base[2] = {0, (uint64_t)c.f * r.w_in.ld};
      const Args g = make_args(c.dtype, d_pre, r.w_in, c.n, c.d, f8, c.f, 2, a_base, b_base, r.dx, c.d);
      rc = launch_product<T, kAlongK, kAcrossK, false>(
          g, r.dx, ToScaledRows<O>{static_cast<O *>(d_x), d_x_ld, c.d, scale}, r.parts, stream);
    }
    if (rc == hipSuccess && d_w_in != nullptr) {
      const Args g = make_args(c.dtype, d_pre, r.x, 2 * half, c.d, c.n, c.n, 1, nullptr, nullptr, r.d_in,
                               c.d);
      rc = launch_product<T, kAcrossK, kAcrossK, false>(
          g, r.d_in, ToGatedRows<O>{static_cast<O *>(d_w_in), d_w_in_ld, c.d, c.f, half, scale},
          r.parts, stream);
    }
    if (rc == hipSuccess && d_w_out != nullptr) {
      const Args g = make_args(c.dtype, r.d_out, h, c.m, c.f, c.n, c.n, 1, nullptr, nullptr, r.d_out_w,
                               c.f);
      rc = launch_product<T, kAcrossK, kAcrossK, false>(
          g, r.d_out_w, ToRows<O>{static_cast<O *>(d_w_out), d_w_out_ld, c.f}, r.parts, stream);
    }
    return rc;
  });
}

}  // namespace seacells
