// Gated feed-forward block and its gradient on gfx950.
//
//   pre = x W_in^T            W_in [2f, d]: f gate rows g, then f up rows u
//   h   = act(g) u            per element
//   y   = h W_out^T           W_out [m, f]
//
// and with dh = dy W_out:
//   d_pre = [dh u act'(g), dh act(g)],  dx = d_pre W_in,
//   dW_in = d_pre^T x,  dW_out = dy^T h.
//
// Each is a product on the matrix cores (mm.hpp) with the work on its results
// in the same kernel: a block multiplies gate and up columns of the same h
// side by side, so that h leaves it finished; the product that gives dh reads
// pre and leaves d_pre and h. h and d_pre are held in x's 16-bit type (f32:
// three bf16), one rounding of half a step beside the output's own; sums are
// f32.
#include <type_traits>

#include "few.hpp"
#include "mm.hpp"

namespace seacells {
namespace {

using namespace mm;

// Gate and up results to pre (where it is kept) and h. Columns behind f are
// products with zeros: h's row ends in zeros, as its own product needs.
template <class O, Act kAct>
struct PutGated {
  O *pre;  // or nullptr
  uint64_t pre_ld;
  uint16_t *h;
  uint64_t h_ld, plane;
  uint32_t f;
  template <bool kWhole>
  __device__ __forceinline__ void put(uint32_t row, uint32_t col, Row8 g, Row8 u) const {
    if (pre != nullptr) {
      O *const at = pre + row * pre_ld;
      put_row<kWhole>(at, col, f, g);
      put_row<kWhole>(at + f, col, f, u);
    }
    Row8 v;
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) v[e] = kWhole || col + e < f ? act<kAct>(g[e]) * u[e] : 0.0f;
    put_operand<O>(h + row * h_ld + col, plane, v);
  }
};

// dh to d_pre (its up half ld columns behind the gate's) and h.
template <class O, Act kAct>
struct PutPre {
  const O *pre;
  uint64_t pre_ld;
  uint16_t *d_pre, *h;
  uint64_t ld, d_plane, h_plane;  // ld: h's; d_pre's is twice that
  uint32_t f;
  template <bool kWhole>
  __device__ __forceinline__ void put(uint32_t row, uint32_t col, Row8 dh) const {
    const O *const at = pre + row * pre_ld;
    const bool whole = kWhole || col + 8 <= f;
    Row8 g, u;
    if (whole) {
      g = __builtin_convertvector(*reinterpret_cast<const Pack<O, 8> *>(at + col), Row8);
      u = __builtin_convertvector(*reinterpret_cast<const Pack<O, 8> *>(at + f + col), Row8);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        const uint32_t c = min(col + e, f - 1);
        g[e] = (float)at[c];
        u[e] = (float)at[f + c];
      }
    }
    Row8 dg, du, v;
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      float a, da;
      act_both<kAct>(g[e], &a, &da);
      const bool in = whole || col + e < f;
      dg[e] = in ? dh[e] * u[e] * da : 0.0f;
      du[e] = in ? dh[e] * a : 0.0f;
      v[e] = in ? a * u[e] : 0.0f;
    }
    uint16_t *const to = d_pre + row * 2 * ld + col;
    put_operand<O>(to, d_plane, dg);
    put_operand<O>(to + ld, d_plane, du);
    put_operand<O>(h + row * ld + col, h_plane, v);
  }
};

// Rows of [gate columns, up columns] of d_pre (`apart` each) to W_in's rows.
template <class O>
struct ToGatedRows {
  O *out;
  uint64_t ld;
  uint32_t n, f, apart;
  template <bool kWhole>
  __device__ __forceinline__ void put(uint32_t row, uint32_t col, Row8 v) const {
    const bool up = row >= apart;
    const uint32_t in = up ? row - apart : row;
    if (in < f) put_row<kWhole>(out + (uint64_t)(up ? f + in : in) * ld, col, n, v);
  }
};

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

struct FfnRoom {
  Matrix x, w_in, w_out;
  uint16_t *h;
  float *parts;
  Pack3 list = {};
  Shape in, out;
  size_t bytes;
};

FfnRoom lay_out(const FfnCall &c, bool x_stays, bool in_stays, bool out_stays, void *ws) {
  FfnRoom r;
  Room room{static_cast<char *>(ws)};
  r.x = operand(c.x, c.dtype, c.x_ld, c.n, c.d, x_stays, room, r.list);
  r.w_in = operand(c.w_in, c.dtype, c.w_in_ld, 2 * c.f, c.d, in_stays, room, r.list);
  r.w_out = operand(c.w_out, c.dtype, c.w_out_ld, c.m, c.f, out_stays, room, r.list);
  r.h = static_cast<uint16_t *>(room.take(matrix_bytes(c.dtype, c.n, c.f)));
  r.in = plan_shape(c.n, 2ull * c.f, tiles_of(c.dtype, 1, up8(c.d)));
  r.out = plan_shape(c.n, c.m, tiles_of(c.dtype, 1, up8(c.f)));
  const size_t a = parts_bytes(r.in, c.n, 2ull * up8(c.f)), b = parts_bytes(r.out, c.n, up8(c.m));
  r.parts = static_cast<float *>(room.take(a > b ? a : b));
  r.bytes = room.used;
  return r;
}

struct GradRoom {
  Matrix x, d_out, w_in, w_out;
  uint16_t *h, *d_pre;
  float *parts;
  Pack3 list = {};
  Shape dh, dx, d_in, d_out_w;
  size_t bytes;
};

GradRoom lay_out_grad(const FfnGradCall &c, const bool stays[4], void *ws) {
  GradRoom r;
  Room room{static_cast<char *>(ws)};
  const uint32_t f8 = up8(c.f), wide = up64(c.f);
  r.x = operand(c.x, c.dtype, c.x_ld, c.n, c.d, stays[0], room, r.list);
  r.d_out = operand(c.d_out, c.dtype, c.d_out_ld, c.n, c.m, stays[1], room, r.list);
  r.w_in = operand(c.w_in, c.dtype, c.w_in_ld, 2 * c.f, c.d, stays[2], room, r.list);
  r.w_out = operand(c.w_out, c.dtype, c.w_out_ld, c.m, c.f, stays[3], room, r.list);
  r.h = static_cast<uint16_t *>(room.take(matrix_bytes(c.dtype, c.n, c.f)));
  r.d_pre = static_cast<uint16_t *>(room.take(matrix_bytes(c.dtype, c.n, 2 * wide)));
  r.dh = plan_shape(c.n, c.f, tiles_of(c.dtype, 1, up8(c.m)));
  r.dx = plan_shape(c.n, c.d, tiles_of(c.dtype, 2, f8));
  r.d_in = plan_shape(2ull * wide, c.d, tiles_of(c.dtype, 1, c.n));
  r.d_out_w = plan_shape(c.m, c.f, tiles_of(c.dtype, 1, c.n));
  size_t most = parts_bytes(r.dh, c.n, f8);
  const size_t more[3] = {parts_bytes(r.dx, c.n, up8(c.d)), parts_bytes(r.d_in, 2ull * wide, up8(c.d)),
                          parts_bytes(r.d_out_w, c.m, f8)};
  for (size_t b : more) most = b > most ? b : most;
  r.parts = static_cast<float *>(room.take(most));
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

// Few rows: h alone.
static size_t few_bytes(const FfnCall &c) {
  return align_up((size_t)c.n * c.f * dtype_size(c.dtype), 256);
}

size_t ffn_workspace(const FfnCall &c, bool aligned) {
  if (c.n == 0) return 0;
  if (c.n <= kFewRows) return few_bytes(c);
  const bool s = aligned && c.dtype != 0u;
  return lay_out(c, s && c.d % 8 == 0, s && c.d % 8 == 0, s && c.f % 8 == 0, nullptr).bytes;
}

size_t ffn_need(const FfnCall &c) {
  if (c.n == 0) return 0;
  if (c.n <= kFewRows) return few_bytes(c);
  return lay_out(c, in_place(c.x, c.dtype, c.x_ld, c.d), in_place(c.w_in, c.dtype, c.w_in_ld, c.d, c.f),
                 in_place(c.w_out, c.dtype, c.w_out_ld, c.f), nullptr)
      .bytes;
}

hipError_t launch_ffn(const FfnCall &c, void *out, uint64_t out_ld, void *pre, uint64_t pre_ld,
                      void *ws, hipStream_t stream) {
  if (c.n == 0) return hipSuccess;
  if (c.n <= kFewRows) {
    const FewProduct in = {c.x, c.w_in, ws, pre, c.x_ld, c.w_in_ld, c.f, pre_ld, c.n, c.d, c.f, c.act};
    const hipError_t e = launch_few_product(in, true, c.dtype, stream);
    if (e != hipSuccess) return e;
    const FewProduct up = {ws, c.w_out, out, nullptr, c.f, c.w_out_ld, out_ld, 0, c.n, c.f, c.m, c.act};
    return launch_few_product(up, false, c.dtype, stream);
  }
  const FfnRoom r =
      lay_out(c, in_place(c.x, c.dtype, c.x_ld, c.d), in_place(c.w_in, c.dtype, c.w_in_ld, c.d, c.f),
              in_place(c.w_out, c.dtype, c.w_out_ld, c.f), ws);
  hipError_t e = launch_pack(r.list, c.dtype, stream);
  if (e != hipSuccess) return e;
  const uint32_t f8 = up8(c.f), d8 = up8(c.d), wide = up64(c.f);
  const uint64_t plane = (uint64_t)c.n * wide;
  const Matrix h = {r.h, wide, plane};
  return with_types(c.dtype, [&](auto o, auto t) {
    typedef decltype(o) O;
    typedef decltype(t) T;
    hipError_t rc = with_act(c.act, [&](auto a) {
      const Args g = make_args(c.dtype, r.x, r.w_in, c.n, c.f, d8, d8, 1, nullptr, nullptr, r.in,
                               2 * c.f);
      const PutGated<O, decltype(a)::value> put = {static_cast<O *>(pre), pre_ld, r.h, wide, plane, c.f};
      return launch_product<T, kAlongK, kAlongK, true>(g, r.in, put, r.parts, stream);
    });
    if (rc != hipSuccess) return rc;
    const Args g = make_args(c.dtype, h, r.w_out, c.n, c.m, f8, f8, 1, nullptr, nullptr, r.out, c.m);
    return launch_product<T, kAlongK, kAlongK, false>(
        g, r.out, ToRows<O>{static_cast<O *>(out), out_ld, c.m}, r.parts, stream);
  });
}

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
  const uint32_t f8 = up8(c.f), m8 = up8(c.m), wide = up64(c.f);
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
  const uint64_t h_plane = (uint64_t)c.n * wide, d_plane = 2 * h_plane;
  const Matrix h = {r.h, wide, h_plane}, d_pre = {r.d_pre, 2ull * wide, d_plane};
  return with_types(c.dtype, [&](auto o, auto t) {
    typedef decltype(o) O;
    typedef decltype(t) T;
    hipError_t rc = with_act(c.act, [&](auto a) {
      const Args g = make_args(c.dtype, r.d_out, r.w_out, c.n, c.f, m8, c.m, 1, nullptr, nullptr,
                               r.dh, c.f);
      const PutPre<O, decltype(a)::value> put = {static_cast<const O *>(c.pre), c.pre_ld, r.d_pre,
                                                 r.h,  wide, d_plane, h_plane, c.f};
      return launch_product<T, kAlongK, kAcrossK, false>(g, r.dh, put, r.parts, stream);
    });
    if (rc == hipSuccess && d_x != nullptr) {
      const uint64_t a_base[2] = {0, wide}, b_base[2] = {0, (uint64_t)c.f * r.w_in.ld};
      const Args g = make_args(c.dtype, d_pre, r.w_in, c.n, c.d, f8, c.f, 2, a_base, b_base, r.dx, c.d);
      rc = launch_product<T, kAlongK, kAcrossK, false>(
          g, r.dx, ToRows<O>{static_cast<O *>(d_x), d_x_ld, c.d}, r.parts, stream);
    }
    if (rc == hipSuccess && d_w_in != nullptr) {
      const Args g = make_args(c.dtype, d_pre, r.x, 2 * wide, c.d, c.n, c.n, 1, nullptr, nullptr, r.d_in,
                               c.d);
      rc = launch_product<T, kAcrossK, kAcrossK, false>(
          g, r.d_in, ToGatedRows<O>{static_cast<O *>(d_w_in), d_w_in_ld, c.d, c.f, wide}, r.parts,
          stream);
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
