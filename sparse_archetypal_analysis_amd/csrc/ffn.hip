// Gated feed-forward block on gfx950.
//
//   pre = x W_in^T            W_in [2f, d]: f gate rows g, then f up rows u
//   h   = act(g) u            per element
//   y   = h W_out^T           W_out [m, f]
//
// Two products on the matrix cores (mm.hpp), the work on the first one's results
// in the same kernel: a block multiplies gate and up columns of the same h side
// by side, so that h leaves it finished. h is held in x's 16-bit type (f32:
// three bf16), one rounding of half a step beside the output's own; sums are
// f32. Few rows: few.hip.
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
  typedef void Ahead;
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

struct FfnRoom {
  Matrix x, w_in, w_out;
  uint16_t *h;
  float *parts;
  PackList list = {};
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
  r.in = plan_shape(c.n, 2ull * c.f, tiles_of(c.dtype, 1, up8(c.d)), c.n > 512);
  r.out = plan_shape(c.n, c.m, tiles_of(c.dtype, 1, up8(c.f)));
  const size_t a = parts_bytes(r.in, c.n, 2ull * up8(c.f)), b = parts_bytes(r.out, c.n, up8(c.m));
  r.parts = static_cast<float *>(room.take(a > b ? a : b));
  r.bytes = room.used;
  return r;
}

}  // namespace

static bool few(const FfnCall &c) {
  return few_rows(c.dtype, c.n, (2ull * c.d + c.m) * c.f, true);
}

// Few rows: h alone.
static size_t few_bytes(const FfnCall &c) {
  return align_up((size_t)c.n * c.f * dtype_size(c.dtype), 256);
}

size_t ffn_workspace(const FfnCall &c, bool aligned) {
  if (c.n == 0) return 0;
  if (few(c)) return few_bytes(c);
  const bool s = aligned && c.dtype != 0u;
  return lay_out(c, s && c.d % 8 == 0, s && c.d % 8 == 0, s && c.f % 8 == 0, nullptr).bytes;
}

size_t ffn_need(const FfnCall &c) {
  if (c.n == 0) return 0;
  if (few(c)) return few_bytes(c);
  return lay_out(c, in_place(c.x, c.dtype, c.x_ld, c.d), in_place(c.w_in, c.dtype, c.w_in_ld, c.d, c.f),
                 in_place(c.w_out, c.dtype, c.w_out_ld, c.f), nullptr)
      .bytes;
}

hipError_t launch_ffn(const FfnCall &c, void *out, uint64_t out_ld, void *pre, uint64_t pre_ld,
                      void *ws, hipStream_t stream) {
  if (c.n == 0) return hipSuccess;
  if (few(c)) {
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
  const uint32_t f8 = up8(c.f), d8 = up8(c.d), wide = apart64(c.f);
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

}  // namespace seacells
