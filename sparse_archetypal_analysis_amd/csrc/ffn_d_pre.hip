// Gradient of the gated block (ffn_grad.hip), first step, on gfx950: with g, u
// the halves of pre and dh = dy W_out, a product on the matrix cores (mm.hpp),
//   d_pre = [dh u act'(g), dh act(g)],  h = act(g) u
// in the product's own kernel.
#include <type_traits>

#include "few.hpp"
#include "ffn_grad.hpp"

namespace seacells {
namespace {

using namespace mm;

// dh to d_pre (its up columns `half` behind the gate's) and h.
template <class O, Act kAct>
struct PutPre {
  const O *pre;
  uint64_t pre_ld;
  uint16_t *d_pre, *h;
  uint64_t d_ld, h_ld, d_plane, h_plane;
  uint32_t f, half;
  Scale *scale;  // f16, or nullptr
  static constexpr bool kScaled = std::is_same<O, _Float16>::value;
  static constexpr float kEnd = 65520.0f;  // what f16 rounds to infinity
  struct Ahead {
    Pack<O, 8> g, u;
    float by;  // the scale's
  };
  template <bool kWhole>
  __device__ __forceinline__ Ahead ahead(uint32_t row, uint32_t col) const {
    const O *const at = pre + row * pre_ld;
    Ahead p;
    p.by = kScaled && scale != nullptr ? scale->by : 1.0f;
    if (kWhole || col + 8 <= f) {
      // (read once: lines that the L2 gives up first leave it to the product's
      // operands, 16384 x 8192 x 2048 bf16 746 -> 713 us; f32's 81 -> 88)
      const Pack<O, 8> *const g = reinterpret_cast<const Pack<O, 8> *>(at + col);
      const Pack<O, 8> *const u = reinterpret_cast<const Pack<O, 8> *>(at + f + col);
      p.g = sizeof(O) == 2 ? __builtin_nontemporal_load(g) : *g;
      p.u = sizeof(O) == 2 ? __builtin_nontemporal_load(u) : *u;
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        const uint32_t c = min(col + e, f - 1);
        p.g[e] = at[c];
        p.u[e] = at[f + c];
      }
    }
    return p;
  }

  template <bool kWhole>
  __device__ __forceinline__ void put(uint32_t row, uint32_t col, Row8 dh, const Ahead &p) const {
    const bool whole = kWhole || col + 8 <= f;
    const Row8 g = __builtin_convertvector(p.g, Row8), u = __builtin_convertvector(p.u, Row8);
    Row8 dg, du, v;
    if (kScaled) dh *= p.by;
#pragma unroll
    for (uint32_t e = 0; e < 8; ++e) {
      float a, da;
      act_both<kAct>(g[e], &a, &da);
      const bool in = whole || col + e < f;
      dg[e] = in ? dh[e] * u[e] * da : 0.0f;
      du[e] = in ? dh[e] * a : 0.0f;
      v[e] = in ? a * u[e] : 0.0f;
    }
    if (kScaled && scale != nullptr) {
      float most = 0.0f;  // (NaN loses)
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) most = fmaxf(most, fmaxf(fabsf(dg[e]), fabsf(du[e])));
      if (most >= kEnd) {
        const float end = kEnd * p.by;
        bool past = false;
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e)
          past = past || (fabsf(dg[e]) >= kEnd && fabsf(dg[e]) < end) ||
                 (fabsf(du[e]) >= kEnd && fabsf(du[e]) < end);
        if (past) {  // (every thread that does writes the same)
          scale->back = 1.0f;
          scale->past = 1u;
        }
      }
    }
    uint16_t *const to = d_pre + row * d_ld + col;
    put_operand<O>(to, d_plane, dg);
    put_operand<O>(to + half, d_plane, du);
    put_operand<O>(h + row * h_ld + col, h_plane, v);
  }
};

}  // namespace

hipError_t launch_d_pre(const DPre &d, hipStream_t stream) {
  return with_types(d.dtype, [&](auto o, auto t) {
    typedef decltype(o) O;
    typedef decltype(t) T;
    return with_act(d.act, [&](auto a) {
      PutPre<O, decltype(a)::value> put = {static_cast<const O *>(d.pre), d.pre_ld, d.d_pre, d.h, d.d_ld,
                                           d.h_ld, d.d_plane, d.h_plane, d.f, d.half, d.scale};
      hipError_t e = launch_product<T, kAlongK, kAcrossK, false>(d.product, d.shape, put, d.parts, stream);
      if (e != hipSuccess || d.scale == nullptr) return e;
      Args again = d.product;
      again.only = &d.scale->past;
      put.scale = nullptr;
      return launch_product<T, kAlongK, kAcrossK, false>(again, d.shape, put, d.parts, stream);
    });
  });
}

}  // namespace seacells
