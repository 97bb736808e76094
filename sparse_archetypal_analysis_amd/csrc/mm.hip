// Operands of the matrix products in a form that they can be multiplied in,
// and how a product is spread over the card.
#include "mm.hpp"

namespace seacells {
namespace mm {
namespace {

// 8 elements a thread: rows of any stride and alignment to rows on 16 bytes
// with zeros behind them (f32: to planes). Bound by memory.
template <class O>
__global__ __launch_bounds__(kThreads) void pack_rows(PackList list) {
  const PackItem &it = list.item[blockIdx.y];
  for (uint64_t id = (uint64_t)blockIdx.x * kThreads + threadIdx.x; id < it.chunks;
       id += (uint64_t)gridDim.x * kThreads) {
    const uint64_t row = id / it.row_chunks;
    const uint32_t col = (uint32_t)(id - row * it.row_chunks) * 8;
    const O *const from = static_cast<const O *>(it.from) + row * it.from_ld;
    Row8 v;
    if (col + 8 <= it.len) {
      v = __builtin_convertvector(*reinterpret_cast<const Pack<O, 8> *>(from + col), Row8);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        const O x = from[min(col + e, it.len - 1)];
        v[e] = col + e < it.len ? (float)x : 0.0f;
      }
    }
    put_operand<O>(it.to + row * it.to_ld + col, it.plane, v);
  }
}

}  // namespace

hipError_t launch_pack(const PackList &list, uint32_t dtype, hipStream_t stream) {
  uint64_t most = 0;
  for (uint32_t i = 0; i < list.count; ++i)
    if (list.item[i].chunks > most) most = list.item[i].chunks;
  if (most == 0) return hipSuccess;
  const uint64_t blocks = (most + kThreads - 1) / kThreads;
  const dim3 grid((uint32_t)(blocks < 16384 ? blocks : 16384), list.count);
  return with_type(dtype, [&](auto t) {
    pack_rows<decltype(t)><<<grid, kThreads, 0, stream>>>(list);
    return hipGetLastError();
  });
}

Shape plan_shape(uint64_t m, uint64_t n, uint32_t tiles, bool heavy) {
  Shape best = {256, 1, tiles};
  double least = 0.0;
  for (uint32_t tile = 256; tile >= 128; tile /= 2) {
    const uint64_t count = ((m + tile - 1) / tile) * ((n + tile - 1) / tile);
    for (uint32_t parts = 1; parts <= 64; parts *= 2) {
      uint32_t per = (tiles + parts - 1) / parts;
      per += per & 1;  // (a block goes by two tiles)
      const uint32_t real = (tiles + per - 1) / per;
      if (parts > 1 && (per < 16 || heavy)) break;
      const uint64_t blocks = count * real;
      double t;
      if (tile == 256)
        t = (double)((blocks + 255) / 256) * ((heavy ? 18000.0 : 8000.0) + 690.0 * per);
      else if (blocks > 512)
        t = ((double)blocks / 512 + 0.25) * ((heavy ? 8500.0 : 3500.0) + 440.0 * per);
      else if (blocks > 256)
        t = (heavy ? 12000.0 : 7000.0) + 440.0 * per;
      else
        t = (heavy ? 10000.0 : 5000.0) + 300.0 * per;
      if (real > 1) t += 3000.0 + (double)(m * n) * 4.0 * (2.0 * real) / 3500.0;
      if (least == 0.0 || t < least) {
        least = t;
        best = Shape{tile, real, per};
      }
    }
  }
  return best;
}

}  // namespace mm
}  // namespace seacells
