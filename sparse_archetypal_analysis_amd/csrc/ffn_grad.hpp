// The first step of the gated block's gradient, for the others. Nothing here is
// exported.
#pragma once

#include "mm.hpp"

namespace seacells {

// dh = d_out w_out (product, shape) turned into d_pre and h. (A source of its
// own: its kernels take longer to compile than all the others of the gradient.)
// With a scale d_pre is held times it; where that takes a number past f16 that
// f16 holds without, all of d_pre is done again without and the scale is 1.
struct DPre {
  uint32_t dtype;
  Act act;
  mm::Args product;
  mm::Shape shape;
  const void *pre;
  uint64_t pre_ld;
  uint16_t *d_pre, *h;
  uint64_t d_ld, h_ld, d_plane, h_plane;
  uint32_t f, half;
  float *parts;
  mm::Scale *scale;  // f16, or nullptr
};
hipError_t launch_d_pre(const DPre &d, hipStream_t stream);

}  // namespace seacells
