// What becomes of the two sums of a gated product, for the tiles that make them.
#pragma once

#include "activation.hpp"
#include "device.hpp"
#include "elem.hpp"
#include "gated_out.hpp"

namespace qlinear {

__device__ __forceinline__ float gated_value(int act, float g, float u) {
  if (act == 1) return gated_one<1>(g, u);
  if (act == 2) return gated_one<2>(g, u);
  return gated_one<3>(g, u);
}

// One output from its two sums.
__device__ __forceinline__ void gated_put(const GatedOut& o, int64_t m, int64_t f, int64_t F, float gate, float up) {
  float g = o.alpha * gate, u = o.alpha_up * up;
  const int64_t at = m * 2 * F + f;
  if (o.addend) {
    g += get_float(o.addend, at, o.addend_bf16);
    u += get_float(o.addend, at + F, o.addend_bf16);
  }
  if (o.pre) {
    put_float(o.pre, at, g, o.pre_bf16);
    put_float(o.pre, at + F, u, o.pre_bf16);
  }
  put_float(o.out, m * F + f, gated_value(o.act, g, u), o.out_bf16);
}

}  // namespace qlinear
