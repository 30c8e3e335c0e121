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

// The addends of one output's factors; 0 where there are none.
struct GatedAdd {
  float gate, up;
  __device__ __forceinline__ void load(const GatedOut& o, int64_t m, int64_t f, int64_t F) {
    gate = up = 0.f;
    if (!o.addend) return;
    const int64_t at = m * 2 * F + f;
    gate = get_float(o.addend, at, o.addend_bf16);
    up = get_float(o.addend, at + F, o.addend_bf16);
  }
};

// One output from its two sums.
__device__ __forceinline__ void gated_put(const GatedOut& o, int64_t m, int64_t f, int64_t F, float gate, float up,
                                          const GatedAdd& add) {
  float g = o.alpha * gate, u = o.alpha_up * up;
  const int64_t at = m * 2 * F + f;
  if (o.addend) {
    g += add.gate;
    u += add.up;
  }
  if (o.pre) {
    put_float(o.pre, at, g, o.pre_bf16);
    put_float(o.pre, at + F, u, o.pre_bf16);
  }
  put_float(o.out, m * F + f, gated_value(o.act, g, u), o.out_bf16);
}
__device__ __forceinline__ void gated_put(const GatedOut& o, int64_t m, int64_t f, int64_t F, float gate, float up) {
  GatedAdd add;
  add.load(o, m, f, F);
  gated_put(o, m, f, F, gate, up, add);
}

}  // namespace qlinear
