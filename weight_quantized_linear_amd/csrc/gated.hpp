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

__device__ __forceinline__ void put_float(void* p, int64_t at, float v, int bf16) {
  if (bf16) reinterpret_cast<uint16_t*>(p)[at] = Elem<1>::put(v);
  else reinterpret_cast<float*>(p)[at] = v;
}
__device__ __forceinline__ float get_float(const void* p, int64_t at, int bf16) {
  return bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[at]) : reinterpret_cast<const float*>(p)[at];
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
