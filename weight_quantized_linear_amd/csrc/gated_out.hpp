// The descriptor of a gated product's result, shared by the C ABI and the kernels (a plain
// struct passed by value).
#pragma once

namespace qlinear {

// y[m, f] = act(alpha gate + c[m, f]) (alpha_up up + c[m, F + f]).  addend c [M, 2F] and pre [M, 2F],
// the two factors before the activation, may be null.
struct GatedOut {
  const void* addend;
  void *out, *pre;
  float alpha, alpha_up;
  int act, out_bf16, addend_bf16, pre_bf16;
};

}  // namespace qlinear
