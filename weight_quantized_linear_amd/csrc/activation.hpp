// The gated activations of a feed-forward layer, y = act(g) u, and their gradients, in
// float32: SiLU (the swiglu calls and the gated products), tanh-form GELU and ReLU.
#pragma once

#include <hip/hip_runtime.h>

namespace qlinear {

// What sigmoid(g) and sigmoid(-g) are made of, from h = exp(-|g| / 2): near = 1 / (1 + h^2) =
// sigmoid(|g|); half = 1 for g >= 0, else h, so that sigmoid(g) = half^2 near; rest = sigmoid(-g).  Nothing
// overflows or cancels.  A negative gate's two halves go to different factors of a
// product: h^2 leaves float32's normal range below g = -87 (and the exponential instruction gives 0
// there), where its product with u or dy need not, and h only below g = -174.
// Good to a few float32 roundings (u = 2^-24): |g| log2(e) / 2 is taken with the
// rounding error of its product, so h is off by 3 u (the instruction itself by 2) and h^2 by 7, 1 + h^2
// adds one, and a Newton step leaves one of the reciprocal.  Beyond |g| = 256 nothing changes (h = 0).
// The library's expf and division would be twice the instructions, and the forward pass over
// bfloat16 was bound by them.
__device__ __forceinline__ void sigmoids(float g, float& near, float& half, float& rest) {
  constexpr float kHi = 0.5f * 1.44269502f, kLo = 0.5f * 1.92596299e-8f;  // log2(e) / 2
  const float a = fminf(fabsf(g), 256.f);
  const float t = -a * kHi;
  const float r = fmaf(-a, kLo, fmaf(-a, kHi, -t));
  float h = __builtin_amdgcn_exp2f(t);
  h = fmaf(h, r * 0.693147182f, h);
  const float d = fmaf(h, h, 1.f), y = __builtin_amdgcn_rcpf(d);
  near = fmaf(y, fmaf(-d, y, 1.f), y);
  half = g >= 0.f ? 1.f : h;
  rest = g >= 0.f ? h * h * near : near;
}

__device__ __forceinline__ float swiglu_one(float g, float u) {
  float near, half, rest;
  sigmoids(g, near, half, rest);
  return (g * near * half) * (u * half);
}

// dgate = dy u sig (1 + g (1 - sig)), dup = dy g sig, with sigmoid(-g) for 1 - sig.  dy u alone
// could overflow where the gradient does not.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dy, float& dg, float& du) {
  float near, half, rest;
  sigmoids(g, near, half, rest);
  const float dh = dy * half;
  dg = dh * (u * half) * (near * fmaf(g, rest, 1.f));
  du = dh * (g * near * half);
}

// GELU in its tanh form is g sigmoid(z), z = 2 sqrt(2 / pi) (g + 0.044715 g^3); beyond |g| = 32 the sigmoid
// is 0 or 1 in float32, so z and its slope are taken at g clamped there, where neither overflows.
constexpr float kGeluRate = 2.f * 0.7978845608028654f, kGeluCube = 0.044715f;

__device__ __forceinline__ float gelu_one(float g, float u) {
  const float c = fminf(fmaxf(g, -32.f), 32.f);
  float near, half, rest;
  sigmoids(kGeluRate * c * fmaf(kGeluCube * c, c, 1.f), near, half, rest);
  return (g * near * half) * (u * half);
}

// d(g sigmoid(z))/dg = sigmoid(z) (1 + g sigmoid(-z) z').  Beyond |g| = 32 either sigmoid is 0, and g z' would
// pass float32's range from 1.5e36 on: g is clamped there too, a NaN stays.
__device__ __forceinline__ void gelu_grad(float g, float u, float dy, float& dg, float& du) {
  const float c = fminf(fmaxf(g, -32.f), 32.f);
  float near, half, rest;
  sigmoids(kGeluRate * c * fmaf(kGeluCube * c, c, 1.f), near, half, rest);
  const float slope = kGeluRate * fmaf(3.f * kGeluCube * c, c, 1.f);
  const float dh = dy * half;
  dg = dh * (u * half) * (near * fmaf(fabsf(g) > 32.f ? c : g, rest * slope, 1.f));
  du = dh * (g * near * half);
}

// ACT as qlinear_activation: 1 ReLU, 2 SiLU, 3 GELU (tanh form).  A NaN gate stays NaN.
template <int ACT>
__device__ __forceinline__ float gated_one(float g, float u) {
  if constexpr (ACT == 1) return (g < 0.f ? 0.f : g) * u;
  else if constexpr (ACT == 2) return swiglu_one(g, u);
  else return gelu_one(g, u);
}

template <int ACT>
__device__ __forceinline__ void gated_grad(float g, float u, float dy, float& dg, float& du) {
  if constexpr (ACT == 1) {
    dg = g <= 0.f ? 0.f : dy * u;
    du = dy * (g < 0.f ? 0.f : g);
  } else if constexpr (ACT == 2) {
    swiglu_grad(g, u, dy, dg, du);
  } else {
    gelu_grad(g, u, dy, dg, du);
  }
}

}  // namespace qlinear
