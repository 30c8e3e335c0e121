// The two element types of the row operators (1 bfloat16, 0 float32): values and 16-byte
// pieces to and from float32.
#pragma once

#include "device.hpp"

namespace qlinear {

template <int BF16> struct Elem;
template <> struct Elem<1> {
  using T = uint16_t;
  static constexpr int kPer16 = 8;
  static __device__ __forceinline__ float get(T v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ T put(float v) { return __builtin_bit_cast(T, static_cast<__bf16>(v)); }
  static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(v[i]);
      f[2 * i + 1] = bf16hi(v[i]);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // one conversion instruction per pair
      v[i] = __builtin_bit_cast(uint32_t, v2bf{static_cast<__bf16>(f[2 * i]), static_cast<__bf16>(f[2 * i + 1])});
    return v;
  }
};
template <> struct Elem<0> {
  using T = float;
  static constexpr int kPer16 = 4;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
  static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};

// Eight values as they lie in memory, at any address of their type (global loads and stores of
// 16 bytes need no alignment here); `left` of them exist, none where it is not positive.  TAIL: a
// row may end inside eight values, else left is 8 or more or nothing.
typedef u32x4 u32x4_loose __attribute__((aligned(2)));
template <int BF16>
struct Eight {
  u32x4 v[BF16 ? 1 : 2];
  static __device__ __forceinline__ u32x4 fetch(const void* p) { return *reinterpret_cast<const u32x4_loose*>(p); }
  // NT: past the caches.
  template <bool NT>
  static __device__ __forceinline__ void leave(void* p, u32x4 x) {
    if constexpr (NT) __builtin_nontemporal_store(x, reinterpret_cast<u32x4_loose*>(p));
    else *reinterpret_cast<u32x4_loose*>(p) = x;
  }
  template <bool TAIL>
  __device__ __forceinline__ void load(const void* p, int64_t i, int64_t left) {
    using V = typename Elem<BF16>::T;
    const V* q = reinterpret_cast<const V*>(p) + i;
    v[0] = u32x4{0, 0, 0, 0};
    if constexpr (!BF16) v[1] = u32x4{0, 0, 0, 0};
    if (left >= 8) {
      v[0] = fetch(q);
      if constexpr (!BF16) v[1] = fetch(q + 4);
    } else if (TAIL) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < left) {
          if constexpr (BF16) v[0][e / 2] |= uint32_t(q[e]) << (16 * (e % 2));
          else v[e / 4][e % 4] = __float_as_uint(q[e]);
        }
    }
  }
  // The same without a condition.
  __device__ __forceinline__ void get_at(const void* p, int64_t i) {
    const auto* q = reinterpret_cast<const typename Elem<BF16>::T*>(p) + i;
    v[0] = fetch(q);
    if constexpr (!BF16) v[1] = fetch(q + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (BF16) {
      Elem<1>::unpack(v[0], f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[e / 4][e % 4]);
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    if constexpr (BF16) {
      v[0] = Elem<1>::pack(f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e / 4][e % 4] = __float_as_uint(f[e]);
    }
  }
  template <bool TAIL, bool NT = false>
  __device__ __forceinline__ void store(void* p, int64_t i, int64_t left) const {
    using V = typename Elem<BF16>::T;
    V* q = reinterpret_cast<V*>(p) + i;
    if (left >= 8) {
      leave<NT>(q, v[0]);
      if constexpr (!BF16) leave<NT>(q + 4, v[1]);
    } else if (TAIL) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < left) {
          if constexpr (BF16) q[e] = uint16_t(v[0][e / 2] >> (16 * (e % 2)));
          else q[e] = __uint_as_float(v[e / 4][e % 4]);
        }
    }
  }
};

// One value at p[at].
__device__ __forceinline__ void put_float(void* p, int64_t at, float v, int bf16) {
  if (bf16) reinterpret_cast<uint16_t*>(p)[at] = Elem<1>::put(v);
  else reinterpret_cast<float*>(p)[at] = v;
}
__device__ __forceinline__ float get_float(const void* p, int64_t at, int bf16) {
  return bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[at]) : reinterpret_cast<const float*>(p)[at];
}

}  // namespace qlinear
