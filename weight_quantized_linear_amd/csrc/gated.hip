// The gated product of a feed-forward layer, both projections, the activation and the product
// in one kernel, and the products of its gradients:
//   pre = x W^T + c  (W = [W_gate; W_up], [2F, K]),   y = act(pre_gate) pre_up
//   dpre = [dy pre_up act'(pre_gate), dy act(pre_gate)],   dx = dpre W,   dW = dpre^T x.
// float32 sums; pre-activations leave the registers only where the caller keeps them for
// the backward pass, so the 2F columns are neither written nor read again.
#include "activation.hpp"
#include "device.hpp"
#include "elem.hpp"
#include "gated.hpp"
#include "launch.hpp"

namespace qlinear {

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- products of any shape

// C[m, n] = sum_k A[m, k] B[n, k] in tiles of 64 x 64, for sizes and addresses that the tiles
// with wide loads do not take.  A and B lie with k contiguous (TA / TB false: rows of `lda`) or
// with the other axis contiguous.  Operands go through LDS as bfloat16 (FP8 codes widen exactly).
// 4 waves of 32 x 32, MFMA 16x16x32.  GATED: rows 0 .. 31 of the tile's B are gate rows, 32 .. 63
// the up rows of the same columns, so a lane holds both factors of its outputs.
constexpr int kAnyTile = 64, kAnyK = 32, kAnyRow = 40;  // LDS row of 32 values and 8 of padding

template <typename T>
__device__ __forceinline__ uint16_t to_bf16(T v) {
  if constexpr (sizeof(T) == 2) return v;
  else return uint16_t(__float_as_uint(e4m3_to_f32(v)) >> 16);
}

// A 64 x 32 piece: rows r0.. (mapped by `row_of`, negative: none) and k0.. of an operand.
template <bool TRANS, typename T, typename RowOf>
__device__ __forceinline__ void any_load(uint16_t (*tile)[kAnyRow], const T* __restrict__ p, int64_t ld, int64_t k0,
                                         int64_t K, RowOf row_of) {
  if constexpr (!TRANS) {
    const int r = threadIdx.x / 4, c = threadIdx.x % 4 * 8;
    const int64_t row = row_of(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t k = k0 + c + e;
      tile[r][c + e] = row >= 0 && k < K ? to_bf16<T>(p[row * ld + k]) : uint16_t(0);
    }
  } else {
    const int r = threadIdx.x % 64;
    const int64_t row = row_of(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = threadIdx.x / 64 * 8 + e;
      tile[r][c] = row >= 0 && k0 + c < K ? to_bf16<T>(p[(k0 + c) * ld + row]) : uint16_t(0);
    }
  }
}

template <bool TA, bool TB, bool GATED, typename T, typename Store>
__device__ __forceinline__ void any_tile(const uint16_t* __restrict__ a, int64_t lda, const T* __restrict__ b,
                                         int64_t ldb, int64_t m0, int64_t n0, int64_t M, int64_t N, int64_t K,
                                         Store store) {
  __shared__ __attribute__((aligned(16))) uint16_t as[kAnyTile][kAnyRow], bs[kAnyTile][kAnyRow];
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const int wy = wid / 2, wx = wid % 2;
  auto row_a = [&](int r) { return m0 + r < M ? m0 + r : int64_t(-1); };
  auto row_b = [&](int r) {
    if constexpr (GATED) return n0 + r % 32 < N ? n0 + r % 32 + (r / 32) * N : int64_t(-1);
    else return n0 + r < N ? n0 + r : int64_t(-1);
  };
  v4f acc[2][2];
#pragma unroll
  for (int m = 0; m < 2; ++m) acc[m][0] = acc[m][1] = v4f{};
  for (int64_t k0 = 0; k0 < K; k0 += kAnyK) {
    any_load<TA>(as, a, lda, k0, K, row_a);
    any_load<TB>(bs, b, ldb, k0, K, row_b);
    __syncthreads();
    v8bf af[2], bf[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      af[m] = *reinterpret_cast<const v8bf*>(&as[32 * wy + 16 * m + i][8 * q]);
      bf[m] = *reinterpret_cast<const v8bf*>(&bs[GATED ? 32 * m + 16 * wx + i : 32 * wx + 16 * m + i][8 * q]);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[m], bf[j], acc[m][j], 0, 0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t row = m0 + 32 * wy + 16 * m + 4 * q + v;
      if (row >= M) continue;
      if constexpr (GATED) {
        const int64_t n = n0 + 16 * wx + i;
        if (n < N) store(row, n, acc[m][0][v], acc[m][1][v]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int64_t n = n0 + 32 * wx + 16 * j + i;
          if (n < N) store(row, n, acc[m][j][v], 0.f);
        }
      }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_any_kernel(const T* __restrict__ w, const uint16_t* __restrict__ x,
                                                            int64_t M, int64_t F, int64_t K, GatedOut o) {
  const int64_t tiles_n = (F + 31) / 32, m0 = blockIdx.x / tiles_n * kAnyTile, n0 = blockIdx.x % tiles_n * 32;
  any_tile<false, false, true>(x, K, w, K, m0, n0, M, F, K,
                               [&](int64_t m, int64_t f, float gate, float up) { gated_put(o, m, f, F, gate, up); });
}

// TA, TB as any_tile; out[m, n] of float32 or bfloat16.
template <bool TA, bool TB>
__global__ __launch_bounds__(kThreads) void product_any_kernel(const uint16_t* __restrict__ a, int64_t lda,
                                                              const uint16_t* __restrict__ b, int64_t ldb,
                                                              void* __restrict__ out, int out_bf16, int64_t M, int64_t N,
                                                              int64_t K) {
  const int64_t tiles_n = (N + kAnyTile - 1) / kAnyTile;
  any_tile<TA, TB, false>(a, lda, b, ldb, blockIdx.x / tiles_n * kAnyTile, blockIdx.x % tiles_n * kAnyTile, M, N, K,
                          [&](int64_t m, int64_t n, float v, float) {
                            if (out_bf16) reinterpret_cast<uint16_t*>(out)[m * N + n] = Elem<1>::put(v);
                            else reinterpret_cast<float*>(out)[m * N + n] = v;
                          });
}

// ---------------------------------------------------------------- gradient of the activation

// dpre of kPer values a thread; VEC: 16-byte aligned rows, whole pieces.
template <int ACT, int DY, int PRE, bool VEC>
__global__ __launch_bounds__(kThreads) void gated_grad_kernel(const void* __restrict__ dy, const void* __restrict__ pre,
                                                             uint16_t* __restrict__ dpre, int64_t M, int64_t F) {
  constexpr int P = VEC ? 8 : 1;
  const int64_t per = (F + P - 1) / P;
  for (int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x; at < M * per; at += int64_t(gridDim.x) * kThreads) {
    const int64_t m = at / per, f = at % per * P;
    float d[P], g[P], u[P];
    if constexpr (VEC) {
      load_eight<DY>(dy, m * F + f, d);
      load_eight<PRE>(pre, m * 2 * F + f, g);
      load_eight<PRE>(pre, m * 2 * F + F + f, u);
    } else {
      d[0] = Elem<DY>::get(reinterpret_cast<const typename Elem<DY>::T*>(dy)[m * F + f]);
      g[0] = Elem<PRE>::get(reinterpret_cast<const typename Elem<PRE>::T*>(pre)[m * 2 * F + f]);
      u[0] = Elem<PRE>::get(reinterpret_cast<const typename Elem<PRE>::T*>(pre)[m * 2 * F + F + f]);
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
      float dg, du;
      gated_grad<ACT>(g[e], u[e], d[e], dg, du);
      g[e] = dg;
      u[e] = du;
    }
    uint16_t* const o = dpre + m * 2 * F + f;
    if constexpr (VEC) {
      *reinterpret_cast<u32x4*>(o) = Elem<1>::pack(g);
      *reinterpret_cast<u32x4*>(o + F) = Elem<1>::pack(u);
    } else {
      o[0] = Elem<1>::put(g[0]);
      o[F] = Elem<1>::put(u[0]);
    }
  }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

template <typename F>
hipError_t by_act(int act, F&& go) {
  if (act == 1) return go(std::integral_constant<int, 1>{});
  if (act == 2) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 3>{});
}

}  // namespace

hipError_t launch_gated_gemm(const void* w, int fp8, const uint16_t* x, const GatedOut& o, int64_t M, int64_t F, int64_t K,
                             int num_cus, hipStream_t s) {
  const int64_t blocks = (M + kAnyTile - 1) / kAnyTile * ((F + 31) / 32);
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  if (fp8)
    return launch(gated_any_kernel<uint8_t>, dim3(unsigned(blocks)), dim3(kThreads), 0, s,
                  static_cast<const uint8_t*>(w), x, M, F, K, o);
  return launch(gated_any_kernel<uint16_t>, dim3(unsigned(blocks)), dim3(kThreads), 0, s,
                static_cast<const uint16_t*>(w), x, M, F, K, o);
}

hipError_t launch_gated_grad(const void* dy, int dy_bf16, const void* pre, int pre_bf16, uint16_t* dpre, int act, int64_t M,
                             int64_t F, hipStream_t s) {
  const bool vec = F % 8 == 0 && aligned16(dy) && aligned16(pre) && aligned16(dpre);
  const int64_t items = M * (vec ? F / 8 : F), blocks = (items + kThreads - 1) / kThreads;
  return by_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    auto go = [&](auto kernel) {
      return launch(kernel, dim3(unsigned(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0, s, dy, pre, dpre, M, F);
    };
    auto by_vec = [&](auto v) {
      constexpr bool VEC = decltype(v)::value;
      if (dy_bf16) return pre_bf16 ? go(gated_grad_kernel<ACT, 1, 1, VEC>) : go(gated_grad_kernel<ACT, 1, 0, VEC>);
      return pre_bf16 ? go(gated_grad_kernel<ACT, 0, 1, VEC>) : go(gated_grad_kernel<ACT, 0, 0, VEC>);
    };
    return vec ? by_vec(std::true_type{}) : by_vec(std::false_type{});
  });
}

// dx[m, k] = sum_n dout[m, n] w[n, k]
hipError_t launch_bf16_grad_x(const uint16_t* dout, const uint16_t* w, void* dx, int dx_bf16, int64_t M, int64_t N,
                              int64_t K, int num_cus, hipStream_t s) {
  const int64_t blocks = (M + kAnyTile - 1) / kAnyTile * ((K + kAnyTile - 1) / kAnyTile);
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  return launch(product_any_kernel<false, true>, dim3(unsigned(blocks)), dim3(kThreads), 0, s, dout, N, w, K, dx, dx_bf16,
                M, K, N);
}

// dw[n, k] = sum_m dout[m, n] x[m, k]
hipError_t launch_bf16_grad_w(const uint16_t* dout, const uint16_t* x, void* dw, int dw_bf16, int64_t M, int64_t N,
                              int64_t K, int num_cus, hipStream_t s) {
  const int64_t blocks = (N + kAnyTile - 1) / kAnyTile * ((K + kAnyTile - 1) / kAnyTile);
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  return launch(product_any_kernel<true, true>, dim3(unsigned(blocks)), dim3(kThreads), 0, s, dout, N, x, K, dw, dw_bf16,
                N, K, M);
}

}  // namespace qlinear
