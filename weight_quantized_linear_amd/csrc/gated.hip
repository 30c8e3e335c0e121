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
#include "product_lds.hpp"

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

// ---------------------------------------------------------------- products in large tiles

// A slab of 32 rows and COLS columns of a wave's results on their way to 16-byte stores.  Rows of
// COLS values and 16 or 32 bytes between them, so that a wave's two halves of a write hit different banks.
template <int OUT, int COLS>
struct OutSlab {
  static constexpr int kEs = OUT ? 2 : 4, kStride = COLS * kEs + (OUT ? 16 : 32), kBytes = 32 * kStride;
  char* base;
  __device__ __forceinline__ void put(int row, int col, float v) const {
    if constexpr (OUT) *reinterpret_cast<__bf16*>(base + row * kStride + col * 2) = static_cast<__bf16>(v);
    else *reinterpret_cast<float*>(base + row * kStride + col * 4) = v;
  }
  // Rows row0 .. + 31 (below M), columns col0 .. + COLS - 1 (below N) of out, rows of ld values; vec: whole
  // 16-byte pieces at aligned addresses.
  __device__ __forceinline__ void flush(void* out, int64_t ld, int64_t row0, int64_t col0, int64_t M, int64_t N,
                                        bool vec) const {
    constexpr int kPiece = 16 / kEs, kPieces = COLS / kPiece;
    const int lane = threadIdx.x & 63;
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 32 * kPieces / 64; ++q) {
      const int row = (64 * q + lane) / kPieces, col = (64 * q + lane) % kPieces * kPiece;
      if (row0 + row >= M || col0 + col >= N) continue;
      const char* from = base + row * kStride + col * kEs;
      char* to = reinterpret_cast<char*>(out) + ((row0 + row) * ld + col0 + col) * kEs;
      if (vec) {
        *reinterpret_cast<u32x4*>(to) = lds16(from);
      } else {
#pragma unroll
        for (int e = 0; e < kPiece; ++e) {
          if (col0 + col + e >= N) break;
          if constexpr (OUT) reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(from)[e];
          else reinterpret_cast<float*>(to)[e] = reinterpret_cast<const float*>(from)[e];
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slab is read before it is written again
  }
};

// TA, TB: operand stored across k.
template <bool TA, bool TB, int BM, int BN, int S, int WY, int NW, int OUT>
__global__ __launch_bounds__(64 * NW) void product_kernel(Operand a, Operand b, void* __restrict__ out, int64_t M,
                                                          int64_t N, int64_t K, int vec) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using AOp = std::conditional_t<TA, TurnedOperand<BM, NW>, RowsOperand<BM, NW, 2, PlainRows>>;
  using BOp = std::conditional_t<TB, TurnedOperand<BN, NW>, RowsOperand<BN, NW, 2, PlainRows>>;
  using L = ProductLayout<AOp, BOp, BM, BN, S, WY, NW>;
  int64_t tm, tn;
  tile_of_block(blockIdx.x, (M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
  AOp ao;
  BOp bo;
  ao.init(a, PlainRows{tm * BM, M}, K);
  bo.init(b, PlainRows{tn * BN, N}, K);
  v16f acc[L::FM][L::FN];
  product_tile<AOp, BOp, BM, BN, S, WY, NW>(lds, ao, bo, K, acc);

  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, r = lane & 31, h = lane >> 5;
  const int64_t m0 = tm * BM + wid / L::WX * (BM / WY), n0 = tn * BN + wid % L::WX * (BN / L::WX);
  using Out = OutSlab<OUT, 32 * L::FN>;
  static_assert(NW * Out::kBytes <= L::kLds, "staging");
  block_barrier();  // every wave is done with the last strip
  const Out slab{lds + wid * Out::kBytes};
#pragma unroll
  for (int i = 0; i < L::FM; ++i) {
#pragma unroll
    for (int j = 0; j < L::FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) slab.put(8 * (v / 4) + 4 * h + v % 4, 32 * j + r, acc[i][j][v]);
    slab.flush(out, N, m0 + 32 * i, n0, M, N, vec);
  }
}

// The gated product: a wave's columns are FN / 2 times 32 gate and the 32 up columns beside them.
template <int EB, int BM, int BF, int S, int WY, int NW, int OUT>
__global__ __launch_bounds__(64 * NW) void gated_kernel(Operand x, Operand w, GatedOut o, int64_t M, int64_t F, int64_t K,
                                                        int vec, int pre_vec) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int BN = 2 * BF;
  using AOp = RowsOperand<BM, NW, 2, PlainRows>;
  using BOp = RowsOperand<BN, NW, EB, GatedRows>;
  using L = ProductLayout<AOp, BOp, BM, BN, S, WY, NW>;
  static_assert(L::FN % 2 == 0, "gate and up of a column in one wave");
  int64_t tm, tn;
  tile_of_block(blockIdx.x, (M + BM - 1) / BM, (F + BF - 1) / BF, tm, tn);
  AOp ao;
  BOp bo;
  ao.init(x, PlainRows{tm * BM, M}, K);
  bo.init(w, GatedRows{tn * BF, F}, K);
  v16f acc[L::FM][L::FN];
  product_tile<AOp, BOp, BM, BN, S, WY, NW>(lds, ao, bo, K, acc);

  constexpr int FC = L::FN / 2;  // blocks of 32 columns
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, r = lane & 31, h = lane >> 5;
  const int64_t m0 = tm * BM + wid / L::WX * (BM / WY), f0 = tn * BF + wid % L::WX * (BF / L::WX);
  using Out = OutSlab<0, 32 * FC>;  // the wider of the types that leave by it
  static_assert(NW * Out::kBytes <= L::kLds, "staging");
  block_barrier();  // every wave is done with the last strip
  char* const mine = lds + wid * Out::kBytes;
#pragma unroll
  for (int i = 0; i < L::FM; ++i) {
#pragma unroll
    for (int j = 0; j < FC; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        float g = o.alpha * acc[i][2 * j][v], u = o.alpha_up * acc[i][2 * j + 1][v];
        if (o.addend) {
          const int64_t m = m0 + 32 * i + 8 * (v / 4) + 4 * h + v % 4, f = f0 + 32 * j + r;
          if (m < M && f < F) {
            g += get_float(o.addend, m * 2 * F + f, o.addend_bf16);
            u += get_float(o.addend, m * 2 * F + F + f, o.addend_bf16);
          }
        }
        acc[i][2 * j][v] = g;
        acc[i][2 * j + 1][v] = u;
      }
    auto leave = [&](auto type, void* out, int64_t ld, int64_t col, int64_t cols, bool v16, auto value) {
      const OutSlab<decltype(type)::value, 32 * FC> slab{mine};
#pragma unroll
      for (int j = 0; j < FC; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) slab.put(8 * (v / 4) + 4 * h + v % 4, 32 * j + r, value(j, v));
      slab.flush(out, ld, m0 + 32 * i, col, M, cols, v16);
    };
    if (o.pre) {
      auto gate = [&](int j, int v) { return acc[i][2 * j][v]; };
      auto up = [&](int j, int v) { return acc[i][2 * j + 1][v]; };
      if (o.pre_bf16) {
        leave(std::integral_constant<int, 1>{}, o.pre, 2 * F, f0, F, pre_vec, gate);
        leave(std::integral_constant<int, 1>{}, reinterpret_cast<uint16_t*>(o.pre) + F, 2 * F, f0, F, pre_vec, up);
      } else {
        leave(std::integral_constant<int, 0>{}, o.pre, 2 * F, f0, F, pre_vec, gate);
        leave(std::integral_constant<int, 0>{}, reinterpret_cast<float*>(o.pre) + F, 2 * F, f0, F, pre_vec, up);
      }
    }
    auto value = [&](auto act) {
      leave(std::integral_constant<int, OUT>{}, o.out, F, f0, F, vec, [&](int j, int v) {
        return gated_one<decltype(act)::value>(acc[i][2 * j][v], acc[i][2 * j + 1][v]);
      });
    };
    if (o.act == 1) value(std::integral_constant<int, 1>{});
    else if (o.act == 2) value(std::integral_constant<int, 2>{});
    else value(std::integral_constant<int, 3>{});
  }
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

template <int V> using Int = std::integral_constant<int, V>;

// The large tiles' loads: 16-byte rows at aligned addresses, and a strip of a tile within 32-bit offsets.
bool tiled_rows(const void* p, int64_t row_bytes) {
  return aligned16(p) && row_bytes % 16 == 0 && row_bytes < (int64_t(1) << 23);
}

template <bool TA, bool TB>
hipError_t launch_product(const Operand& a, const Operand& b, void* out, int out_bf16, int64_t M, int64_t N, int64_t K,
                          int num_cus, hipStream_t s) {
  const int vec = aligned16(out) && N * (out_bf16 ? 2 : 4) % 16 == 0;
  auto go = [&](auto bm, auto bn, auto stages, auto wy, auto type) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, S = decltype(stages)::value;
    constexpr int WY = decltype(wy)::value, OUT = decltype(type)::value;
    const int64_t blocks = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
    if (blocks > kMaxGrid) return hipErrorInvalidValue;
    return launch_big_lds<product_kernel<TA, TB, BM, BN, S, WY, 8, OUT>>(S * (BM + BN) * 128, blocks, 512, s, a, b, out, M,
                                                                         N, K, vec);
  };
  auto by_type = [&](auto bm, auto bn, auto stages, auto wy) {
    return out_bf16 ? go(bm, bn, stages, wy, Int<1>{}) : go(bm, bn, stages, wy, Int<0>{});
  };
  if (((M + 255) / 256) * ((N + 255) / 256) >= num_cus) return by_type(Int<256>{}, Int<256>{}, Int<2>{}, Int<2>{});
  return by_type(Int<128>{}, Int<256>{}, Int<3>{}, Int<2>{});
}

template <bool TA, bool TB>
hipError_t launch_product_any(const uint16_t* a, int64_t lda, const uint16_t* b, int64_t ldb, void* out, int out_bf16,
                              int64_t M, int64_t N, int64_t K, hipStream_t s) {
  const int64_t blocks = (M + kAnyTile - 1) / kAnyTile * ((N + kAnyTile - 1) / kAnyTile);
  if (blocks > kMaxGrid) return hipErrorInvalidValue;
  return launch(product_any_kernel<TA, TB>, dim3(unsigned(blocks)), dim3(kThreads), 0, s, a, lda, b, ldb, out, out_bf16, M,
                N, K);
}

}  // namespace

hipError_t launch_gated_gemm(const void* w, int fp8, const uint16_t* x, const GatedOut& o, int64_t M, int64_t F, int64_t K,
                             int num_cus, hipStream_t s) {
  const int eb = fp8 ? 1 : 2;
  if (tiled_rows(x, K * 2) && tiled_rows(w, K * eb) && 2 * F * K * eb < kNowhere) {
    const Operand xo{reinterpret_cast<const char*>(x), 2 * K, M}, wo{static_cast<const char*>(w), K * eb, 2 * F};
    const int vec = aligned16(o.out) && F * (o.out_bf16 ? 2 : 4) % 16 == 0;
    const int pre_vec = aligned16(o.pre) && F * (o.pre_bf16 ? 2 : 4) % 16 == 0;
    auto go = [&](auto bytes, auto bm, auto bf, auto stages, auto wy, auto out) {
      constexpr int EB = decltype(bytes)::value, BM = decltype(bm)::value, BF = decltype(bf)::value;
      constexpr int S = decltype(stages)::value, WY = decltype(wy)::value, OUT = decltype(out)::value;
      using L = ProductLayout<RowsOperand<BM, 8, 2, PlainRows>, RowsOperand<2 * BF, 8, EB, GatedRows>, BM, 2 * BF, S, WY, 8>;
      const int64_t blocks = ((M + BM - 1) / BM) * ((F + BF - 1) / BF);
      if (blocks > kMaxGrid) return hipErrorInvalidValue;
      return launch_big_lds<gated_kernel<EB, BM, BF, S, WY, 8, OUT>>(L::kLds, blocks, 512, s, xo, wo, o, M, F, K, vec,
                                                                     pre_vec);
    };
    auto by_tile = [&](auto bytes, auto out) {
      if (M > 128) return go(bytes, Int<256>{}, Int<128>{}, Int<2>{}, Int<2>{}, out);
      return go(bytes, Int<64>{}, Int<128>{}, Int<3>{}, Int<2>{}, out);
    };
    auto by_out = [&](auto bytes) { return o.out_bf16 ? by_tile(bytes, Int<1>{}) : by_tile(bytes, Int<0>{}); };
    return fp8 ? by_out(Int<1>{}) : by_out(Int<2>{});
  }
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
  if (tiled_rows(dout, 2 * N) && tiled_rows(w, 2 * K))
    return launch_product<false, true>(Operand{reinterpret_cast<const char*>(dout), 2 * N, M},
                                       Operand{reinterpret_cast<const char*>(w), 2 * K, N}, dx, dx_bf16, M, K, N, num_cus, s);
  return launch_product_any<false, true>(dout, N, w, K, dx, dx_bf16, M, K, N, s);
}

// dw[n, k] = sum_m dout[m, n] x[m, k]
hipError_t launch_bf16_grad_w(const uint16_t* dout, const uint16_t* x, void* dw, int dw_bf16, int64_t M, int64_t N,
                              int64_t K, int num_cus, hipStream_t s) {
  if (tiled_rows(dout, 2 * N) && tiled_rows(x, 2 * K))
    return launch_product<true, true>(Operand{reinterpret_cast<const char*>(dout), 2 * N, M},
                                      Operand{reinterpret_cast<const char*>(x), 2 * K, M}, dw, dw_bf16, N, K, M, num_cus, s);
  return launch_product_any<true, true>(dout, N, x, K, dw, dw_bf16, N, K, M, s);
}

}  // namespace qlinear
