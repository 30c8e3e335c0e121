// The gated product of a feed-forward layer, both projections, the activation and the product
// in one kernel, and the products of its gradients:
//   pre = x W^T + c  (W = [W_gate; W_up], [2F, K]),   y = act(pre_gate) pre_up
//   dpre = [dy pre_up act'(pre_gate), dy act(pre_gate)],   dx = dpre W,   dW = dpre^T x.
// float32 sums; pre-activations leave the registers only where the caller keeps them for
// the backward pass, so the 2F columns are neither written nor read again.
#include <algorithm>

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

// C[m, n] = sum_k A[m, k] B[n, k] in tiles of 64 x 64, for K below the 8 or 16 values that the other tiles
// load at once.  A and B lie with k contiguous (TA / TB false: rows of `lda`) or
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

// ---------------------------------------------------------------- few rows

// Sixteen bytes at any address (global loads need no alignment here).
typedef u32x4 u32x4_loose __attribute__((aligned(1)));
__device__ __forceinline__ u32x4 ld16_loose(const void* p) { return *reinterpret_cast<const u32x4_loose*>(p); }
__device__ __forceinline__ u32x4 ld16_loose_stream(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_loose*>(p));
}

// M <= 4 rows at any size and address, on the vector ALU: a wave has one column, whose gate and up rows it reads in
// contiguous KiB, 2 U loads in flight a lane; products of pairs by the bfloat16 dot instruction (exact,
// float32 sums).  Bound by HBM: one row of x, F = 14336, K = 4096, FP8: 18.6 us, 6.3 TB/s;
// bfloat16 35, 6.7 TB/s (here and below: the kernel alone, no operand in a cache, if nothing else is said).
template <int EB, int M, int U>
__global__ __launch_bounds__(256) void gated_gemv_kernel(const char* __restrict__ w, const uint16_t* __restrict__ x,
                                                        GatedOut o, int64_t F, int64_t K) {
  constexpr int kValues = 16 / EB, X = kValues / 8;  // values of a load of w, loads of x beside it
  const int lane = threadIdx.x % kWave;
  const int64_t f = int64_t(blockIdx.x) * (256 / kWave) + threadIdx.x / kWave;
  if (f >= F) return;  // the whole wave
  const int64_t row_bytes = K * EB;
  const char* const rows[2] = {w + f * row_bytes, w + (F + f) * row_bytes};
  float acc[M][2];
#pragma unroll
  for (int m = 0; m < M; ++m) acc[m][0] = acc[m][1] = 0.f;
  const int64_t whole = K / kValues;  // whole loads of a row
  for (int64_t c0 = 0; c0 < whole; c0 += kWave * U) {
    u32x4 wv[U][2], xv[U][M][X];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int64_t c = c0 + n * kWave + lane, at = c < whole ? c : whole - 1;
#pragma unroll
      for (int r = 0; r < 2; ++r) wv[n][r] = ld16_loose_stream(rows[r] + 16 * at);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int e = 0; e < X; ++e) xv[n][m][e] = ld16_loose(x + m * K + at * kValues + 8 * e);
    }
    if (c0 + kWave * U > whole) {  // loads are never conditional: what lies past the row's end is dropped here
#pragma unroll
      for (int n = 0; n < U; ++n) {
        if (c0 + n * kWave + lane < whole) continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) wv[n][r] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int e = 0; e < X; ++e) xv[n][m][e] = u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int n = 0; n < U; ++n)
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const uint32_t word = wv[n][r][d];
            if constexpr (EB == 1) {
              const u32x4& xa = xv[n][m][d / 2];
              const uint32_t x01 = xa[2 * (d % 2)], x23 = xa[2 * (d % 2) + 1];
              acc[m][r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(e4m3x2_to_bf16x2<false>(word)), as_bf16x2(x01),
                                                          acc[m][r], false);
              acc[m][r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(e4m3x2_to_bf16x2<true>(word)), as_bf16x2(x23),
                                                          acc[m][r], false);
            } else {
              const uint32_t xw = xv[n][m][0][d];
              acc[m][r] = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(word), as_bf16x2(xw), acc[m][r], false);
            }
          }
  }
  if (const int64_t k = whole * kValues + lane; k < K) {  // the values behind the last whole load, one a lane
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float v;
        if constexpr (EB == 1) v = e4m3_to_f32(uint8_t(rows[r][k]));
        else v = bf16_to_f32(reinterpret_cast<const uint16_t*>(rows[r])[k]);
        acc[m][r] = fmaf(v, bf16_to_f32(x[m * K + k]), acc[m][r]);
      }
  }
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float g = wave_sum(acc[m][0]), u = wave_sum(acc[m][1]);
    if (lane == m) gated_put(o, m, f, F, g, u);
  }
}

// M <= 16 rows: bound by the weights' bytes, which therefore go to LDS in whole 1 KiB pieces of a row (into
// registers, 64 bytes of 16 rows a load, the same bytes come at 3.5 to 4.5 TB/s).  A block walks tiles of 8 columns, that
// is 8 gate and 8 up rows, as the 16 rows of one MFMA operand, through a ring of S stages of 2 KiB a row; each of its
// 8 waves takes an eighth of every stage, so the part of x that it meets stays in its registers (KS
// stages a row), and the waves' sums meet in LDS at a tile's end.  MFMA 16x16x32: the weights' rows are the
// result's rows and the tokens its columns: lanes 0 .. 31 end with four gate columns of a token, lanes 32 .. 63
// with the up ones.  FP8: a lane's 16 bytes are the operands of two steps, and x is held in that order.
// ADD: the addends of eight tiles at a time wait in LDS; loaded at a tile's end they would come behind all weights on
// their way (F = 5504, K = 2048, bfloat16 15 us, 12 from LDS).  The form without has no registers for that in FP8.
// M = 13, K = 4096, F = 14336: 25 us FP8 (4.7 TB/s), 43 bfloat16 (5.4), with addends 32 and 46 to 49; K = 2048, F = 5504,
// bfloat16 11
// (4.0: of its 1.3 tiles a block the first loads' and the last sums' latency shows).  Weights kept in the caches: 1 to
// 2 us more.
constexpr int kAddTiles = 8, kAddBytes = kAddTiles * 16 * 16 * 4;  // tiles whose addends LDS holds
template <int EB, int KS, int S, bool ADD>
__global__ __launch_bounds__(512) void gated_rows_kernel(const char* __restrict__ w, const uint16_t* __restrict__ x,
                                                        GatedOut o, int M, int64_t F, int64_t K) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int NW = 8, kRow = 2048, kStage = 16 * kRow;
  constexpr int kParts = kRow / 1024, kDma = 16 * kParts / NW;
  constexpr int kSteps = kRow / NW / 64;      // loads of 16 bytes a lane per stage
  constexpr int kValues = 16 / EB, E = kValues / 8;  // values of a load, MFMA steps of it
  v4f(*const sums)[kWave] = reinterpret_cast<v4f(*)[kWave]>(lds + S * kStage);
  float* const adds = reinterpret_cast<float*>(lds + S * kStage + NW * kWave * 16);  // [tile][token][gate, up][8]
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const int64_t tiles = (F + 7) / 8, row_bytes = K * EB;
  const int stages = int((tiles - 1 - blockIdx.x) / gridDim.x + 1) * KS;

  // Stage j is part j % KS of the rows of the block's tile j / KS.  Row r: gate f0 + r, or up f0 + r - 8.
  // Pieces past a row's end are zeros; rows past F hold others' values or zeros and are not stored.
  uint32_t off[kDma];
#pragma unroll
  for (int n = 0; n < kDma; ++n) {
    const int r = (wid * kDma + n) / kParts;
    off[n] = uint32_t(((r & 7) + (r & 8 ? F : 0)) * row_bytes);
  }
  auto issue = [&](int j) {
    const int64_t f0 = (blockIdx.x + int64_t(j / KS) * gridDim.x) * 8;
    const __amdgpu_buffer_rsrc_t res = strip_rsrc(w + f0 * row_bytes, (2 * F - f0) * row_bytes, false);
    char* const slot = lds + j % S * kStage;
#pragma unroll
    for (int n = 0; n < kDma; ++n) {
      const int r = (wid * kDma + n) / kParts, p = (wid * kDma + n) % kParts;
      const uint32_t at = j % KS * kRow + 1024 * p + 16 * (lane ^ r);
      bdma16_nt(res, slot + r * kRow + 1024 * p, at < uint32_t(row_bytes) ? off[n] + at : kNowhere);
    }
  };
  issue(0);
  // This lane's part of x: bounded loads, so that none waits for another's condition.
  v8bf xf[KS][kSteps][E];
  const __amdgpu_buffer_rsrc_t xres = make_rsrc(x, M * K * 2);
#pragma unroll
  for (int h = 0; h < KS; ++h)
#pragma unroll
    for (int c = 0; c < kSteps; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t k = (h * kRow + wid * (kRow / NW) + 64 * c + 16 * q) / EB + 8 * e;
        const uint32_t at = i < M && k < uint32_t(K) ? (i * uint32_t(K) + k) * 2 : kNowhere;
        xf[h][c][e] = __builtin_bit_cast(v8bf, __builtin_amdgcn_raw_buffer_load_b128(xres, at, 0, 0));
      }
#pragma unroll
  for (int j = 1; j < S; ++j)
    if (j < stages) issue(j);

  v4f acc[2] = {v4f{}, v4f{}};
  for (int j = 0; j < stages; ++j) {
    const int ahead = stages - 1 - j;  // later stages, of which at most S - 1 are on their way
    if (ahead >= S - 1) wait_vm<(S - 1) * kDma>();
    else if (ahead == 2) wait_vm<2 * kDma>();
    else if (ahead == 1) wait_vm<kDma>();
    else wait_vm<0>();
    block_barrier();
    const int n = j / KS, h = j % KS;
    if (ADD && h == 0 && n % kAddTiles == 0) {
#pragma unroll
      for (int e = 0; e < kAddTiles * 256 / 512; ++e) {
        const int at = e * 512 + int(threadIdx.x), i2 = at / 16 % 16;
        const int64_t f = (blockIdx.x + (n + at / 256) * int64_t(gridDim.x)) * 8 + at % 8;
        if (i2 < M && f < F) adds[at] = get_float(o.addend, (2 * i2 + at / 8 % 2) * F + f, o.addend_bf16);
      }
    }
    const char* const row = lds + j % S * kStage + i * kRow;
    u32x4 wv[kSteps];
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      const int at = wid * (kRow / NW) + 64 * c + 16 * q;  // a permuted piece stays in its KiB
      wv[c] = lds16(row + (at ^ (i << 4)));
    }
#pragma unroll
    for (int hh = 0; hh < KS; ++hh) {
      if (hh != h) continue;  // uniform; the register arrays keep constant indexes
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v8bf a;
          if constexpr (EB == 1) a = e4m3x8_to_bf16x8(wv[c][2 * e], wv[c][2 * e + 1]);
          else a = __builtin_bit_cast(v8bf, wv[c]);
          acc[(c * E + e) % 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, xf[hh][c][e], acc[(c * E + e) % 2], 0, 0, 0);
        }
    }
    const bool last = h == KS - 1;
    if (last) sums[wid][lane] = acc[0] + acc[1];
    wait_lds();
    block_barrier();  // the slot is read, and at a tile's end the sums are there
    if (j + S < stages) issue(j + S);
    if (last) {
      if (wid == n % NW) {
        v4f sum = sums[0][lane];
#pragma unroll
        for (int v = 1; v < NW; ++v) sum += sums[v][lane];
        v4f add[2] = {v4f{}, v4f{}};
        if (ADD)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            add[e] = *reinterpret_cast<const v4f*>(adds + ((n % kAddTiles * 16 + i) * 2 + e) * 8 + 4 * (q & 1));
        const int64_t f = (blockIdx.x + int64_t(n) * gridDim.x) * 8 + 4 * (q & 1);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float up = __shfl_down(sum[v], 32, kWave);
          if (q < 2 && i < M && f + v < F) gated_put(o, i, f + v, F, sum[v], up, GatedAdd{add[0][v], add[1][v]});
        }
      }
      acc[0] = acc[1] = v4f{};
    }
  }
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

// A wave's results, FM x FN blocks of 32 x 32 from row m0 and column n0 on, through its slab at `mine`.
template <int OUT, int FM, int FN>
__device__ __forceinline__ void product_out(char* mine, const v16f (&acc)[FM][FN], void* out, int64_t m0, int64_t n0,
                                            int64_t M, int64_t N, bool vec) {
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const OutSlab<OUT, 32 * FN> slab{mine};
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) slab.put(8 * (v / 4) + 4 * h + v % 4, 32 * j + r, acc[i][j][v]);
    slab.flush(out, N, m0 + 32 * i, n0, M, N, vec);
  }
}

// TA, TB: operand stored across k.  Bound by the matrix cores: 8192 x 4096 x 8192 in tiles of 256 x 256 484 us, 1.14
// PFLOP/s, of whose
// time the SIMDs' matrix cores work 64 % (dx) and 60 % (dw), bank conflicts take 1 %; 4096 x 2048, K = 11264 (dx) 219
// us in tiles of 128 x 128, 11264 x 2048, K = 4096 (dw) 180 in tiles of 192 x 128.  blockIdx.y: a part of K, whose sums
// go to the float32 plane of its own behind out.
template <bool TA, bool TB, int BM, int BN, int S, int WY, int NW, int OUT>
__global__ __launch_bounds__(64 * NW) void product_kernel(Operand a, Operand b, void* __restrict__ out, int64_t M,
                                                          int64_t N, int64_t K, int64_t strips, int vec) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using AOp = std::conditional_t<TA, TurnedOperand<BM, NW>, RowsOperand<BM, NW, 2, PlainRows>>;
  using BOp = std::conditional_t<TB, TurnedOperand<BN, NW>, RowsOperand<BN, NW, 2, PlainRows>>;
  using L = ProductLayout<AOp, BOp, BM, BN, S, WY, NW>;
  static_assert(NW * OutSlab<OUT, 32 * L::FN>::kBytes <= L::kLds, "staging");
  int64_t tm, tn;
  tile_of_block(blockIdx.x, (M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
  AOp ao;
  BOp bo;
  ao.init(a, PlainRows{tm * BM, M}, K);
  bo.init(b, PlainRows{tn * BN, N}, K);
  v16f acc[L::FM][L::FN];
  const int64_t all = (K + kStripK - 1) / kStripK, s0 = blockIdx.y * strips;
  product_tile<AOp, BOp, BM, BN, S, WY, NW>(lds, ao, bo, K, s0, all - s0 < strips ? all - s0 : strips, acc);
  const int wid = threadIdx.x >> 6;
  block_barrier();  // every wave is done with the last strip
  product_out<OUT>(lds + wid * OutSlab<OUT, 32 * L::FN>::kBytes, acc,
                   reinterpret_cast<char*>(out) + blockIdx.y * M * N * (OUT ? 2 : 4), tm * BM + wid / L::WX * (BM / WY),
                   tn * BN + wid % L::WX * (BN / L::WX), M, N, vec);
}

// The same at any address, 128 x 128: 515 x 1023, K = 2730 (dx, split in five) 20 us and 6 for the sum of its parts,
// 2730 x 1023, K = 515
// (dw) 20; few blocks whose strips come through registers, so the strips' latency shows.  K and the widths of turned
// operands are 8 at least.
template <bool TA, bool TB, int OUT>
__global__ __launch_bounds__(256) void product_staged_kernel(Operand a, Operand b, void* __restrict__ out, int64_t M,
                                                            int64_t N, int64_t K, int64_t strips) {
  constexpr int BM = 128, BN = 128, WY = 2, NW = 4;
  using AOp = std::conditional_t<TA, StagedTurned<BM, NW, 8>, StagedRows<BM, NW, 2, PlainRows, 8>>;
  using BOp = std::conditional_t<TB, StagedTurned<BN, NW, 8>, StagedRows<BN, NW, 2, PlainRows, 8>>;
  constexpr int kSlab = OutSlab<OUT, 64>::kBytes, kTiles = AOp::kBytes + BOp::kBytes;
  __shared__ __attribute__((aligned(16))) char lds[kTiles > NW * kSlab ? kTiles : NW * kSlab];
  int64_t tm, tn;
  tile_of_block(blockIdx.x, (M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn);
  const int64_t all = (K + kStripK - 1) / kStripK, s0 = blockIdx.y * strips;
  AOp ao;
  BOp bo;
  ao.init(a, PlainRows{tm * BM, M}, K, s0);
  bo.init(b, PlainRows{tn * BN, N}, K, s0);
  v16f acc[2][2];
  staged_tile<AOp, BOp, BM, BN, WY, NW>(lds, ao, bo, s0, all - s0 < strips ? all - s0 : strips, acc);
  const int wid = threadIdx.x >> 6;
  wait_lds();
  block_barrier();
  product_out<OUT>(lds + wid * kSlab, acc, reinterpret_cast<char*>(out) + blockIdx.y * M * N * (OUT ? 2 : 4),
                   tm * BM + wid / 2 * 64, tn * BN + wid % 2 * 64, M, N, false);
}

// A wave's part of a gated product: its columns are FN / 2 times 32 gate and the 32 up columns beside them.
template <int OUT, int FM, int FN>
__device__ __forceinline__ void gated_out(char* mine, v16f (&acc)[FM][FN], const GatedOut& o, int64_t m0, int64_t f0,
                                          int64_t M, int64_t F, bool vec, bool pre_vec) {
  static_assert(FN % 2 == 0, "gate and up of a column in one wave");
  constexpr int FC = FN / 2;  // blocks of 32 columns
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
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
    auto leave = [&](auto type, void* out, int64_t ld, bool v16, auto value) {
      const OutSlab<decltype(type)::value, 32 * FC> slab{mine};
#pragma unroll
      for (int j = 0; j < FC; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) slab.put(8 * (v / 4) + 4 * h + v % 4, 32 * j + r, value(j, v));
      slab.flush(out, ld, m0 + 32 * i, f0, M, F, v16);
    };
    if (o.pre) {
      auto gate = [&](int j, int v) { return acc[i][2 * j][v]; };
      auto up = [&](int j, int v) { return acc[i][2 * j + 1][v]; };
      if (o.pre_bf16) {
        leave(std::integral_constant<int, 1>{}, o.pre, 2 * F, pre_vec, gate);
        leave(std::integral_constant<int, 1>{}, reinterpret_cast<uint16_t*>(o.pre) + F, 2 * F, pre_vec, up);
      } else {
        leave(std::integral_constant<int, 0>{}, o.pre, 2 * F, pre_vec, gate);
        leave(std::integral_constant<int, 0>{}, reinterpret_cast<float*>(o.pre) + F, 2 * F, pre_vec, up);
      }
    }
    auto value = [&](auto act) {
      leave(std::integral_constant<int, OUT>{}, o.out, F, vec,
            [&](int j, int v) { return gated_one<decltype(act)::value>(acc[i][2 * j][v], acc[i][2 * j + 1][v]); });
    };
    if (o.act == 1) value(std::integral_constant<int, 1>{});
    else if (o.act == 2) value(std::integral_constant<int, 2>{});
    else value(std::integral_constant<int, 3>{});
  }
}

// Bound by the matrix cores from 256 rows on, below by the weights' bytes.  bfloat16, M = 4096, F = 5632, K = 2048 with
// float32
// pre-activations 208 us, 0.91 PFLOP/s, the matrix cores at work 69 % of the cycles at K = 8192; FP8, F = 14336, K = 4096:
// M = 500 110 us, 1.06 PFLOP/s, M = 64 32 us, 3.7 TB/s.  SK: values of k in a strip; NT: weights past the caches.
template <int EB, int BM, int BF, int SK, int S, int NW, bool NT, int OUT>
__global__ __launch_bounds__(64 * NW) void gated_kernel(Operand x, Operand w, GatedOut o, int64_t M, int64_t F, int64_t K,
                                                        int vec, int pre_vec) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int BN = 2 * BF, WY = 2;
  using AOp = RowsOperand<BM, NW, 2, PlainRows, SK>;
  using BOp = RowsOperand<BN, NW, EB, GatedRows, SK, NT>;
  using L = ProductLayout<AOp, BOp, BM, BN, S, WY, NW>;
  constexpr int kSlab = OutSlab<0, 16 * L::FN>::kBytes;  // the wider of the types that leave by it
  static_assert(NW * kSlab <= L::kLds, "staging");
  int64_t tm, tn;
  tile_of_block(blockIdx.x, (M + BM - 1) / BM, (F + BF - 1) / BF, tm, tn);
  AOp ao;
  BOp bo;
  ao.init(x, PlainRows{tm * BM, M}, K);
  bo.init(w, GatedRows{tn * BF, F}, K);
  v16f acc[L::FM][L::FN];
  product_tile<AOp, BOp, BM, BN, S, WY, NW>(lds, ao, bo, K, 0, (K + SK - 1) / SK, acc);
  const int wid = threadIdx.x >> 6;
  block_barrier();  // every wave is done with the last strip
  gated_out<OUT>(lds + wid * kSlab, acc, o, tm * BM + wid / L::WX * (BM / WY), tn * BF + wid % L::WX * (BF / L::WX), M, F,
                 vec, pre_vec);
}

// The same at any address and size (K >= 8, 16 with FP8): 515 x 1365, K = 1023 with pre-activations 22 us.
template <int EB, int BM, int OUT>
__global__ __launch_bounds__(256) void gated_staged_kernel(Operand x, Operand w, GatedOut o, int64_t M, int64_t F,
                                                          int64_t K) {
  constexpr int BF = 64, WY = 2, NW = 4, G = 16 / EB;
  using AOp = StagedRows<BM, NW, 2, PlainRows, G>;
  using BOp = StagedRows<2 * BF, NW, EB, GatedRows, G>;
  constexpr int kSlab = OutSlab<0, 32>::kBytes, kTiles = AOp::kBytes + BOp::kBytes;
  __shared__ __attribute__((aligned(16))) char lds[kTiles > NW * kSlab ? kTiles : NW * kSlab];
  int64_t tm, tn;
  tile_of_block(blockIdx.x, (M + BM - 1) / BM, (F + BF - 1) / BF, tm, tn);
  AOp ao;
  BOp bo;
  ao.init(x, PlainRows{tm * BM, M}, K, 0);
  bo.init(w, GatedRows{tn * BF, F}, K, 0);
  v16f acc[BM / 64][2];
  staged_tile<AOp, BOp, BM, 2 * BF, WY, NW>(lds, ao, bo, 0, (K + kStripK - 1) / kStripK, acc);
  const int wid = threadIdx.x >> 6;
  wait_lds();
  block_barrier();
  gated_out<OUT>(lds + wid * kSlab, acc, o, tm * BM + wid / 2 * (BM / 2), tn * BF + wid % 2 * 32, M, F, false, false);
}

// ---------------------------------------------------------------- gradient of the activation

// Eight columns of a row a thread, at any address; TAIL: F % 8 != 0.  dpre is rounded to bfloat16, half a step of 2^-8 a
// value: it is the operand of the matrix cores in both products behind it, where a form of more pieces would be two or
// three times the work; the gradients are off by 0.0023 of their norm for it, 0.0017 from a float32 dpre.  Bound by HBM: 4096 x 5632 from float32 pre-activations
// 53 us, 6.1 TB/s.
template <int ACT, int DY, int PRE, bool TAIL>
__global__ __launch_bounds__(kThreads) void gated_grad_kernel(const void* __restrict__ dy, const void* __restrict__ pre,
                                                             uint16_t* __restrict__ dpre, int64_t M, int64_t F) {
  const int64_t per = (F + 7) / 8;
  for (int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x; at < M * per; at += int64_t(gridDim.x) * kThreads) {
    const int64_t m = at / per, f = at % per * 8, left = F - f;
    Eight<DY> d8;
    Eight<PRE> g8, u8;
    d8.template load<TAIL>(dy, m * F + f, left);
    g8.template load<TAIL>(pre, m * 2 * F + f, left);
    u8.template load<TAIL>(pre, m * 2 * F + F + f, left);
    float d[8], g[8], u[8];
    d8.get(d);
    g8.get(g);
    u8.get(u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float dg, du;
      gated_grad<ACT>(g[e], u[e], d[e], dg, du);
      g[e] = dg;
      u[e] = du;
    }
    Eight<1> o;
    o.put(g);
    o.template store<TAIL>(dpre, m * 2 * F + f, left);
    o.put(u);
    o.template store<TAIL>(dpre, m * 2 * F + F + f, left);
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
constexpr int64_t kRowsSpan = 2048;  // bytes of a weight row in a stage of gated_rows_kernel

// The large tiles' loads: 16-byte rows at aligned addresses, and a strip of a tile within 32-bit offsets.
bool tiled_rows(const void* p, int64_t row_bytes) {
  return aligned16(p) && row_bytes % 16 == 0 && row_bytes < (int64_t(1) << 23);
}

int64_t rounds(int64_t M, int64_t N, int64_t bm, int64_t bn, int64_t slots) {
  return (((M + bm - 1) / bm) * ((N + bn - 1) / bn) + slots - 1) / slots;
}

// The products' tiles: 256 x 256 has a CU to itself, of the others two blocks share one and cover each
// other's barriers.  Measured per strip of K and round over the card, us (8192 x 4096, K = 8192 and 4096 x 2048, K =
// 11264): 1.7, 1.26 (192 x 128), 1.0 (128 x 128), and 8 more a round.  The one with the least time is taken.
enum ProductTile { kTile256, kTile192, kTile128 };
ProductTile product_tile_of(int64_t M, int64_t N, int64_t strips, int num_cus) {
  const double t256 = rounds(M, N, 256, 256, num_cus) * (8 + 1.7 * strips);
  const double t192 = rounds(M, N, 192, 128, 2 * num_cus) * (8 + 1.26 * strips);
  const double t128 = rounds(M, N, 128, 128, 2 * num_cus) * (8 + 1.0 * strips);
  return t256 <= t192 && t256 <= t128 ? kTile256 : t192 <= t128 ? kTile192 : kTile128;
}

// Parts of K where tiles of 128 x 128 leave more than half of the places for them empty: so many that they are
// full, of 8 strips (512 values) at least.  4096 x 2048 never; 512 x 2048, K = 11264 148 us whole, 41 split.
int product_parts(int64_t M, int64_t N, int64_t K, int num_cus) {
  const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128), strips = (K + kStripK - 1) / kStripK;
  if (tiles * 2 > 2 * num_cus) return 1;
  return int(std::max<int64_t>(1, std::min({int64_t(16), 2 * num_cus / tiles, strips / 8})));
}

// The product of [M, K] and [N, K], either of them stored across k, in the workspace's planes where it is split.
template <bool TA, bool TB>
hipError_t launch_product(const uint16_t* a, const uint16_t* b, void* out, int out_bf16, int64_t M, int64_t N, int64_t K,
                          int num_cus, float* ws, size_t ws_bytes, hipStream_t s) {
  const int64_t lda = TA ? M : K, ldb = TB ? N : K, strips = (K + kStripK - 1) / kStripK;
  const Operand ao{reinterpret_cast<const char*>(a), 2 * lda, TA ? K : M};
  const Operand bo{reinterpret_cast<const char*>(b), 2 * ldb, TB ? K : N};
  if (K < 8 || (TA && M < 8) || (TB && N < 8)) {
    const int64_t blocks = (M + kAnyTile - 1) / kAnyTile * ((N + kAnyTile - 1) / kAnyTile);
    if (blocks > kMaxGrid) return hipErrorInvalidValue;
    return launch(product_any_kernel<TA, TB>, dim3(unsigned(blocks)), dim3(kThreads), 0, s, a, lda, b, ldb, out, out_bf16,
                  M, N, K);
  }
  const bool aligned = tiled_rows(a, 2 * lda) && tiled_rows(b, 2 * ldb);
  auto go = [&](auto bm, auto bn, auto nw, auto type, void* to, int parts) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, NW = decltype(nw)::value, OUT = decltype(type)::value;
    const int64_t blocks = ((M + BM - 1) / BM) * ((N + BN - 1) / BN), per = (strips + parts - 1) / parts;
    if (blocks > kMaxGrid) return hipErrorInvalidValue;
    const dim3 grid{unsigned(blocks), unsigned((strips + per - 1) / per)};  // no part is empty
    if constexpr (BM == 128) {
      if (!aligned) return launch(product_staged_kernel<TA, TB, OUT>, grid, dim3(256), 0, s, ao, bo, to, M, N, K, per);
    }
    constexpr int kLds = 2 * (BM + BN) * 128;
    static std::atomic<uint64_t> lds_set{0};
    constexpr auto kernel = product_kernel<TA, TB, BM, BN, 2, 2, NW, OUT>;
    if (hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), kLds, lds_set)) return e;
    const int vec = aligned16(to) && N * (OUT ? 2 : 4) % 16 == 0;
    return launch(kernel, grid, dim3(64 * NW), kLds, s, ao, bo, to, M, N, K, per, vec);
  };
  const int parts = product_parts(M, N, K, num_cus);
  if (parts > 1 && ws && ws_bytes >= size_t(parts) * M * N * 4) {
    if (hipError_t e = go(Int<128>{}, Int<128>{}, Int<4>{}, Int<0>{}, ws, parts)) return e;
    const int64_t per = (strips + parts - 1) / parts;
    return launch_splitk_reduce(ws, out, out_bf16, M, N, int((strips + per - 1) / per), 1.f, s, Epilogue{});
  }
  auto by_type = [&](auto bm, auto bn, auto nw) {
    return out_bf16 ? go(bm, bn, nw, Int<1>{}, out, 1) : go(bm, bn, nw, Int<0>{}, out, 1);
  };
  switch (aligned ? product_tile_of(M, N, strips, num_cus) : kTile128) {
    case kTile256: return by_type(Int<256>{}, Int<256>{}, Int<8>{});
    case kTile192: return by_type(Int<192>{}, Int<128>{}, Int<4>{});
    default: return by_type(Int<128>{}, Int<128>{}, Int<4>{});
  }
}

}  // namespace

hipError_t launch_gated_gemm(const void* w, int fp8, const uint16_t* x, const GatedOut& o, int64_t M, int64_t F, int64_t K,
                             int num_cus, hipStream_t s) {
  const int eb = fp8 ? 1 : 2;
  // Few rows.  F = 14336, K = 4096, us (vector ALU, stages in LDS, tiles of 64 rows): FP8 M = 1 19, 22, -; M = 2
  // 22, 22, -; M = 4 38, 22, -; M = 13 -, 25, 31; bfloat16 M = 2 37, 41, -; M = 4 48, 41, -; M = 13 -, 43, 48.
  const bool in_stages = K * eb <= (fp8 ? 4 : 8) * kRowsSpan && aligned16(x) && aligned16(w) && K * eb % 16 == 0 &&
                         K % 8 == 0 && 2 * F * K * eb < kNowhere;
  if (M <= 2 || (M <= 4 && !in_stages)) {
    const int64_t blocks = (F + 3) / 4;
    if (blocks > kMaxGrid) return hipErrorInvalidValue;
    auto go = [&](auto kernel) {
      return launch(kernel, dim3(unsigned(blocks)), dim3(256), 0, s, static_cast<const char*>(w), x, o, F, K);
    };
    if (fp8)
      return M == 1   ? go(gated_gemv_kernel<1, 1, 4>)
             : M == 2 ? go(gated_gemv_kernel<1, 2, 2>)
             : M == 3 ? go(gated_gemv_kernel<1, 3, 2>)
                      : go(gated_gemv_kernel<1, 4, 2>);
    return M == 1   ? go(gated_gemv_kernel<2, 1, 4>)
           : M == 2 ? go(gated_gemv_kernel<2, 2, 4>)
           : M == 3 ? go(gated_gemv_kernel<2, 3, 2>)
                    : go(gated_gemv_kernel<2, 4, 2>);
  }
  if (M <= 16 && in_stages) {
    // Two blocks a CU with two stages each cover each other's barriers and ends, one with four has as many bytes on their
    // way.  Two pay where a block has few tiles or a row few stages, us, M = 13 (two stages, four): K = 1024, F = 14336 FP8
    // 11.7, 14.6, bfloat16 13.0, 15.5; K = 2048, F = 5504 8.9, 9.9 and 11.2, 12.6, with addends 9.3, 10.7 and 11.7, 14.0;
    // K = 4096, F = 14336 25.3 and 43 either way, with addends 31.8, 29.7 and 48.7, 45.8.  K = 8192 in bfloat16, F = 8192:
    // 55.9, 50.2.
    auto go = [&](auto bytes, auto parts, auto stages) {
      constexpr int EB = decltype(bytes)::value, KS = decltype(parts)::value, S = decltype(stages)::value;
      constexpr int kLds = S * 16 * kRowsSpan + 8 * kWave * 16;
      const int64_t blocks = std::min<int64_t>((F + 7) / 8, (S == 2 ? 2 : 1) * num_cus);
      const char* const wp = static_cast<const char*>(w);
      return o.addend ? launch_big_lds<gated_rows_kernel<EB, KS, S, true>>(kLds + kAddBytes, blocks, 512, s, wp, x, o, int(M), F, K)
                      : launch_big_lds<gated_rows_kernel<EB, KS, S, false>>(kLds, blocks, 512, s, wp, x, o, int(M), F, K);
    };
    auto by_parts = [&](auto bytes) {
      if (K * eb <= kRowsSpan) return go(bytes, Int<1>{}, Int<2>{});
      if (K * eb <= 2 * kRowsSpan) return go(bytes, Int<2>{}, Int<2>{});
      if (K * eb <= 4 * kRowsSpan) return go(bytes, Int<4>{}, Int<2>{});
      return go(Int<2>{}, Int<8>{}, Int<4>{});
    };
    return fp8 ? by_parts(Int<1>{}) : by_parts(Int<2>{});
  }
  const Operand xo{reinterpret_cast<const char*>(x), 2 * K, M}, wo{static_cast<const char*>(w), K * eb, 2 * F};
  if (tiled_rows(x, K * 2) && tiled_rows(w, K * eb) && 2 * F * K * eb < kNowhere) {
    const int vec = aligned16(o.out) && F * (o.out_bf16 ? 2 : 4) % 16 == 0;
    const int pre_vec = aligned16(o.pre) && F * (o.pre_bf16 ? 2 : 4) % 16 == 0;
    auto go = [&](auto bytes, auto bm, auto bf, auto strip, auto stages, auto nw, auto nt, auto out) {
      constexpr int EB = decltype(bytes)::value, BM = decltype(bm)::value, BF = decltype(bf)::value;
      constexpr int SK = decltype(strip)::value, S = decltype(stages)::value, NW = decltype(nw)::value;
      constexpr int OUT = decltype(out)::value;
      constexpr bool NT = decltype(nt)::value;
      using L = ProductLayout<RowsOperand<BM, NW, 2, PlainRows, SK>, RowsOperand<2 * BF, NW, EB, GatedRows, SK>, BM, 2 * BF, S,
                              2, NW>;
      const int64_t blocks = ((M + BM - 1) / BM) * ((F + BF - 1) / BF);
      if (blocks > kMaxGrid) return hipErrorInvalidValue;
      return launch_big_lds<gated_kernel<EB, BM, BF, SK, S, NW, NT, OUT>>(L::kLds, blocks, 64 * NW, s, xo, wo, o, M, F, K, vec,
                                                                     pre_vec);
    };
    // To 128 rows one tile has them all and the weights are read once, past the caches where a strip's rows are whole
    // 128-byte lines (F = 14336, K = 4096, M = 64: bfloat16 48 us, 54 through them), as many bytes of them on their way as
    // LDS holds.  32 columns where tiles of 64 leave half the CUs idle (F = 5504, K = 2048, M = 64: 16 us, 17 FP8 and 20
    // bfloat16 with 64; F = 14336 40 us FP8, 32 with 64).  Strips of 128: FP8 M = 64 32 us, 34 in strips of 64; M =
    // 128 46, 48.
    const bool narrow = 2 * ((F + 63) / 64) <= num_cus;
    // Beyond, tiles of 256 x 128 columns with a CU to themselves, or of 128 x 64 of which two blocks share one, by
    // the time of
    // their rounds as for the products above: M = 256, F = 14336, K = 4096 FP8 107 and 67 us, bfloat16 116 and 85; M = 500
    // 112 and 126, 115 and 148.
    const bool wide = 1.75 * rounds(M, F, 256, 128, num_cus) <= 1.05 * rounds(M, F, 128, 64, 2 * num_cus);
    auto by_tile = [&](auto bytes, auto out) {
      constexpr bool kFp8 = decltype(bytes)::value == 1;
      if (M <= 64 && narrow) return go(bytes, Int<64>{}, Int<32>{}, Int<64>{}, Int<4>{}, Int<2>{}, Int<!kFp8>{}, out);
      if (M <= 64) return go(bytes, Int<64>{}, Int<64>{}, Int<128>{}, Int<3>{}, Int<4>{}, Int<1>{}, out);
      if (M <= 128) return go(bytes, Int<128>{}, Int<64>{}, Int<kFp8 ? 128 : 64>{}, Int<kFp8 ? 3 : 4>{}, Int<4>{}, Int<1>{}, out);
      if (wide) return go(bytes, Int<256>{}, Int<128>{}, Int<64>{}, Int<2>{}, Int<8>{}, Int<0>{}, out);
      return go(bytes, Int<128>{}, Int<64>{}, Int<64>{}, Int<2>{}, Int<4>{}, Int<0>{}, out);
    };
    auto by_out = [&](auto bytes) { return o.out_bf16 ? by_tile(bytes, Int<1>{}) : by_tile(bytes, Int<0>{}); };
    return fp8 ? by_out(Int<1>{}) : by_out(Int<2>{});
  }
  if (K >= 16 / eb) {
    // 64 rows a tile also where tiles of 128 leave CUs idle (515 x 1365, K = 1023, a call among others: 17 us, 23 with 128).
    const int64_t bm = M <= 64 || (M + 127) / 128 * ((F + 63) / 64) <= num_cus ? 64 : 128;
    const int64_t blocks = (M + bm - 1) / bm * ((F + 63) / 64);
    if (blocks > kMaxGrid) return hipErrorInvalidValue;
    auto go = [&](auto kernel) { return launch(kernel, dim3(unsigned(blocks)), dim3(256), 0, s, xo, wo, o, M, F, K); };
    auto by_out = [&](auto bytes, auto rows) {
      constexpr int EB = decltype(bytes)::value, BM = decltype(rows)::value;
      return o.out_bf16 ? go(gated_staged_kernel<EB, BM, 1>) : go(gated_staged_kernel<EB, BM, 0>);
    };
    auto by_rows = [&](auto bytes) { return bm == 64 ? by_out(bytes, Int<64>{}) : by_out(bytes, Int<128>{}); };
    return fp8 ? by_rows(Int<1>{}) : by_rows(Int<2>{});
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
  const int64_t blocks = (M * ((F + 7) / 8) + kThreads - 1) / kThreads;
  return by_act(act, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    auto go = [&](auto kernel) {
      return launch(kernel, dim3(unsigned(blocks < 65536 ? blocks : 65536)), dim3(kThreads), 0, s, dy, pre, dpre, M, F);
    };
    auto by_tail = [&](auto tail) {
      constexpr bool TAIL = decltype(tail)::value;
      if (dy_bf16) return pre_bf16 ? go(gated_grad_kernel<ACT, 1, 1, TAIL>) : go(gated_grad_kernel<ACT, 1, 0, TAIL>);
      return pre_bf16 ? go(gated_grad_kernel<ACT, 0, 1, TAIL>) : go(gated_grad_kernel<ACT, 0, 0, TAIL>);
    };
    return F % 8 ? by_tail(std::true_type{}) : by_tail(std::false_type{});
  });
}

// Bytes of workspace that the product of [M, K] and [N, K] takes, 0: none.
size_t bf16_product_ws_bytes(int64_t M, int64_t N, int64_t K, int num_cus) {
  const int parts = product_parts(M, N, K, num_cus);
  return parts > 1 ? size_t(parts) * M * N * 4 : 0;
}

// dx[m, k] = sum_n dout[m, n] w[n, k]
hipError_t launch_bf16_grad_x(const uint16_t* dout, const uint16_t* w, void* dx, int dx_bf16, int64_t M, int64_t N,
                              int64_t K, int num_cus, float* ws, size_t ws_bytes, hipStream_t s) {
  return launch_product<false, true>(dout, w, dx, dx_bf16, M, K, N, num_cus, ws, ws_bytes, s);
}

// dw[n, k] = sum_m dout[m, n] x[m, k]
hipError_t launch_bf16_grad_w(const uint16_t* dout, const uint16_t* x, void* dw, int dw_bf16, int64_t M, int64_t N,
                              int64_t K, int num_cus, float* ws, size_t ws_bytes, hipStream_t s) {
  return launch_product<true, true>(dout, x, dw, dw_bf16, N, K, M, num_cus, ws, ws_bytes, s);
}

}  // namespace qlinear
