// Low-rank adapters of many requests beside a shared projection, and their gradients.  Rows
// b .. e - 1 of group z (offsets z, z + 1) have adapter l = ids[z], A [R, K] and B [N, R]:
//   z   = x A^T                     (float32, unscaled)
//   out = base + s z B^T
// and with the gradient dout of out
//   dz  = dout B,   dx = dx0 + s dz A,   dA = s sum_t dz x^T,   dB = s sum_t dout z^T.
// R is 4 to 256 against thousands of K and N, so all of it is bound by the rows x, base, out,
// dout and dx, and with few rows by the adapters themselves.  Two kernels carry it: the one
// contracts a long axis to R values a row (z; dz with B transposed), the other takes R
// values back to a long axis (out; dx with A transposed); the third sums over rows (dA, dB).
//
// What has R values a row stays float32 in memory.  The matrix cores take it as bfloat16 pieces
// side by side along the contraction: three for float32 results (24 bits, exact), two for bfloat16
// ones (16 bits, against the result's 8), P R values of k instead of R in a product that is
// small beside the bytes.
//
// MFMA 16x16x32: lane l holds k = 8 (l / 16) .. + 7 of row l % 16 of both operands, and of the
// result column l % 16, rows 4 (l / 16) .. + 3.
#include <algorithm>

#include "device.hpp"
#include "elem.hpp"
#include "launch.hpp"

namespace qlinear {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;

// v as the sum of P bfloat16 pieces, each what is left rounded.  A first piece that rounding would
// take out of bfloat16's range is cut instead; an infinity or NaN has no further pieces.
template <int P>
__device__ __forceinline__ void split_bf16(float v, __bf16 (&piece)[P]) {
  const uint32_t u = __float_as_uint(v);
  const bool finite = (u & 0x7F800000u) != 0x7F800000u;
  float h = float(static_cast<__bf16>(v));
  if (finite && (__float_as_uint(h) & 0x7F800000u) == 0x7F800000u) h = __uint_as_float(u & 0xFFFF0000u);
  piece[0] = static_cast<__bf16>(h);
  float left = finite ? v - h : 0.f;
#pragma unroll
  for (int p = 1; p < P; ++p) {
    piece[p] = static_cast<__bf16>(left);
    left -= float(piece[p]);
  }
}
constexpr int pieces_of(bool bf16) { return bf16 ? 2 : 3; }

// Eight bfloat16 at p; `left` of them exist (VEC: 16-byte aligned, and all or none do).
template <bool VEC>
__device__ __forceinline__ v8bf load_k8(const uint16_t* p, int64_t left) {
  u32x4 v{0, 0, 0, 0};
  if constexpr (VEC) {
    if (left > 0) v = ld16(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) v[e / 2] |= uint32_t(p[e]) << (16 * (e % 2));
  }
  return __builtin_bit_cast(v8bf, v);
}

// The groups of rows of a call.
struct Groups {
  const uint32_t* offsets;
  const int32_t* ids;
  int64_t G, L, T;
};

// Tile `tile` of the BM-row tiles of all groups: its first row, how many it has (0: there is no
// such tile) and its adapter (-1: none).  cum: LDS of G + 1.  Meets one barrier.
template <int BM>
__device__ __forceinline__ int find_tile(const Groups& g, int* cum, int tile, int64_t* row0, int* adapter) {
  if (threadIdx.x < kWave) count_group_tiles<BM>(cum, g.offsets, g.G, g.T);
  __syncthreads();
  if (tile >= cum[g.G]) return 0;
  int lo = 0, hi = int(g.G);  // cum[lo] <= tile < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cum[mid] <= tile) lo = mid;
    else hi = mid;
  }
  const int64_t begin = int64_t(g.offsets[lo]) + int64_t(tile - cum[lo]) * BM;
  const int64_t end = int64_t(g.offsets[lo + 1]) < g.T ? int64_t(g.offsets[lo + 1]) : g.T;
  const int id = g.ids[lo];
  *adapter = id >= 0 && id < g.L ? id : -1;
  *row0 = begin;
  return int(end - begin < BM ? end - begin : BM);
}

// ---------------------------------------------------------------- long axis -> R

// plane[split][t][r] = sum over the split's part of K of x[t, k] a[l, r, k].  Block: a tile of
// BM rows, a part of K, 16 FR of the R; its waves take 128 values of k in turn and add up at
// the end through LDS.  Both operands come straight from memory: neither is used by two waves.
template <int BM, int FR, bool VEC>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(const uint16_t* __restrict__ x,
                                                              const uint16_t* __restrict__ a, Groups g,
                                                              float* __restrict__ plane, int64_t K, int64_t R,
                                                              int64_t per) {
  extern __shared__ int cum[];
  __shared__ v4f sums[kWaves][FR][kWave];
  constexpr int FM = BM / 16, KS = 4;  // KS MFMA steps of 32 at a time
  int64_t row0 = 0;
  int id = -1;
  const int rows = find_tile<BM>(g, cum, int(blockIdx.x), &row0, &id);
  if (rows <= 0) return;
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const int64_t r0 = int64_t(blockIdx.z) * 16 * FR;
  plane += int64_t(blockIdx.y) * g.T * R;
  const int64_t begin = int64_t(blockIdx.y) * per, end = begin + per < K ? begin + per : K;

  v4f acc[FM][FR];
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[m][f] = v4f{};
  if (id >= 0) {
    const uint16_t* ap = a + (int64_t(id) * R + r0) * K;
    for (int64_t k0 = begin + 32 * KS * wid; k0 < end; k0 += 32 * KS * kWaves) {
      v8bf xf[FM][KS], af[FR][KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int64_t k = k0 + 32 * s + 8 * q;
#pragma unroll
        for (int m = 0; m < FM; ++m)
          xf[m][s] = load_k8<VEC>(x + (row0 + 16 * m + i) * K + k, 16 * m + i < rows ? end - k : 0);
#pragma unroll
        for (int f = 0; f < FR; ++f)
          af[f][s] = load_k8<VEC>(ap + int64_t(16 * f + i) * K + k, r0 + 16 * f + i < R ? end - k : 0);
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int f = 0; f < FR; ++f)
            acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[f][s], xf[m][s], acc[m][f], 0, 0, 0);
    }
  }
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    if (16 * m >= rows) break;
#pragma unroll
    for (int f = 0; f < FR; ++f) sums[wid][f][lane] = acc[m][f];
    __syncthreads();
    for (int f = wid; f < FR; f += kWaves) {
      v4f v = sums[0][f][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += sums[w][f][lane];
      const int64_t r = r0 + 16 * f + 4 * q;
      if (16 * m + i < rows) {
        float* out = plane + (row0 + 16 * m + i) * R + r;
        if (R % 4 == 0) {
          if (r < R) *reinterpret_cast<v4f*>(out) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (r + e < R) out[e] = v[e];
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- R -> long axis

// out[t, n] = base[t, n] + s sum_r z[t, r] b[l, n, r], z the sum of `splits` planes, written to
// z_out where that is given.  Block: a tile of BM rows, kSpan columns; a wave takes 64 columns
// at a time, as four MFMA tiles whose rows are permuted so that a lane's two results of a pair
// are eight consecutive columns: one 16-byte store of bfloat16.  LDS: the pieces of z.
constexpr int kSpan = 1024;

template <int BM, int OUT, bool VEC, bool OVEC>
__global__ __launch_bounds__(kThreads) void lora_expand_kernel(const float* __restrict__ plane, int splits,
                                                              const uint16_t* __restrict__ b, Groups g,
                                                              const float* __restrict__ scale,
                                                              const void* base, void* out,
                                                              float* __restrict__ z_out, int64_t N, int64_t R,
                                                              int64_t span) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using E = Elem<OUT>;
  using V = typename E::T;
  constexpr int FM = BM / 16, P = pieces_of(OUT);
  const int R8 = int((R + 7) / 8), row_bytes = 16 * P * R8 + 16;
  char* const zs = lds;                                   // [BM][P R8 eights + 1 of padding]
  int* const cum = reinterpret_cast<int*>(lds + BM * row_bytes);
  int64_t row0 = 0;
  int id = -1;
  const int rows = find_tile<BM>(g, cum, int(blockIdx.x), &row0, &id);
  if (rows <= 0) return;
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const float s = id >= 0 && scale ? scale[id] : 1.f;

  if (id >= 0 || z_out) {
    for (int p = threadIdx.x; p < BM * R8; p += kThreads) {
      const int row = p / R8, c = p % R8;
      v8bf eight[P];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = 0.f;
        if (row < rows && 8 * c + e < R) {
          const int64_t at = (row0 + row) * R + 8 * c + e;
          for (int n = 0; n < splits; ++n) v += plane[n * g.T * R + at];
          if (z_out && blockIdx.y == 0) z_out[at] = v;
        }
        __bf16 piece[P];
        split_bf16<P>(v * s, piece);
#pragma unroll
        for (int n = 0; n < P; ++n) eight[n][e] = piece[n];
      }
#pragma unroll
      for (int n = 0; n < P; ++n) *reinterpret_cast<v8bf*>(zs + row * row_bytes + 16 * (n * R8 + c)) = eight[n];
    }
    __syncthreads();
  }

  const int steps = (P * R8 + 3) / 4;
  const int64_t first = int64_t(blockIdx.y) * span, last = first + span < N ? first + span : N;
  for (int64_t n0 = first + 64 * wid; n0 < last; n0 += 64 * kWaves) {
    v4f acc[FM][2][2];
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int p = 0; p < 2; ++p) acc[m][p][0] = acc[m][p][1] = v4f{};
    if (id >= 0)
      for (int t = 0; t < steps; ++t) {
        const int c = 4 * t + q, cc = c < R8 ? c : c < 2 * R8 ? c - R8 : c - 2 * R8;
        v8bf bf[2][2], zf[FM];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int64_t n = n0 + 32 * p + 8 * (i / 4) + 4 * f + i % 4;
            bf[p][f] = load_k8<VEC>(b + (int64_t(id) * N + n) * R + 8 * cc, n < N && c < P * R8 ? R - 8 * cc : 0);
          }
#pragma unroll
        for (int m = 0; m < FM; ++m)
          zf[m] = c < P * R8 ? *reinterpret_cast<const v8bf*>(zs + (16 * m + i) * row_bytes + 16 * c) : v8bf{};
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int f = 0; f < 2; ++f)
              acc[m][p][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[p][f], zf[m], acc[m][p][f], 0, 0, 0);
      }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      if (16 * m + i >= rows) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int64_t n = n0 + 32 * p + 8 * q, at = (row0 + 16 * m + i) * N + n;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[m][p][e / 4][e % 4];
        const V* bp = reinterpret_cast<const V*>(base) + at;
        V* op = reinterpret_cast<V*>(out) + at;
        if constexpr (OVEC) {
          if (n >= N) continue;
          constexpr int W = E::kPer16;
#pragma unroll
          for (int h = 0; h < 8; h += W) {
            float o[W];
#pragma unroll
            for (int e = 0; e < W; ++e) o[e] = v[h + e];
            if (base) {
              float add[W];
              E::unpack(ld16(bp + h), add);
#pragma unroll
              for (int e = 0; e < W; ++e) o[e] += add[e];
            }
            *reinterpret_cast<u32x4*>(op + h) = E::pack(o);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) op[e] = E::put(v[e] + (base ? E::get(bp[e]) : 0.f));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- sums over rows

// DA: out[l, r, c] = s sum_t z[t, r] p[t, c] (dA: z = dz, p = x);
// else out[l, c, r] (dB: z, p = dout), over the rows of adapter l's groups.  Block: one
// adapter, 16 FR of the R, 512 columns (128 a wave), every splits-th step of 32 rows.  A lane loads 8
// rows x 8 columns and turns them by byte permutations into its pieces of eight MFMA
// operands, whose row i is column 8 i + j of the wave's 128.
template <bool DA, int FR, int P, bool VEC>
__global__ __launch_bounds__(kThreads) void lora_sum_kernel(const uint16_t* __restrict__ p,
                                                           const float* __restrict__ z, Groups g,
                                                           const float* __restrict__ scale, void* __restrict__ out,
                                                           int out_bf16, int64_t C, int64_t R, int r_blocks, int splits) {
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const int64_t l = blockIdx.y / r_blocks, r0 = int64_t(blockIdx.y % r_blocks) * 16 * FR;
  const int64_t c0 = int64_t(blockIdx.x) * 512 + 128 * wid;
  if (c0 >= C) return;
  const float s = scale ? scale[l] : 1.f;
  v4f acc[8][FR];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[j][f] = v4f{};

  int turn = int(blockIdx.z);  // steps to skip until this block's next one
  for (int64_t z0 = 0; z0 < g.G; z0 += kWave) {
    int64_t b = 0, e = 0;
    bool mine = false;
    if (z0 + lane < g.G) {
      b = g.offsets[z0 + lane];
      e = g.offsets[z0 + lane + 1];
      e = e < g.T ? e : g.T;
      mine = g.ids[z0 + lane] == l && b < e;
    }
    for (uint64_t left = __ballot(mine); left; left &= left - 1) {
      const int src = __builtin_ctzll(left);
      const int64_t begin = __builtin_amdgcn_readlane(int(b), src), end = __builtin_amdgcn_readlane(int(e), src);
      const int64_t steps = (end - begin + 31) / 32;
      int64_t n = turn;
      for (; n < steps; n += splits) {
        const int64_t t0 = begin + 32 * n + 8 * q;
        u32x4 row[8];
        float zv[FR][8];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const int64_t t = t0 + d, c = c0 + 8 * i;
          row[d] = __builtin_bit_cast(u32x4, load_k8<VEC>(p + t * C + c, t < end ? C - c : 0));
#pragma unroll
          for (int f = 0; f < FR; ++f) {
            const int64_t r = r0 + 16 * f + i;
            zv[f][d] = t < end && r < R ? z[t * R + r] * s : 0.f;
          }
        }
        v8bf zf[FR][P];
#pragma unroll
        for (int f = 0; f < FR; ++f)
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            __bf16 piece[P];
            split_bf16<P>(zv[f][d], piece);
#pragma unroll
            for (int w = 0; w < P; ++w) zf[f][w][d] = piece[w];
          }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u32x4 w;
#pragma unroll
          for (int d = 0; d < 4; ++d)
            w[d] = __builtin_amdgcn_perm(row[2 * d + 1][j / 2], row[2 * d][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
          const v8bf pf = __builtin_bit_cast(v8bf, w);
#pragma unroll
          for (int f = 0; f < FR; ++f)
#pragma unroll
            for (int o = 0; o < P; ++o) {
              if constexpr (DA) acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(zf[f][o], pf, acc[j][f], 0, 0, 0);
              else acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf, zf[f][o], acc[j][f], 0, 0, 0);
            }
        }
      }
      turn = int(n - steps);
    }
  }

  const int64_t size = g.L * C * R;
  auto put = [&](int64_t at, float v) {
    if (out_bf16) reinterpret_cast<uint16_t*>(out)[at] = Elem<1>::put(v);
    else reinterpret_cast<float*>(out)[blockIdx.z * size + at] = v;
  };
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t r = r0 + 16 * f + (DA ? 4 * q + e : i), c = c0 + 8 * (DA ? i : 4 * q + e) + j;
        if (r < R && c < C) put((l * (DA ? R : C) + (DA ? r : c)) * (DA ? C : R) + (DA ? c : r), acc[j][f][e]);
      }
}

// out[n] = the sum of the planes' values n, in their order.
__global__ __launch_bounds__(kThreads) void lora_join_kernel(const float* __restrict__ plane, int splits,
                                                             void* __restrict__ out, int out_bf16, int64_t count) {
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (at >= count) return;
  float v = 0.f;
  for (int n = 0; n < splits; ++n) v += plane[n * count + at];
  if (out_bf16) reinterpret_cast<uint16_t*>(out)[at] = Elem<1>::put(v);
  else reinterpret_cast<float*>(out)[at] = v;
}

__global__ __launch_bounds__(kThreads) void clear_kernel(uint16_t* __restrict__ p, int64_t count) {
  const int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (at < count) p[at] = 0;
}

// out[l, c, r] = in[l, r, c], in pieces of 32 x 32 through LDS.
__global__ __launch_bounds__(kThreads) void lora_turn_kernel(const uint16_t* __restrict__ in,
                                                             uint16_t* __restrict__ out, int64_t rows, int64_t cols) {
  __shared__ uint16_t tile[32][33];
  const int64_t l = blockIdx.z, r0 = int64_t(blockIdx.y) * 32, c0 = int64_t(blockIdx.x) * 32;
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
#pragma unroll
  for (int n = 0; n < 32; n += 8)
    if (r0 + ty + n < rows && c0 + tx < cols) tile[ty + n][tx] = in[(l * rows + r0 + ty + n) * cols + c0 + tx];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < 32; n += 8)
    if (c0 + ty + n < cols && r0 + tx < rows) out[(l * cols + c0 + ty + n) * rows + r0 + tx] = tile[tx][ty + n];
}

// ---------------------------------------------------------------- launches

bool vec16(const void* p, int64_t row) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % 8 == 0; }

// Rows of a tile: 64 where a group has more than 16 on average.
bool tall(int64_t T, int64_t G) { return T > 16 * G; }

int64_t tile_count(int64_t T, int64_t G, int bm) { return std::min(T, T / bm + G); }

// Parts of the long axis: as many as fill the card twice (512 blocks), of 512 values at least.
int shrink_splits(int64_t T, int64_t G, int64_t K, int64_t R) {
  const int64_t tiles = tile_count(T, G, tall(T, G) ? 64 : 16) * ((R + 63) / 64);
  return int(std::max<int64_t>(1, std::min({int64_t(16), (512 + tiles - 1) / tiles, K / 512})));
}

hipError_t launch_shrink(const uint16_t* x, const uint16_t* a, const Groups& g, float* plane, int splits, int64_t K,
                         int64_t R, hipStream_t s) {
  const int64_t per = (((K + splits - 1) / splits + 127) / 128) * 128;
  const bool vec = vec16(x, K) && vec16(a, K);
  const size_t lds = size_t(g.G + 1) * 4;
  auto go = [&](auto kernel, int bm, int fr) {
    const dim3 grid(unsigned(tile_count(g.T, g.G, bm)), unsigned(splits), unsigned((R + 16 * fr - 1) / (16 * fr)));
    return launch(kernel, grid, dim3(kThreads), lds, s, x, a, g, plane, K, R, per);
  };
  auto by_rank = [&](auto bm, auto v) {
    constexpr int BM = decltype(bm)::value;
    constexpr bool VEC = decltype(v)::value;
    if (R <= 16) return go(lora_shrink_kernel<BM, 1, VEC>, BM, 1);
    if (R <= 32) return go(lora_shrink_kernel<BM, 2, VEC>, BM, 2);
    return go(lora_shrink_kernel<BM, 4, VEC>, BM, 4);
  };
  auto by_rows = [&](auto v) {
    if (tall(g.T, g.G)) return by_rank(std::integral_constant<int, 64>{}, v);
    return by_rank(std::integral_constant<int, 16>{}, v);
  };
  return vec ? by_rows(std::true_type{}) : by_rows(std::false_type{});
}

hipError_t launch_expand(const float* plane, int splits, const uint16_t* b, const Groups& g, const float* scale,
                         const void* base, void* out, int out_bf16, float* z_out, int64_t N, int64_t R, hipStream_t s) {
  const bool vec = vec16(b, R), ovec = vec16(base, N) && vec16(out, N);
  const int bm = tall(g.T, g.G) && R <= 64 ? 64 : 16;  // LDS: 64 rows of R = 64 are 25 KiB, and 16 KiB of groups
  const int64_t tiles = tile_count(g.T, g.G, bm);
  const int64_t span = tiles * ((N + kSpan - 1) / kSpan) >= 1024 ? kSpan : 256;
  const dim3 grid(unsigned(tiles), unsigned((N + span - 1) / span));
  const size_t lds = size_t(bm) * (16 * pieces_of(out_bf16) * ((R + 7) / 8) + 16) + size_t(g.G + 1) * 4;
  auto go = [&](auto kernel) {
    return launch(kernel, grid, dim3(kThreads), lds, s, plane, splits, b, g, scale, base, out, z_out, N, R, span);
  };
  auto by_rows = [&](auto o, auto v, auto w) {
    constexpr int OUT = decltype(o)::value;
    constexpr bool VEC = decltype(v)::value, OVEC = decltype(w)::value;
    if (bm == 64) return go(lora_expand_kernel<64, OUT, VEC, OVEC>);
    return go(lora_expand_kernel<16, OUT, VEC, OVEC>);
  };
  auto by_out = [&](auto v, auto w) {
    if (out_bf16) return by_rows(std::integral_constant<int, 1>{}, v, w);
    return by_rows(std::integral_constant<int, 0>{}, v, w);
  };
  if (vec) return ovec ? by_out(std::true_type{}, std::true_type{}) : by_out(std::true_type{}, std::false_type{});
  return ovec ? by_out(std::false_type{}, std::true_type{}) : by_out(std::false_type{}, std::false_type{});
}

// Blocks that share an adapter's rows: 512 blocks, and 128 rows for each on average.
int sum_splits(int64_t T, int64_t L, int64_t C, int64_t R) {
  const int64_t blocks = ((C + 511) / 512) * L * ((R + 63) / 64);
  return int(std::max<int64_t>(1, std::min({int64_t(16), 512 / blocks, T / (128 * L)})));
}

hipError_t launch_sum(bool da, const uint16_t* p, const float* z, const Groups& g, const float* scale, void* out,
                      int out_bf16, int64_t C, int64_t R, float* parts, hipStream_t s) {
  const int splits = sum_splits(g.T, g.L, C, R);
  const int fr = R <= 16 ? 1 : R <= 32 ? 2 : 4, r_blocks = int((R + 16 * fr - 1) / (16 * fr));
  const bool vec = vec16(p, C);
  void* const to = splits > 1 ? parts : out;
  const int to_bf16 = splits > 1 ? 0 : out_bf16;
  const dim3 grid(unsigned((C + 511) / 512), unsigned(g.L * r_blocks), unsigned(splits));
  auto go = [&](auto kernel) {
    return launch(kernel, grid, dim3(kThreads), 0, s, p, z, g, scale, to, to_bf16, C, R, r_blocks, splits);
  };
  auto by_rank = [&](auto d, auto v, auto n) {
    constexpr bool DA = decltype(d)::value, VEC = decltype(v)::value;
    constexpr int P = decltype(n)::value;
    if (fr == 1) return go(lora_sum_kernel<DA, 1, P, VEC>);
    if (fr == 2) return go(lora_sum_kernel<DA, 2, P, VEC>);
    return go(lora_sum_kernel<DA, 4, P, VEC>);
  };
  auto by_type = [&](auto d, auto v) {
    return out_bf16 ? by_rank(d, v, std::integral_constant<int, 2>{}) : by_rank(d, v, std::integral_constant<int, 3>{});
  };
  auto by_vec = [&](auto d) { return vec ? by_type(d, std::true_type{}) : by_type(d, std::false_type{}); };
  const hipError_t e = da ? by_vec(std::true_type{}) : by_vec(std::false_type{});
  if (e != hipSuccess || splits == 1) return e;
  const int64_t count = g.L * C * R;
  return launch(lora_join_kernel, dim3(unsigned((count + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, parts, splits,
                out, out_bf16, count);
}

hipError_t launch_turn(const uint16_t* in, uint16_t* out, int64_t L, int64_t rows, int64_t cols, hipStream_t s) {
  return launch(lora_turn_kernel, dim3(unsigned((cols + 31) / 32), unsigned((rows + 31) / 32), unsigned(L)),
                dim3(kThreads), 0, s, in, out, rows, cols);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// The workspace of the backward pass, in this order.
struct GradSpace {
  size_t dz, planes, turned_a, turned_b, parts, total;
  GradSpace(int64_t T, int64_t G, int64_t L, int64_t N, int64_t K, int64_t R) {
    const size_t row = size_t(T) * R * 4;
    dz = 0;
    planes = up16(dz + row);
    turned_a = up16(planes + row * shrink_splits(T, G, N, R));
    turned_b = up16(turned_a + size_t(L) * R * K * 2);
    parts = up16(turned_b + size_t(L) * R * N * 2);
    const int sa = sum_splits(T, L, K, R), sb = sum_splits(T, L, N, R);
    total = parts + std::max(sa > 1 ? size_t(sa) * L * K * R * 4 : 0, sb > 1 ? size_t(sb) * L * N * R * 4 : 0);
  }
};

}  // namespace

hipError_t launch_clear(void* p, int64_t bytes, hipStream_t s) {
  const int64_t count = bytes / 2;
  if (count == 0) return hipSuccess;
  return launch(clear_kernel, dim3(unsigned((count + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                static_cast<uint16_t*>(p), count);
}

size_t lora_ws_bytes(int64_t T, int64_t G, int64_t K, int64_t R) {
  return T > 0 ? size_t(shrink_splits(T, G, K, R)) * T * R * 4 : 0;
}

size_t lora_grad_ws_bytes(int64_t T, int64_t G, int64_t L, int64_t N, int64_t K, int64_t R) {
  return T > 0 ? GradSpace(T, G, L, N, K, R).total : 0;
}

hipError_t launch_lora(const uint16_t* x, const uint16_t* a, const uint16_t* b, const uint32_t* offsets,
                       const int32_t* ids, const float* scale, const void* base, void* out, int out_bf16, float* z,
                       int64_t G, int64_t L, int64_t T, int64_t N, int64_t K, int64_t R, float* ws, hipStream_t s) {
  const Groups g{offsets, ids, G, L, T};
  const int splits = shrink_splits(T, G, K, R);
  float* const plane = splits == 1 && z ? z : ws;
  if (hipError_t e = launch_shrink(x, a, g, plane, splits, K, R, s)) return e;
  return launch_expand(plane, splits, b, g, scale, base, out, out_bf16, plane == z ? nullptr : z, N, R, s);
}

hipError_t launch_lora_grad(const uint16_t* dout, const uint16_t* x, const float* z, const uint16_t* a, const uint16_t* b,
                            const uint32_t* offsets, const int32_t* ids, const float* scale, const void* base, void* dx,
                            int dx_bf16, void* da, void* db, int grad_bf16, int64_t G, int64_t L, int64_t T, int64_t N,
                            int64_t K, int64_t R, char* ws, hipStream_t s) {
  const Groups g{offsets, ids, G, L, T};
  const GradSpace at(T, G, L, N, K, R);
  uint16_t *ta = reinterpret_cast<uint16_t*>(ws + at.turned_a), *tb = reinterpret_cast<uint16_t*>(ws + at.turned_b);
  float *dz = reinterpret_cast<float*>(ws + at.dz), *planes = reinterpret_cast<float*>(ws + at.planes);
  float* parts = reinterpret_cast<float*>(ws + at.parts);
  const int splits = shrink_splits(T, G, N, R);
  if (hipError_t e = launch_turn(a, ta, L, R, K, s)) return e;
  if (hipError_t e = launch_turn(b, tb, L, N, R, s)) return e;
  if (hipError_t e = launch_shrink(dout, tb, g, planes, splits, N, R, s)) return e;
  if (hipError_t e = launch_expand(planes, splits, ta, g, scale, base, dx, dx_bf16, dz, K, R, s)) return e;
  if (hipError_t e = launch_sum(true, x, dz, g, scale, da, grad_bf16, K, R, parts, s)) return e;
  return launch_sum(false, dout, z, g, scale, db, grad_bf16, N, R, parts, s);
}

}  // namespace qlinear
