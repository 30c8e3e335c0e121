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

// Loads are never conditional (a lane's condition would make the wave wait for one load before the next): indexes
// past an operand's rows are held at its last row, whose results are not stored, and the eights of a row that its end cuts
// are the row's last eight values, of which one operand zeroes those that an earlier eight had.
typedef u32x4 u32x4_any __attribute__((aligned(2)));  // global loads and stores need no alignment here

// Eight bfloat16 from k on of a row of `len` (at p), held inside it.  SMALL: len may be below 8.
template <bool SMALL>
__device__ __forceinline__ u32x4 load_eight_of(const uint16_t* p, int64_t k, int64_t len) {
  if constexpr (!SMALL) {
    return *reinterpret_cast<const u32x4_any*>(p + (k < len - 8 ? k : len - 8));
  } else {
    u32x4 v{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e / 2] |= uint32_t(p[k + e < len ? k + e : len - 1]) << (16 * (e % 2));
    return v;
  }
}
// Zeros for what load_eight_of(p, k, len) repeats.
template <bool SMALL>
__device__ __forceinline__ u32x4 only_new(u32x4 v, int64_t k, int64_t len) {
  const int64_t past = k - (len - 8);  // values of the eight past the row's end
  const int none = past <= 0 ? 0 : past < 8 ? int(past) : 8;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (SMALL ? 2 * w >= 8 - none : 2 * w < none) v[w] &= 0xFFFF0000u;
    if (SMALL ? 2 * w + 1 >= 8 - none : 2 * w + 1 < none) v[w] &= 0x0000FFFFu;
  }
  return v;
}

// The groups of rows of a call.
struct Groups {
  const uint32_t* offsets;
  const int32_t* ids;
  int64_t G, L, T;
};

// Tile `tile` of the BM-row tiles of all groups: its first row, how many it has (0: there is no
// such tile) and its adapter (-1: none).  Up to 64 groups every wave finds it by itself; beyond, cum (LDS of
// G + 1) and one barrier are used.
template <int BM>
__device__ __forceinline__ int find_tile(const Groups& g, int* cum, int tile, int64_t* row0, int* adapter) {
  int64_t begin, end;
  int id, before;
  if (g.G <= kWave) {  // as count_group_tiles counts them
    const int lane = threadIdx.x % kWave, z = lane < g.G ? lane : int(g.G) - 1;
    const uint32_t limit = uint32_t(g.T);
    uint32_t b = g.offsets[z], e = g.offsets[z + 1];
    const int mine = g.ids[z];
    b = b < limit ? b : limit;
    e = e < limit ? e : limit;
    if (lane >= g.G) b = e = 0;
    uint32_t top = e;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const uint32_t o = __shfl_up(top, d, kWave);
      if (lane >= d) top = top > o ? top : o;
    }
    top = __shfl_up(top, 1, kWave);
    const int tiles = e > b && (lane == 0 || b >= top) ? int((e - b + BM - 1) / BM) : 0;
    int upto = tiles;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(upto, d, kWave);
      if (lane >= d) upto += o;
    }
    const uint64_t behind = __ballot(upto > tile);
    if (!behind) return 0;
    const int at = __builtin_ctzll(behind);
    begin = __builtin_amdgcn_readlane(int(b), at);
    end = __builtin_amdgcn_readlane(int(e), at);
    id = __builtin_amdgcn_readlane(mine, at);
    before = __builtin_amdgcn_readlane(upto - tiles, at);
  } else {
    if (threadIdx.x < kWave) count_group_tiles<BM>(cum, g.offsets, g.G, g.T);
    __syncthreads();
    if (tile >= cum[g.G]) return 0;
    int lo = 0, hi = int(g.G);  // cum[lo] <= tile < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (cum[mid] <= tile) lo = mid;
      else hi = mid;
    }
    begin = int64_t(g.offsets[lo]);
    end = int64_t(g.offsets[lo + 1]) < g.T ? int64_t(g.offsets[lo + 1]) : g.T;
    id = g.ids[lo];
    before = cum[lo];
  }
  *adapter = id >= 0 && id < g.L ? id : -1;
  begin += int64_t(tile - before) * BM;
  *row0 = begin;
  return int(end - begin < BM ? end - begin : BM);
}

// ---------------------------------------------------------------- long axis -> R

// plane[split][t][r] = sum over the split's part of K of x[t, k] a[l, r, k].  Block: a tile of
// BM rows, a part of K, 16 FR of the R; its waves take 64 values of k in turn, the next ones on their way, and
// add up at the end through LDS.  Both operands come straight from memory: neither is used by two waves.  Bound by
// the way to memory, at 64-byte pieces of 16 rows a load: 4096 rows, K = 4096 16 us at R = 16, 25 at R = 64; 4099 rows,
// K = 8192 28 us, 2.4 TB/s (here and below: the kernel alone, no operand in a cache, if nothing else is said).  64 rows of
// 64 groups, K = 4096: 6.0 us.  Twice the loads on their way, 8 waves a block, blocks that begin at
// different k change nothing; x past the caches costs a tenth more.
template <int BM, int FR, bool SMALL>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(const uint16_t* __restrict__ x,
                                                              const uint16_t* __restrict__ a, Groups g,
                                                              float* __restrict__ plane, int64_t K, int64_t R,
                                                              int64_t per, int tile0) {
  extern __shared__ int cum[];
  __shared__ v4f sums[kWaves][FR][kWave];
  constexpr int FM = BM / 16, KS = 2;  // KS MFMA steps of 32 at a time
  int64_t row0 = 0;
  int id = -1;
  const int rows = find_tile<BM>(g, cum, tile0 + int(blockIdx.x), &row0, &id);
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
    const uint16_t *xr[FM], *ar[FR];
#pragma unroll
    for (int m = 0; m < FM; ++m) xr[m] = x + (row0 + (16 * m + i < rows ? 16 * m + i : rows - 1)) * K;
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      const int64_t r = r0 + 16 * f + i;
      ar[f] = a + (int64_t(id) * R + (r < R ? r : R - 1)) * K;
    }
    u32x4 xf[2][FM][KS], af[2][FR][KS];
    auto load = [&](int to, int64_t k0) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int64_t k = k0 + 32 * s + 8 * q;
#pragma unroll
        for (int m = 0; m < FM; ++m) xf[to][m][s] = load_eight_of<SMALL>(xr[m], k, K);
#pragma unroll
        for (int f = 0; f < FR; ++f) af[to][f][s] = load_eight_of<SMALL>(ar[f], k, K);
      }
    };
    auto multiply = [&](int from, int64_t k0) {
      if (k0 + 32 * KS > K) {  // the row's end
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int f = 0; f < FR; ++f) af[from][f][s] = only_new<SMALL>(af[from][f][s], k0 + 32 * s + 8 * q, K);
      }
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int f = 0; f < FR; ++f)
            acc[m][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, af[from][f][s]),
                                                                __builtin_bit_cast(v8bf, xf[from][m][s]), acc[m][f], 0, 0, 0);
    };
    constexpr int kStep = 32 * KS * kWaves;  // `per` is a multiple
    int64_t k0 = begin + 32 * KS * wid;
    if (k0 < end) load(0, k0);
    for (; k0 < end; k0 += 2 * kStep) {
      load(1, k0 + kStep);  // past the end: the row's last values again, unused
      multiply(0, k0);
      if (k0 + kStep >= end) break;
      load(0, k0 + 2 * kStep);
      multiply(1, k0 + kStep);
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
// z_out where that is given.  Block: a tile of BM rows, `span` columns; a wave takes 64 columns
// at a time, as four MFMA tiles whose rows are permuted so that a lane's two results of a pair
// are eight consecutive columns: one 16-byte store of bfloat16.  LDS: the pieces of z as eights of r, the last one
// the row's last eight values with zeros for those that it repeats, as b's eights are loaded.
// WHOLE: an MFMA step is four eights of one piece, and b's are loaded once for all pieces; else the pieces' eights
// follow each other.  SMALL: R < 8.  TAIL: N % 8 != 0.  Bound by base and out: 4096 rows of 12
// groups, N = 14336, bfloat16, R = 64 68 us, 3.5 TB/s, R = 16 50, 4.7; of 8 groups, whose fewer tiles get spans of 256, R = 64
// 85, 3.2, float32 167, 3.0; 4099 rows, N = 8192, R = 16 38, 3.5; 64 rows, N = 4096 6.6.  From R = 64 on the matrix cores' and LDS's
// part shows beside the bytes.
constexpr int kSpan = 1024;

// Even lanes' second against odd lanes' first pieces.  Lanes 2 j and 2 j + 1 that hold pieces (first, second) of their
// own rows come to hold pieces 0 of both rows, and pieces 1 of both; and back.
__device__ __forceinline__ void swap_pairs(Eight<1>& first, Eight<1>& second, bool odd) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t mine = odd ? first.v[0][w] : second.v[0][w];
    const uint32_t other = __builtin_amdgcn_update_dpp(0, int(mine), 0xB1, 0xF, 0xF, false);  // the neighbour's
    if (odd) first.v[0][w] = other;
    else second.v[0][w] = other;
  }
}

template <int BM, int OUT, bool WHOLE, bool SMALL, bool TAIL>
__global__ __launch_bounds__(kThreads) void lora_expand_kernel(const float* __restrict__ plane, int splits,
                                                              const uint16_t* __restrict__ b, Groups g,
                                                              const float* __restrict__ scale,
                                                              const void* base, void* out,
                                                              float* __restrict__ z_out, int64_t N, int64_t R,
                                                              int64_t span, int tile0) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int FM = BM / 16, P = pieces_of(OUT);
  constexpr bool kPaired = OUT == 1;  // whole 128-byte lines a load and a store; float32 pieces are 32 bytes a lane
  const int R8 = int((R + 7) / 8), row_bytes = 16 * P * R8 + 16;
  char* const zs = lds;                                   // [BM][P R8 eights + 1 of padding]
  int* const cum = reinterpret_cast<int*>(lds + BM * row_bytes);
  int64_t row0 = 0;
  int id = -1;
  const int rows = find_tile<BM>(g, cum, tile0 + int(blockIdx.x), &row0, &id);
  if (rows <= 0) return;
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const float s = id >= 0 && scale ? scale[id] : 1.f;

  if (id >= 0 || z_out) {
    const bool keep = z_out && blockIdx.y == 0;
    for (int p = threadIdx.x; p < BM * R8; p += kThreads) {
      const int row = p / R8, c = p % R8;
      const int start = !SMALL && 8 * c > int(R) - 8 ? int(R) - 8 : 8 * c;
      const float* const from = plane + (row0 + (row < rows ? row : rows - 1)) * R;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
      for (int n = 0; n < splits; n += 4) {  // four planes on their way at once
        float part[4][8];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = SMALL && start + e >= int(R) ? int(R) - 1 : start + e;
            part[m][e] = from[(n + m < splits ? n + m : n) * g.T * R + r];
          }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += n + m < splits ? part[m][e] : 0.f;
      }
      v8bf eight[P];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = start + e;
        if (keep && row < rows && r < R) z_out[(row0 + row) * R + r] = v[e];
        __bf16 piece[P];
        split_bf16<P>(r >= 8 * c && r < R ? v[e] * s : 0.f, piece);
#pragma unroll
        for (int n = 0; n < P; ++n) eight[n][e] = piece[n];
      }
#pragma unroll
      for (int n = 0; n < P; ++n) *reinterpret_cast<v8bf*>(zs + row * row_bytes + 16 * (n * R8 + c)) = eight[n];
    }
    __syncthreads();
  }

  const int64_t first = int64_t(blockIdx.y) * span, last = first + span < N ? first + span : N;
  for (int64_t n0 = first + 64 * wid; n0 < last; n0 += 64 * kWaves) {
    Eight<OUT> add[FM][2];
    if (base) {
#pragma unroll
      for (int m = 0; m < FM; ++m) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int r = 16 * m + (kPaired ? (i & ~1) + p : i);
          const int64_t row = row0 + (r < rows ? r : rows - 1), n = n0 + 32 * (kPaired ? i & 1 : p) + 8 * q;
          if constexpr (TAIL) add[m][p].template load<true>(base, row * N + n, N - n);
          else add[m][p].get_at(base, row * N + (n < N ? n : N - 8));
        }
        if constexpr (kPaired) swap_pairs(add[m][0], add[m][1], i & 1);
      }
    }
    v4f acc[FM][2][2];
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int p = 0; p < 2; ++p) acc[m][p][0] = acc[m][p][1] = v4f{};
    if (id >= 0) {
      const uint16_t* br[2][2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int64_t n = n0 + 32 * p + 8 * (i / 4) + 4 * f + i % 4;
          br[p][f] = b + (int64_t(id) * N + (n < N ? n : N - 1)) * R;
        }
      v8bf bf[2][2];
      auto load = [&](int c) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int f = 0; f < 2; ++f) bf[p][f] = __builtin_bit_cast(v8bf, load_eight_of<SMALL>(br[p][f], 8 * c, R));
      };
      auto multiply = [&](int c, bool real) {
#pragma unroll
        for (int m = 0; m < FM; ++m) {
          const v8bf zf = real ? *reinterpret_cast<const v8bf*>(zs + (16 * m + i) * row_bytes + 16 * c) : v8bf{};
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int f = 0; f < 2; ++f)
              acc[m][p][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[p][f], zf, acc[m][p][f], 0, 0, 0);
        }
      };
      if constexpr (WHOLE) {
        for (int t = 0; t < R8 / 4; ++t) {
          load(4 * t + q);
#pragma unroll
          for (int p = 0; p < P; ++p) multiply(p * R8 + 4 * t + q, true);
        }
      } else {
        for (int t = 0; t < (P * R8 + 3) / 4; ++t) {
          const int c = 4 * t + q;
          load(c < R8 ? c : c < 2 * R8 ? c - R8 : c < P * R8 ? c - 2 * R8 : 0);
          multiply(c < P * R8 ? c : 0, c < P * R8);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      Eight<OUT> to[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[m][p][e / 4][e % 4];
        if (base) {
          float o[8];
          add[m][p].get(o);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        to[p].put(v);
      }
      if constexpr (kPaired) swap_pairs(to[0], to[1], i & 1);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int r = 16 * m + (kPaired ? (i & ~1) + p : i);
        const int64_t n = n0 + 32 * (kPaired ? i & 1 : p) + 8 * q;
        if (r < rows) to[p].template store<TAIL>(out, (row0 + r) * N + n, N - n);
      }
    }
  }
}

// ---------------------------------------------------------------- sums over rows

// The highest end of the groups before this lane's: `top`, that of all earlier waves of groups, and those of the lanes
// below.  b, e: the lane's group, clipped, 0 for lanes without one; `last`: the last lane with one.  `top` moves
// on.  Where no end in the wave falls a group begins at the end before it, so only what came before the wave counts.
__device__ __forceinline__ uint32_t ends_before(uint32_t b, uint32_t e, int last, uint32_t& top) {
  const int lane = threadIdx.x % kWave;
  uint32_t before = top, ends = e;
  if (__ballot(e < b) != 0) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const uint32_t o = __shfl_up(ends, d, kWave);
      if (lane >= d) ends = ends > o ? ends : o;
    }
    const uint32_t o = __shfl_up(ends, 1, kWave);
    if (lane > 0) before = before > o ? before : o;
    last = kWave - 1;
  }
  const uint32_t highest = __builtin_amdgcn_readlane(ends, last);
  top = top > highest ? top : highest;
  return before;
}

// dA[l, r, c] = s sum_t z[t, r] p[t, c] with z = dz, p = x, or dB[l, c, r] with z, p = dout, over the rows of adapter
// l's groups.  Block: one adapter, 16 FR of the R, 512 columns (128 a wave), every splits-th step of 32 rows, the next
// one on its way.  A lane loads 8 rows x 8 columns and turns them by byte permutations into its pieces of eight MFMA
// operands, whose row i is column 8 i + j of the wave's 128.  P: pieces of z.  Bound by x and dout: 4099 rows, K = 2048,
// N = 8192 30 us at R = 16, 2.8 TB/s; at R = 64 64, since each 32 of R read them again.  Blocks are shared out by the
// adapters that there are, not by their rows: 512 rows of each of 8 take 42 and 141 us, and 4096 rows of one of 32 (R = 16,
// K = N = 4096) 266, 25 where it is the only one.
struct SumArgs {
  const uint16_t* p;
  const float* z;
  void* out;  // [splits][L, R, C] or [L, C, R]
  int64_t C;
  int blocks;  // of 512 columns
};

template <bool DA, int FR, int P, bool SMALL>
__device__ __forceinline__ void lora_sum(const SumArgs& w, const Groups& g, const float* scale, int out_bf16, int64_t R,
                                         int column, int l, int64_t r0, int split, int splits) {
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const int64_t C = w.C, c0 = int64_t(column) * 512 + 128 * wid;
  if (c0 >= C) return;
  const float s = scale ? scale[l] : 1.f;
  const int64_t c = c0 + 8 * i, start = SMALL || c < C - 8 ? c : C - 8;
  v4f acc[8][FR];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[j][f] = v4f{};

  u32x4 row[2][8];
  float zv[2][FR][8];
  auto load = [&](int to, int64_t t0, int64_t end) {
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const int64_t t = t0 + 8 * q + d < end ? t0 + 8 * q + d : end - 1;
      row[to][d] = load_eight_of<SMALL>(w.p + t * C, c, C);
#pragma unroll
      for (int f = 0; f < FR; ++f) {
        const int64_t r = r0 + 16 * f + i;
        zv[to][f][d] = w.z[t * R + (r < R ? r : R - 1)];
      }
    }
  };
  auto add = [&](int from, int64_t t0, int64_t end) {
    v8bf zf[FR][P];
#pragma unroll
    for (int f = 0; f < FR; ++f)
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        __bf16 piece[P];
        split_bf16<P>(t0 + 8 * q + d < end ? zv[from][f][d] * s : 0.f, piece);
#pragma unroll
        for (int o = 0; o < P; ++o) zf[f][o][d] = piece[o];
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u32x4 v;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        v[d] = __builtin_amdgcn_perm(row[from][2 * d + 1][j / 2], row[from][2 * d][j / 2],
                                     j % 2 ? 0x07060302u : 0x05040100u);
      const v8bf pf = __builtin_bit_cast(v8bf, v);
#pragma unroll
      for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int o = 0; o < P; ++o) {
          if constexpr (DA) acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(zf[f][o], pf, acc[j][f], 0, 0, 0);
          else acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf, zf[f][o], acc[j][f], 0, 0, 0);
        }
    }
  };

  // The groups that the other kernels give tiles: a group that begins before an earlier one's end has no dz, and its
  // rows may be another's.
  int turn = split;  // steps to skip until this block's next one
  uint32_t top = 0;
  for (int64_t z0 = 0; z0 < g.G; z0 += kWave) {
    const int last = int(g.G - 1 - z0 < kWave - 1 ? g.G - 1 - z0 : kWave - 1);
    const int64_t z = z0 + (lane < last ? lane : last);
    const uint32_t limit = uint32_t(g.T);
    uint32_t b = g.offsets[z], e = g.offsets[z + 1];
    b = b < limit ? b : limit;
    e = e < limit ? e : limit;
    if (lane > last) b = e = 0;
    const uint32_t before = ends_before(b, e, last, top);  // by the whole wave
    const bool mine = g.ids[z] == l && b < e && b >= before;
    for (uint64_t left = __ballot(mine); left; left &= left - 1) {
      const int src = __builtin_ctzll(left);
      const int64_t begin = __builtin_amdgcn_readlane(int(b), src), end = __builtin_amdgcn_readlane(int(e), src);
      const int64_t steps = (end - begin + 31) / 32;
      int64_t n = turn;
      if (n < steps) load(0, begin + 32 * n, end);
      for (; n < steps; n += 2 * splits) {
        const int64_t t0 = begin + 32 * n, t1 = t0 + 32 * splits;
        load(1, t1 < end ? t1 : t0, end);
        add(0, t0, end);
        if (n + splits >= steps) {
          n += splits;
          break;
        }
        load(0, t1 + 32 * splits < end ? t1 + 32 * splits : t1, end);
        add(1, t1, end);
      }
      turn = int(n - steps);
    }
  }

  const int64_t size = g.L * C * R;
  if (DA && c >= C) return;
#pragma unroll
  for (int f = 0; f < FR; ++f)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // DA: this lane's columns start + j, rows r; else its r, and columns of lanes 4 q + e
        const int64_t r = r0 + 16 * f + (DA ? 4 * q + e : i);
        const int64_t from = c0 + 8 * (4 * q + e);
        const int64_t col = DA ? start + j : (SMALL || from < C - 8 ? from : C - 8) + j;
        if (r >= R || col >= C || (!DA && from >= C)) continue;
        const int64_t at = (int64_t(l) * (DA ? R : C) + (DA ? r : col)) * (DA ? C : R) + (DA ? col : r);
        if (out_bf16) reinterpret_cast<uint16_t*>(w.out)[at] = Elem<1>::put(acc[j][f][e]);
        else reinterpret_cast<float*>(w.out)[split * size + at] = acc[j][f][e];
      }
}

// Both sums in one launch: block columns of dA, then of dB.
template <int FR, int P, bool SMALL>
__global__ __launch_bounds__(kThreads) void lora_sum_kernel(SumArgs a, SumArgs b, Groups g, const float* __restrict__ scale,
                                                           int out_bf16, int64_t R, int r_blocks, int splits) {
  const int l = blockIdx.y / r_blocks, split = blockIdx.z;
  const int64_t r0 = int64_t(blockIdx.y % r_blocks) * 16 * FR;
  if (int(blockIdx.x) < a.blocks)
    lora_sum<true, FR, P, SMALL>(a, g, scale, out_bf16, R, blockIdx.x, l, r0, split, splits);
  else
    lora_sum<false, FR, P, SMALL>(b, g, scale, out_bf16, R, blockIdx.x - a.blocks, l, r0, split, splits);
}

// out[n] = the sum of the planes' values n, in their order; the planes hold dA's count_a and then dB's count_b values.
__global__ __launch_bounds__(kThreads) void lora_join_kernel(const float* __restrict__ part_a,
                                                             const float* __restrict__ part_b, int splits,
                                                             void* __restrict__ a, void* __restrict__ b, int out_bf16,
                                                             int64_t count_a, int64_t count_b) {
  int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (at >= count_a + count_b) return;
  const bool second = at >= count_a;
  if (second) at -= count_a;
  const float* const from = (second ? part_b : part_a) + at;
  const int64_t count = second ? count_b : count_a;
  float v = 0.f;
  for (int n = 0; n < splits; n += 4) {
    float part[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) part[m] = from[(n + m < splits ? n + m : n) * count];
#pragma unroll
    for (int m = 0; m < 4; ++m) v += n + m < splits ? part[m] : 0.f;
  }
  put_float(second ? b : a, at, v, out_bf16);
}

__global__ __launch_bounds__(kThreads) void clear_kernel(uint16_t* __restrict__ p, int64_t count) {
  for (int64_t at = int64_t(blockIdx.x) * kThreads + threadIdx.x; at < count; at += int64_t(gridDim.x) * kThreads) p[at] = 0;
}

// turned[l, c, r] = in[l, r, c] of A [L, R, K] and of B [L, N, R], in pieces of 32 x 32 through LDS; block columns of A's
// pieces, then B's.
struct Turn {
  const uint16_t* in;
  uint16_t* out;
  int64_t rows, cols;
  unsigned pieces;
};

__global__ __launch_bounds__(kThreads) void lora_turn_kernel(Turn a, Turn b) {
  __shared__ uint16_t tile[32][33];
  const bool second = blockIdx.x >= a.pieces;
  const Turn t = second ? b : a;
  const int64_t piece = second ? blockIdx.x - a.pieces : blockIdx.x, across = (t.cols + 31) / 32;
  const int64_t l = blockIdx.y, r0 = piece / across * 32, c0 = piece % across * 32;
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
#pragma unroll
  for (int n = 0; n < 32; n += 8)
    if (r0 + ty + n < t.rows && c0 + tx < t.cols) tile[ty + n][tx] = t.in[(l * t.rows + r0 + ty + n) * t.cols + c0 + tx];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < 32; n += 8)
    if (c0 + ty + n < t.cols && r0 + tx < t.rows) t.out[(l * t.cols + c0 + ty + n) * t.rows + r0 + tx] = tile[tx][ty + n];
}

// ---------------------------------------------------------------- launches

template <int V> using Int = std::integral_constant<int, V>;

// Tiles of more than 16 rows where a group has more on average.  The longest group is on the device: 900 rows beside 63
// groups of one row (R = 16, K = N = 4096) take 9 and 12 us in tiles of 16, alone 7.5 and 8.2 in tiles of 32.
bool tall(int64_t T, int64_t G) { return T > 16 * G; }

int64_t tile_count(int64_t T, int64_t G, int bm) { return std::min(T, T / bm + G); }

// go(first tile, tiles) for launches of at most 2^23 tiles: a launch has fewer than 2^32 threads along an axis, and the
// 2^30 rows that a call may have are 2^25 tiles and more.
template <typename F>
hipError_t by_launches(int64_t tiles, F&& go) {
  constexpr int64_t kMost = int64_t(1) << 23;
  for (int64_t t = 0; t < tiles; t += kMost)
    if (hipError_t e = go(int(t), unsigned(std::min(tiles - t, kMost)))) return e;
  return hipSuccess;
}

// Rows of the first product's tiles: 32 to R = 32 (4096 rows, R = 16: 16.4 us, 17.4 with 64), 64 beyond (R = 64: 25, 31 with
// 32, which read the adapters twice as often).
int shrink_rows(int64_t T, int64_t G, int64_t R) { return !tall(T, G) ? 16 : R <= 32 ? 32 : 64; }

// Parts of the long axis: as many as make 128 blocks, of few rows 256, of 512 values at least.  More blocks take the first
// product of few rows less time and that of many more (64 rows, K = 4096: 6.0 us, 7.4 with 128; 4096 rows, R = 64: 29 us, 25
// with 128), and the second product adds the parts.
int shrink_splits(int64_t T, int64_t G, int64_t K, int64_t R) {
  const int64_t tiles = tile_count(T, G, shrink_rows(T, G, R)) * ((R + 63) / 64), blocks = tall(T, G) ? 128 : 256;
  return int(std::max<int64_t>(1, std::min({int64_t(16), (blocks + tiles - 1) / tiles, K / 512})));
}

hipError_t launch_shrink(const uint16_t* x, const uint16_t* a, const Groups& g, float* plane, int splits, int64_t K,
                         int64_t R, hipStream_t s) {
  const int64_t per = (((K + splits - 1) / splits + 255) / 256) * 256;
  const size_t lds = size_t(g.G + 1) * 4;
  auto go = [&](auto kernel, int bm, int fr) {
    return by_launches(tile_count(g.T, g.G, bm), [&](int tile0, unsigned tiles) {
      const dim3 grid(tiles, unsigned(splits), unsigned((R + 16 * fr - 1) / (16 * fr)));
      return launch(kernel, grid, dim3(kThreads), lds, s, x, a, g, plane, K, R, per, tile0);
    });
  };
  auto by_rank = [&](auto bm, auto small) {
    constexpr int BM = decltype(bm)::value;
    constexpr bool SMALL = decltype(small)::value;
    if constexpr (BM != 64) {
      if (R <= 16) return go(lora_shrink_kernel<BM, 1, SMALL>, BM, 1);
      if (R <= 32) return go(lora_shrink_kernel<BM, 2, SMALL>, BM, 2);
    }
    if constexpr (BM != 32) return go(lora_shrink_kernel<BM, 4, SMALL>, BM, 4);
    return hipErrorInvalidValue;  // tiles of 32 rows have no other rank
  };
  auto by_rows = [&](auto small) {
    const int bm = shrink_rows(g.T, g.G, R);
    return bm == 64 ? by_rank(Int<64>{}, small) : bm == 32 ? by_rank(Int<32>{}, small) : by_rank(Int<16>{}, small);
  };
  return K < 8 ? by_rows(std::true_type{}) : by_rows(std::false_type{});
}

hipError_t launch_expand(const float* plane, int splits, const uint16_t* b, const Groups& g, const float* scale,
                         const void* base, void* out, int out_bf16, float* z_out, int64_t N, int64_t R, hipStream_t s) {
  const int64_t R8 = (R + 7) / 8;
  auto lds_of = [&](int bm) { return size_t(bm) * (16 * pieces_of(out_bf16) * R8 + 16) + size_t(g.G + 1) * 4; };
  // Rows of a tile: 32 where b is small enough to be read for each (R = 16: a training step of 4099 rows 135 us, 145 with
  // 64), else 64 (R = 64: 4096 prompt rows 96, 110 with 32).
  const int bm = !tall(g.T, g.G) ? 16 : R <= 32 ? 32 : lds_of(64) <= 64 * 1024 ? 64 : 16;
  const int64_t tiles = tile_count(g.T, g.G, bm);
  const int64_t span = tiles * ((N + kSpan - 1) / kSpan) >= 1024 ? kSpan : 256;
  auto go = [&](auto kernel) {
    return by_launches(tiles, [&](int tile0, unsigned count) {
      return launch(kernel, dim3(count, unsigned((N + span - 1) / span)), dim3(kThreads), lds_of(bm), s, plane, splits, b, g,
                    scale, base, out, z_out, N, R, span, tile0);
    });
  };
  auto by_rank = [&](auto rows, auto o, auto tail) {
    constexpr int BM = decltype(rows)::value, OUT = decltype(o)::value;
    constexpr bool TAIL = decltype(tail)::value;
    if (R < 8) return go(lora_expand_kernel<BM, OUT, false, true, TAIL>);
    if (R8 % 4 == 0) return go(lora_expand_kernel<BM, OUT, true, false, TAIL>);
    return go(lora_expand_kernel<BM, OUT, false, false, TAIL>);
  };
  auto by_tail = [&](auto rows, auto o) {
    return N % 8 ? by_rank(rows, o, std::true_type{}) : by_rank(rows, o, std::false_type{});
  };
  auto by_out = [&](auto rows) { return out_bf16 ? by_tail(rows, Int<1>{}) : by_tail(rows, Int<0>{}); };
  return bm == 64 ? by_out(Int<64>{}) : bm == 32 ? by_out(Int<32>{}) : by_out(Int<16>{});
}

// Blocks that share an adapter's rows: 512 blocks in all, and 128 rows for each on average.
int sum_splits(int64_t T, int64_t L, int64_t N, int64_t K, int64_t R) {
  const int64_t blocks = ((K + 511) / 512 + (N + 511) / 512) * L * ((R + 31) / 32);
  return int(std::max<int64_t>(1, std::min({int64_t(16), 512 / blocks, T / (128 * L)})));
}

// dA from x and dz, dB from dout and z.
hipError_t launch_sum(const uint16_t* x, const float* dz, const uint16_t* dout, const float* z, const Groups& g,
                      const float* scale, void* da, void* db, int out_bf16, int64_t N, int64_t K, int64_t R, float* parts,
                      hipStream_t s) {
  const int splits = sum_splits(g.T, g.L, N, K, R);
  const int fr = R <= 16 ? 1 : 2, r_blocks = int((R + 16 * fr - 1) / (16 * fr));
  const int64_t count_a = g.L * R * K, count_b = g.L * R * N;
  float* const parts_b = parts + splits * count_a;
  const SumArgs a{x, dz, splits > 1 ? parts : da, K, int((K + 511) / 512)};
  const SumArgs b{dout, z, splits > 1 ? parts_b : db, N, int((N + 511) / 512)};
  const dim3 grid(unsigned(a.blocks + b.blocks), unsigned(g.L * r_blocks), unsigned(splits));
  const int to_bf16 = splits > 1 ? 0 : out_bf16;
  auto go = [&](auto kernel) {
    return launch(kernel, grid, dim3(kThreads), 0, s, a, b, g, scale, to_bf16, R, r_blocks, splits);
  };
  auto by_rank = [&](auto n, auto small) {
    constexpr int P = decltype(n)::value;
    constexpr bool SMALL = decltype(small)::value;
    return fr == 1 ? go(lora_sum_kernel<1, P, SMALL>) : go(lora_sum_kernel<2, P, SMALL>);
  };
  auto by_type = [&](auto small) { return out_bf16 ? by_rank(Int<2>{}, small) : by_rank(Int<3>{}, small); };
  const hipError_t e = K < 8 || N < 8 ? by_type(std::true_type{}) : by_type(std::false_type{});
  if (e != hipSuccess || splits == 1) return e;
  return launch(lora_join_kernel, dim3(unsigned((count_a + count_b + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, parts,
                parts_b, splits, da, db, out_bf16, count_a, count_b);
}

hipError_t launch_turn(const uint16_t* a, uint16_t* ta, const uint16_t* b, uint16_t* tb, int64_t L, int64_t N, int64_t K,
                       int64_t R, hipStream_t s) {
  const int64_t r = (R + 31) / 32;
  const Turn at{a, ta, R, K, unsigned(r * ((K + 31) / 32))}, bt{b, tb, N, R, unsigned(r * ((N + 31) / 32))};
  return launch(lora_turn_kernel, dim3(at.pieces + bt.pieces, unsigned(L)), dim3(kThreads), 0, s, at, bt);
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
    const int n = sum_splits(T, L, N, K, R);
    total = parts + (n > 1 ? size_t(n) * L * (K + N) * R * 4 : 0);
  }
};

}  // namespace

hipError_t launch_clear(void* p, int64_t bytes, hipStream_t s) {
  const int64_t count = bytes / 2;
  if (count == 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((count + kThreads - 1) / kThreads, 65536);
  return launch(clear_kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, s, static_cast<uint16_t*>(p), count);
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
  if (hipError_t e = launch_turn(a, ta, b, tb, L, N, K, R, s)) return e;
  if (hipError_t e = launch_shrink(dout, tb, g, planes, splits, N, R, s)) return e;
  if (hipError_t e = launch_expand(planes, splits, ta, g, scale, base, dx, dx_bf16, dz, K, R, s)) return e;
  return launch_sum(x, dz, dout, z, g, scale, da, db, grad_bf16, N, K, R, parts, s);
}

}  // namespace qlinear
