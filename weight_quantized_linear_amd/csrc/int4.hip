// W4A16 with integer codes: out[m, n] = alpha * sum_k x[m, k] * D[n, k],
// D[n, k] = (code(n, k) - zero[n, k / g]) * scale[n, k / g], codes 0 .. 15
// two per byte (even k in the low nibble), one bfloat16 scale and, if given,
// one uint8 zero point per g consecutive k of a row (no zero points: 8).
//
// Arithmetic.  A code widened to bfloat16 is exact, a product of two
// bfloat16 values is exact in float32, and scale and zero point are constant
// over a group, so each group is summed first and corrected afterwards:
//   sum_k x D = sum_groups scale * (sum_k x code - zero * sum_k x),
// all sums in float32.  Nothing is rounded before the output, and a code
// costs one conversion per pair instead of a subtraction and a product each.
// The group's sum of x does not depend on n and is shared by all rows.
//
// Decoding.  A byte 0 .. 15 read as E4M3 is code * 2^-9 (the subnormals and
// the first binade are one linear range), so the hardware's E4M3 -> bfloat16
// pair conversion with scale 2^9 turns two masked bytes into two exact
// codes.  One dword gives the k order 0 2 4 6 1 3 5 7; the activation pairs
// are put in the same order once per tile (a dot product has no order).
#include "device.hpp"
#include "launch.hpp"

#include <algorithm>

namespace qlinear {

namespace {

// 16 bytes from any byte address (weight rows of odd length, weight views)
// and from any 2-byte address (activation rows); gfx950 takes unaligned
// global accesses.
struct __attribute__((packed)) Bytes16 {
  u32x4 v;
};
struct __attribute__((packed, aligned(2))) Halves16 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 ldw16(const uint8_t* p) { return reinterpret_cast<const Bytes16*>(p)->v; }
__device__ __forceinline__ u32x4 ldx16(const uint16_t* p) { return reinterpret_cast<const Halves16*>(p)->v; }

// Eight codes of a dword -> bfloat16 in the order 0 2 4 6 1 3 5 7.
__device__ __forceinline__ u32x4 int4x8_to_bf16x8(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.f, true);
  return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
               __builtin_bit_cast(uint32_t, d)};
}

// Eight consecutive activation values in the decoder's order.
__device__ __forceinline__ u32x4 decoder_order(u32x4 x) {
  return u32x4{__builtin_amdgcn_perm(x.y, x.x, 0x05040100u), __builtin_amdgcn_perm(x.w, x.z, 0x05040100u),
               __builtin_amdgcn_perm(x.y, x.x, 0x07060302u), __builtin_amdgcn_perm(x.w, x.z, 0x07060302u)};
}

__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(a[i]), as_bf16x2(b[i]), c, false);
  return c;
}
__device__ __forceinline__ float sum8(u32x4 a, float c) {
  const uint32_t ones = 0x3F803F80u;
  return dot8(a, u32x4{ones, ones, ones, ones}, c);
}

struct Int4Args {
  const uint8_t* w;       // [N, row_bytes]
  const uint16_t* scale;  // bfloat16 [N, groups]
  const uint8_t* zero;    // [N, groups], or null: 8
  int64_t row_bytes;      // ceil(K / 2)
  int64_t groups;
  int shift;              // log2 of the group size (62: one group per row)
};

__device__ __forceinline__ float zero_at(const Int4Args& a, int64_t i) { return a.zero ? float(a.zero[i]) : 8.f; }

// ---------------------------------------------------------------- GEMV

// 1 <= M <= 4 on the vector ALU.  Each wave owns ROWS weight rows; lane l
// takes the 32-code chunks c = l, l + 64, ... (16 bytes, inside one group),
// U of them in flight.  The at most 31 codes behind the last whole chunk are
// taken one per lane.
template <int M, int ROWS, int U>
__global__ __launch_bounds__(256) void int4_gemv_kernel(Int4Args a, const uint16_t* __restrict__ x,
                                                        void* __restrict__ out, int out_bf16, int64_t N, int64_t K,
                                                        float alpha, Epilogue epi) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t wave = int64_t(blockIdx.x) * (blockDim.x / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row0 = wave * ROWS;
  if (row0 >= N) return;  // uniform per wave
  const int64_t nchunks = K >> 5;
  int64_t row[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) row[r] = row0 + r < N ? row0 + r : N - 1;  // tail rows re-read the last, never stored

  float acc[M][ROWS];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) acc[m][r] = 0.f;

  for (int64_t c0 = 0; c0 < nchunks; c0 += int64_t(kWave) * U) {
    u32x4 wv[U][ROWS];
    float sv[U][ROWS], zv[U][ROWS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + int64_t(u) * kWave + lane;
      const bool ok = c < nchunks;
      const int64_t g = (c << 5) >> a.shift;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        wv[u][r] = ok ? ldw16(a.w + row[r] * a.row_bytes + c * 16) : u32x4{0u, 0u, 0u, 0u};
        sv[u][r] = ok ? bf16_to_f32(a.scale[row[r] * a.groups + g]) : 0.f;
        zv[u][r] = ok ? zero_at(a, row[r] * a.groups + g) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + int64_t(u) * kWave + lane;
      const bool ok = c < nchunks;
      u32x4 xv[M][4];
      float xs[M];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        xs[m] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          xv[m][q] = decoder_order(ok ? ldx16(x + m * K + c * 32 + 8 * q) : u32x4{0u, 0u, 0u, 0u});
          xs[m] = sum8(xv[m][q], xs[m]);
        }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float part[M];
#pragma unroll
        for (int m = 0; m < M; ++m) part[m] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const u32x4 codes = int4x8_to_bf16x8(wv[u][r][q]);
#pragma unroll
          for (int m = 0; m < M; ++m) part[m] = dot8(codes, xv[m][q], part[m]);
        }
#pragma unroll
        for (int m = 0; m < M; ++m) acc[m][r] = fmaf(sv[u][r], fmaf(-zv[u][r], xs[m], part[m]), acc[m][r]);
      }
    }
  }
  const int64_t k = (nchunks << 5) + lane;
  if (k < K) {
    const int64_t g = k >> a.shift;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const uint32_t byte = a.w[row[r] * a.row_bytes + (k >> 1)];
      const float code = float((k & 1) ? byte >> 4 : byte & 15u);
      const float d = bf16_to_f32(a.scale[row[r] * a.groups + g]) * (code - zero_at(a, row[r] * a.groups + g));
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m][r] = fmaf(d, bf16_to_f32(x[m * K + k]), acc[m][r]);
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float t = wave_sum(acc[m][r]);
      if (lane == 0 && row0 + r < N) store_epi(out, m, row0 + r, N, t, alpha, out_bf16, epi);
    }
}

// ---------------------------------------------------------------- matrix-core tile

// A block computes BM = 16 MT rows by BN = 16 NT WN columns with 16x16x32
// MFMA; WN waves stand side by side along N (each weight byte is read by one
// wave, straight into its registers), WK waves split the 128-value strips of
// K between them and add their tiles at the end.
//
// Weights: lane (n = l % 16, quarter h = l / 16) reads the 16 bytes k = 32 h
// .. 32 h + 31 of its row's strip.  Two half-wave swap stages transpose the
// 4x4 dwords over the quarters, after which dword t holds k = 32 t + 8 h ..
// + 7: MFMA step t covers 32 consecutive k, so a group of 32 is a whole step.
// Activation: the strip [BM][128] goes through registers into LDS in the
// decoder's order (16-byte chunks XOR-permuted by row against bank
// conflicts), and with it the float32 sum of each row over each group.
// After the last step of a group: acc += scale * (group - zero * sum).
constexpr int kStrip = 128;

template <int MT, int NT, int WN, int WK> struct Int4Tile {
  static constexpr int kBM = 16 * MT, kBN = 16 * NT * WN, kThreads = 64 * WN * WK;
  static constexpr int kStagers = WK > 1 ? 64 : 64 * WN;  // threads that fill one activation buffer
  static constexpr int kChunks = kBM * 16 / kStagers;     // 16-byte chunks per staging thread
  static constexpr int kXBytes = kBM * kStrip * 2;
  static constexpr int kBufs = WK > 1 ? 1 : 2;            // private buffers need no second one
  static constexpr int kSumBytes = kBM * 4 * 4;           // [group of the strip][BM] float32
  static constexpr int kOne = kXBytes + kSumBytes;
  static constexpr int kRing = kOne * (WK > 1 ? WK : kBufs);
  static constexpr int kReduce = WK > 1 ? WK * 64 * MT * NT * 16 : 0;
  static constexpr int kLds = kRing > kReduce ? kRing : kReduce;
  static_assert(WK == 1 || WN == 1, "either the columns or K are split over the waves");
};

// 4x4 transpose of dwords between register index and lane quarter.
__device__ __forceinline__ u32x4 transpose_quarters(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// Sum over groups of 2^LOG neighbouring lanes (LOG = 2, 3, 4), in each lane.
template <int LOG>
__device__ __forceinline__ float lanes_sum(float v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  if constexpr (LOG >= 3) v = dpp_add<0x141>(v);
  if constexpr (LOG >= 4) v = dpp_add<0x140>(v);
  return v;
}

// GS: MFMA steps per group inside a strip (1, 2, 4; 4 also for larger groups).
// store(m, n, value): m relative to the tile's first row.
template <int MT, int NT, int WN, int WK, int GS, typename Store>
__device__ __forceinline__ void int4_tile(char* lds, const Int4Args& a, const uint16_t* __restrict__ x, int64_t rows,
                                          int64_t N, int64_t K, int64_t n0, Store&& store) {
  using L = Int4Tile<MT, NT, WN, WK>;
  constexpr int G = 4 / GS;  // groups per strip
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int ln = lane & 15, quarter = lane >> 4;
  const int wn = WK > 1 ? 0 : wave, wk = WK > 1 ? wave : 0;
  const int stager = WK > 1 ? lane : threadIdx.x;
  const int nstrips = int((K + kStrip - 1) / kStrip);
  const int live = int((rows + 15) / 16);  // 16-row tiles that hold a row

  const uint8_t* wrow[NT];
  int64_t srow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    int64_t n = n0 + wn * 16 * NT + i * 16 + ln;
    n = n < N ? n : N - 1;  // columns past N re-read the last row, never stored
    wrow[i] = a.w + n * a.row_bytes;
    srow[i] = n * a.groups;
  }

  u32x4 wreg[NT], xreg[L::kChunks];
  uint16_t sreg[NT][G];
  uint8_t zreg[NT][G];

  auto fetch = [&](int strip) {
    const int64_t k = int64_t(strip) * kStrip;
    const int64_t kw = k + quarter * 32;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (kw + 32 <= K) {
        wreg[i] = ldw16(wrow[i] + (kw >> 1));
      } else {
        u32x4 v{0u, 0u, 0u, 0u};
        for (int64_t b = kw >> 1; b < a.row_bytes; ++b) {
          const int at = int(b - (kw >> 1));
          const uint32_t byte = uint32_t(wrow[i][b]) << (8 * (at & 3));
          if (at < 4) v.x |= byte;
          else if (at < 8) v.y |= byte;
          else if (at < 12) v.z |= byte;
          else v.w |= byte;
        }
        wreg[i] = v;
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        int64_t at = (k + g * 32 * GS) >> a.shift;
        at = srow[i] + (at < a.groups ? at : a.groups - 1);  // groups past K multiply zeros
        sreg[i][g] = a.scale[at];
        zreg[i][g] = a.zero ? a.zero[at] : uint8_t(8);
      }
    }
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j) {
      const int idx = stager + j * L::kStagers, m = idx >> 4;
      const int64_t kx = k + (idx & 15) * 8;
      u32x4 v{0u, 0u, 0u, 0u};
      if (m < rows) {
        const uint16_t* p = x + m * K + kx;
        if (kx + 8 <= K) {
          v = ldx16(p);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (kx + i < K) v[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
        }
      }
      xreg[j] = v;
    }
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[mt][i] = v4f{0.f, 0.f, 0.f, 0.f};

  int buf = 0;
  if (wk < nstrips) fetch(wk);
  for (int strip = wk; strip < nstrips; strip += WK) {
    char* xs = lds + (WK > 1 ? wk : buf) * L::kOne;
    float* sums = reinterpret_cast<float*>(xs + L::kXBytes);
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j) {
      const int idx = stager + j * L::kStagers, m = idx >> 4, c = idx & 15;
      const u32x4 v = decoder_order(xreg[j]);
      *reinterpret_cast<u32x4*>(xs + m * (kStrip * 2) + ((c ^ (m & 15)) << 4)) = v;
      const float s = lanes_sum<(GS == 4 ? 4 : GS == 2 ? 3 : 2)>(sum8(v, 0.f));
      if ((c & (4 * GS - 1)) == 0) sums[(c / (4 * GS)) * L::kBM + m] = s;
    }
    u32x4 w[NT];
    float sc[NT][G], zc[NT][G];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      w[i] = transpose_quarters(wreg[i]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        sc[i][g] = bf16_to_f32(sreg[i][g]);
        zc[i][g] = -float(zreg[i][g]);
      }
    }
    if (strip + WK < nstrips) fetch(strip + WK);
    wait_lds();
    if constexpr (WK == 1) block_barrier();
#pragma unroll
    for (int g = 0; g < G; ++g) {
      v8bf codes[NT][GS];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < GS; ++t)
          codes[i][t] = __builtin_bit_cast(v8bf, int4x8_to_bf16x8(w[i][g * GS + t]));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt >= live) break;  // uniform over the block
        v4f part[NT];
#pragma unroll
        for (int t = 0; t < GS; ++t) {
          const int c = (g * GS + t) * 4 + quarter;
          const v8bf xa = *reinterpret_cast<const v8bf*>(xs + (mt * 16 + ln) * (kStrip * 2) + ((c ^ ln) << 4));
#pragma unroll
          for (int i = 0; i < NT; ++i)
            part[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, codes[i][t], t == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : part[i],
                                                              0, 0, 0);
        }
        const v4f xsum = *reinterpret_cast<const v4f*>(sums + g * L::kBM + mt * 16 + quarter * 4);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[mt][i][r] = fmaf(sc[i][g], fmaf(zc[i][g], xsum[r], part[i][r]), acc[mt][i][r]);
      }
    }
    buf ^= 1;
  }

  if constexpr (WK > 1) {
    // Add the waves' tiles in wave order: each wave leaves its tile in LDS
    // (one 16-byte store per lane and 16x16 tile) and takes every WK-th one.
    __syncthreads();
    v4f* red = reinterpret_cast<v4f*>(lds);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < NT; ++i) red[((wk * MT + mt) * NT + i) * 64 + lane] = acc[mt][i];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < MT * NT; ++q) {
      if (q % WK != wk) continue;
      v4f v = red[q * 64 + lane];
#pragma unroll
      for (int o = 1; o < WK; ++o) {
        const v4f b = red[(o * MT * NT + q) * 64 + lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += b[r];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) store((q / NT) * 16 + quarter * 4 + r, (q % NT) * 16 + ln, v[r]);
    }
  } else {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          store(mt * 16 + quarter * 4 + r, wn * 16 * NT + i * 16 + ln, acc[mt][i][r]);
  }
}

template <int MT, int NT, int WN, int WK, int GS>
__global__ __launch_bounds__(64 * WN * WK) void int4_gemm_kernel(Int4Args a, const uint16_t* __restrict__ x,
                                                                 void* __restrict__ out, int out_bf16, int64_t M,
                                                                 int64_t N, int64_t K, float alpha, Epilogue epi) {
  using L = Int4Tile<MT, NT, WN, WK>;
  __shared__ __attribute__((aligned(16))) char lds[L::kLds];
  // Row tiles of one column tile follow each other on one XCD, whose L2 then
  // holds the column tile's weights.
  const int64_t mtiles = (M + L::kBM - 1) / L::kBM, ntiles = (N + L::kBN - 1) / L::kBN, total = mtiles * ntiles;
  const int64_t per = (total + 7) / 8;
  const int64_t tile = int64_t(blockIdx.x % 8) * per + blockIdx.x / 8;
  if (int64_t(blockIdx.x / 8) >= per || tile >= total) return;  // uniform over the block
  const int64_t m0 = tile % mtiles * L::kBM, n0 = tile / mtiles * L::kBN;
  int4_tile<MT, NT, WN, WK, GS>(lds, a, x + m0 * K, M - m0, N, K, n0, [&](int m, int n, float v) {
    if (m0 + m < M && n0 + n < N) store_epi(out, m0 + m, n0 + n, N, v, alpha, out_bf16, epi);
  });
}

// Grouped: group z owns rows a_offsets[z] .. a_offsets[z + 1] - 1 (clipped to
// T) and multiplies them by expert expert_ids[z]; an id outside 0 .. E - 1
// writes zeros, an empty group nothing.  Every block builds the prefix sum of
// the groups' row tiles in LDS and walks its XCD's contiguous part of the
// (group, row tile, column tile) list.
template <int MT, int NT, int WN, int WK, int GS>
__global__ __launch_bounds__(64 * WN * WK) void int4_grouped_kernel(
    Int4Args a, const uint16_t* __restrict__ x, const uint32_t* __restrict__ a_offsets,
    const int32_t* __restrict__ expert_ids, void* __restrict__ out, int out_bf16, int64_t groups, int64_t T, int64_t N,
    int64_t K, int64_t E) {
  using L = Int4Tile<MT, NT, WN, WK>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int* cum = reinterpret_cast<int*>(lds + L::kLds);  // cum[z] = row tiles of groups 0 .. z - 1
  auto span = [&](int64_t z, int64_t& start, int64_t& rows) {
    int64_t b = a_offsets[z], e = a_offsets[z + 1];
    b = b < T ? b : T;
    e = e < T ? e : T;
    start = b;
    rows = e > b ? e - b : 0;
  };
  if (threadIdx.x < kWave) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int64_t z0 = 0; z0 <= groups; z0 += kWave) {
      const int64_t z = z0 + lane;
      int t = 0;
      if (z < groups) {
        int64_t start, rows;
        span(z, start, rows);
        t = int((rows + L::kBM - 1) / L::kBM);
      }
      int incl = t;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += o;
      }
      if (z <= groups) cum[z] = carry + incl - t;
      carry += __shfl(incl, kWave - 1, kWave);
    }
  }
  __syncthreads();
  const int64_t ntiles = (N + L::kBN - 1) / L::kBN, work = int64_t(cum[groups]) * ntiles;
  const int64_t xcd = blockIdx.x % 8, per_xcd = gridDim.x / 8;  // gridDim.x is a multiple of 8
  const int64_t first = xcd * work / 8, last = (xcd + 1) * work / 8;
  for (int64_t i = first + blockIdx.x / 8; i < last; i += per_xcd) {
    const int mt = int(i / ntiles);
    const int64_t n0 = i % ntiles * L::kBN;
    int64_t lo = 0, hi = groups;  // cum[lo] <= mt < cum[hi]
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (cum[mid] <= mt) lo = mid;
      else hi = mid;
    }
    int64_t start, rows;
    span(lo, start, rows);
    const int64_t m0 = start + int64_t(mt - cum[lo]) * L::kBM, end = start + rows;
    const int64_t e = expert_ids[lo];
    auto put = [&](int m, int n, float v) {
      if (m0 + m >= end || n0 + n >= N) return;
      store_out(out, (m0 + m) * N + n0 + n, v, 1.f, out_bf16);
    };
    if (e < 0 || e >= E) {
      for (int idx = threadIdx.x; idx < L::kBM * L::kBN; idx += L::kThreads) put(idx / L::kBN, idx % L::kBN, 0.f);
      continue;
    }
    Int4Args b = a;
    b.w += e * N * a.row_bytes;
    b.scale += e * N * a.groups;
    if (b.zero) b.zero += e * N * a.groups;
    __syncthreads();  // the previous tile's buffers are free
    int4_tile<MT, NT, WN, WK, GS>(lds, b, x + m0 * K, end - m0, N, K, n0, put);
  }
}

// ---------------------------------------------------------------- launch

Int4Args make_args(const uint8_t* w, const uint16_t* scale, const uint8_t* zero, int64_t K, int64_t group) {
  Int4Args a{w, scale, zero, (K + 1) / 2, (K + group - 1) / group, 62};
  if (group < K) {
    a.shift = 0;
    while ((int64_t(1) << a.shift) < group) ++a.shift;
  }
  return a;
}

template <typename F>
hipError_t by_group(const Int4Args& a, F&& go) {
  if (a.shift == 5) return go(std::integral_constant<int, 1>{});
  if (a.shift == 6) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 4>{});
}

template <int M>
hipError_t gemv_m(const Int4Args& a, const uint16_t* x, void* out, int bf16, int64_t N, int64_t K, float alpha,
                  int num_cus, const Epilogue& epi, hipStream_t s) {
  const int64_t waves = int64_t(num_cus) * 8;
  auto go = [&](auto kernel, int rows) {
    return launch(kernel, dim3(unsigned((N + 4 * rows - 1) / (4 * rows))), dim3(256), 0, s, a, x, out, bf16, N, K,
                  alpha, epi);
  };
  if (N >= waves * 4) return go(int4_gemv_kernel<M, 4, 2>, 4);
  if (N >= waves * 2) return go(int4_gemv_kernel<M, 2, 2>, 2);
  return go(int4_gemv_kernel<M, 1, 2>, 1);
}

template <int MT, int NT, int WN, int WK>
hipError_t gemm_cfg(const Int4Args& a, const uint16_t* x, void* out, int bf16, int64_t M, int64_t N, int64_t K,
                    float alpha, const Epilogue& epi, hipStream_t s) {
  using L = Int4Tile<MT, NT, WN, WK>;
  const int64_t total = ((M + L::kBM - 1) / L::kBM) * ((N + L::kBN - 1) / L::kBN);
  const int64_t blocks = (total + 7) / 8 * 8;
  if (blocks * L::kThreads >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  return by_group(a, [&](auto gs) {
    return launch(int4_gemm_kernel<MT, NT, WN, WK, decltype(gs)::value>, dim3(unsigned(blocks)), dim3(L::kThreads), 0,
                  s, a, x, out, bf16, M, N, K, alpha, epi);
  });
}

template <int MT, int NT, int WN, int WK>
hipError_t grouped_cfg(const Int4Args& a, const uint16_t* x, const uint32_t* offsets, const int32_t* ids, void* out,
                       int bf16, int64_t G, int64_t E, int64_t T, int64_t N, int64_t K, int num_cus, hipStream_t s) {
  using L = Int4Tile<MT, NT, WN, WK>;
  const int lds = int(L::kLds + 4 * (G + 1));
  constexpr int kMaxLds = 160 * 1024;
  if (lds > kMaxLds) return hipErrorInvalidValue;
  // At most ceil(T / BM) + min(G, T) row tiles exist.
  const int64_t upper = ((T + L::kBM - 1) / L::kBM + std::min(G, T)) * ((N + L::kBN - 1) / L::kBN);
  const int64_t per_cu = std::max<int64_t>(1, std::min<int64_t>(kMaxLds / lds, 16 / (WN * WK)));
  const int64_t blocks = (std::min(upper, per_cu * num_cus) + 7) / 8 * 8;
  return by_group(a, [&](auto gs) -> hipError_t {
    auto kernel = int4_grouped_kernel<MT, NT, WN, WK, decltype(gs)::value>;
    static std::atomic<uint64_t> lds_set{0};
    if (hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), kMaxLds, lds_set)) return e;
    return launch(kernel, dim3(unsigned(blocks)), dim3(L::kThreads), lds, s, a, x, offsets, ids, out, bf16, G, T, N, K,
                  E);
  });
}

}  // namespace

hipError_t launch_int4_gemm(const uint8_t* w, const uint16_t* scale, const uint8_t* zero, const uint16_t* x, void* out,
                            int out_bf16, int64_t M, int64_t N, int64_t K, int64_t group, float alpha, int num_cus,
                            hipStream_t s, const Epilogue& epi) {
  const Int4Args a = make_args(w, scale, zero, K, group);
  switch (M) {
    case 1: return gemv_m<1>(a, x, out, out_bf16, N, K, alpha, num_cus, epi, s);
    case 2: return gemv_m<2>(a, x, out, out_bf16, N, K, alpha, num_cus, epi, s);
    default: break;
  }
  if (M <= 16) return gemm_cfg<1, 1, 1, 4>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
  if (M <= 64) return gemm_cfg<2, 2, 1, 4>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
  return gemm_cfg<4, 4, 4, 1>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
}

hipError_t launch_int4_grouped(const uint8_t* w, const uint16_t* scale, const uint8_t* zero, const uint16_t* x,
                               const uint32_t* a_offsets, const int32_t* expert_ids, void* out, int out_bf16,
                               int64_t G, int64_t E, int64_t T, int64_t N, int64_t K, int64_t group, int num_cus,
                               hipStream_t s) {
  const Int4Args a = make_args(w, scale, zero, K, group);
  if (T <= 8 * G) return grouped_cfg<1, 4, 1, 4>(a, x, a_offsets, expert_ids, out, out_bf16, G, E, T, N, K, num_cus, s);
  return grouped_cfg<4, 4, 4, 1>(a, x, a_offsets, expert_ids, out, out_bf16, G, E, T, N, K, num_cus, s);
}

}  // namespace qlinear
