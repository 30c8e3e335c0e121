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
#include <cstddef>

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

template <typename T> struct __attribute__((packed, aligned(1))) Packed1 {
  T v;
};
template <typename T> struct __attribute__((packed, aligned(2))) Packed2 {
  T v;
};
template <typename T> __device__ __forceinline__ T ld_any1(const void* p) {
  return reinterpret_cast<const Packed1<T>*>(p)->v;
}
template <typename T> __device__ __forceinline__ T ld_any2(const void* p) {
  return reinterpret_cast<const Packed2<T>*>(p)->v;
}

// The first `left` (< 16) bytes at p, zeros behind: at most four loads, all in flight together.
__device__ __forceinline__ u32x4 ld_bytes(const uint8_t* p, int left) {
  left = left < 0 ? 0 : left;
  uint64_t a = 0, rest = 0;
  if (left & 8) a = ld_any1<uint64_t>(p);
  if (left & 4) rest = ld_any1<uint32_t>(p + (left & 8));
  if (left & 2) rest |= uint64_t(ld_any1<uint16_t>(p + (left & 12))) << (8 * (left & 4));
  if (left & 1) rest |= uint64_t(p[left & 14]) << (8 * (left & 6));
  const uint64_t lo = (left & 8) ? a : rest, hi = (left & 8) ? rest : 0;
  return u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
}
// The first `left` (< 8) 16-bit values at p, zeros behind.
__device__ __forceinline__ u32x4 ld_halves(const uint16_t* p, int left) {
  left = left < 0 ? 0 : left;
  uint64_t a = 0, rest = 0;
  if (left & 4) a = ld_any2<uint64_t>(p);
  if (left & 2) rest = ld_any2<uint32_t>(p + (left & 4));
  if (left & 1) rest |= uint64_t(p[left & 6]) << (16 * (left & 2));
  const uint64_t lo = (left & 4) ? a : rest, hi = (left & 4) ? rest : 0;
  return u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
}

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

// The same in the order 0 .. 7, for two instructions more.
__device__ __forceinline__ u32x4 int4x8_to_bf16x8_ordered(uint32_t w) {
  const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u), hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true);
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

// How the arguments of every kernel here begin, and where they lie.  The address exists in
// a kernel's own body only: each kernel takes it there and hands it on, so that what uses it may also be a
// function of its own (where it does not exist, and reading through it faults).
struct Int4Head {
  Int4Args a;
  const uint16_t* x;
};
static_assert(offsetof(Int4Head, x) == sizeof(Int4Args) && sizeof(Int4Args) % 8 == 0, "arguments lie side by side");
typedef const __attribute__((address_space(4))) Int4Head* Int4HeadPtr;
#define QL_INT4_HEAD() ((Int4HeadPtr)__builtin_amdgcn_kernarg_segment_ptr())

// One output by the definition, sum_k x[k] (code - zero) scale, in float64: what a result that is not finite is
// replaced with.  The factored sum has no finite value where sum x code or zero sum x passes float32's range,
// and is inf - inf = NaN wherever an activation is infinite; here only the result's own value counts.
// at: QL_INT4_HEAD() of the kernel; m: row of x, n: row of the weights (of all experts).
// One lane walks K, which costs nothing where all results are finite, and it stops at the first
// NaN (M = 500, N = 14336, K = 4096: 108 us a call of its own, 188 if all x is NaN, 363 with one
// infinity, 8 ms with one in every row).  The operands are read from the kernel's arguments anew:
// kept for this from the start, they took 13 scalar registers from the tiles that have none to spare.
__device__ __forceinline__ float int4_defined(Int4HeadPtr at, int64_t m, int64_t n, int64_t K) {
  uint64_t args = reinterpret_cast<uint64_t>(at);
  asm volatile("" : "+s"(args));
  const Int4HeadPtr head = reinterpret_cast<Int4HeadPtr>(args);
  const int64_t row_bytes = head->a.row_bytes, groups = head->a.groups;
  const int shift = head->a.shift;
  const uint8_t* const w = head->a.w + n * row_bytes;
  const uint16_t* const scale = head->a.scale + n * groups;
  const uint8_t* const zeros = head->a.zero ? head->a.zero + n * groups : nullptr;
  const uint16_t* const x = head->x + m * K;
  double sum = 0.0;
  for (int64_t k = 0; k < K && sum == sum; k += 32) {  // 32 values lie in one group
    const int64_t g = k >> shift;
    const int left = int(K - k);
    const u32x4 c = left >= 31 ? ldw16(w + (k >> 1)) : ld_bytes(w + (k >> 1), (left + 1) >> 1);
    const float zero = zeros ? float(zeros[g]) : 8.f;
    double part = 0.0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint16_t* const p = x + k + 8 * t;
      const u32x4 v = left >= 8 * t + 8 ? ldx16(p) : ld_halves(p, left - 8 * t);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xi = (i & 1) ? bf16hi(v[i / 2]) : bf16lo(v[i / 2]);
        part = fma(double(xi), double(float((c[t] >> (4 * i)) & 15u) - zero), part);
      }
    }
    sum = fma(part, double(bf16_to_f32(scale[g])), sum);
  }
  return float(sum);
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

constexpr int kStrip = 128;  // values of k that the four quarters of a wave take with one 16-byte load each

// 4x4 transpose of dwords between register index and lane quarter.
__device__ __forceinline__ u32x4 transpose_quarters(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------- streaming products of few rows

// 1 <= M <= 4 rows of x: the weight is read once, straight into registers,
// and the matrix cores contract it, so that a code costs its decoding alone
// (7 vector instructions per 8 codes; the dot products would be 4 more per row of x).
//
// A wave owns NT tiles of 16 weight rows; lane (n = l % 16, quarter q = l / 16)
// reads 16-byte chunks (32 codes) of row n, chunk 4 s + q of strip s, four
// strips (a step of 512 codes) at a time.  The 16x16x32 MFMA takes codes as
// its column operand: column n, and quarter q's 8 of 32 k slots hold dword t of
// the lane's chunk.  The slots' order is free as long as x has the same.
// Row 4 g + m of the other operand is x row m in the slots of quarter g and zero
// elsewhere.  Four MFMAs then leave in lane (n, g) the sum over that lane's own
// chunk for each m, to be scaled with the lane's own group, whatever the group
// size: no lane exchanges, and only M of the 4 results per lane to correct.  The
// quarters are added at the end.
//
// x (decoder's order) and its sums over 32 values lie in LDS, kChunkK values of k at
// a time; WK waves split the steps of a chunk and add their sums through LDS at
// the end, where there are too few rows to fill the card.
//
// Bound by HBM where the weight is large (128256 x 4096, one row: 52 us, 5.2 TB/s of
// 5.7 that loads of 64 bytes from each of 16 rows reach without any work), by the launch
// and the way to the first weights where it is small (4096 x 4096: 5.5 us).

constexpr int kStep = 512;  // codes per lane quarter set and step: 4 strips

template <int M, int NT, int WN, int WK> struct StreamLayout {
  static constexpr int kWaves = WN * WK, kThreads = 64 * kWaves;
  static constexpr int kChunkK = 4096;
  static constexpr int kZeros = 1024;  // what the rows outside a quarter read
  static constexpr int kRowBytes = kChunkK * 2 + 16;
  static constexpr int kSums = kZeros + M * kRowBytes;  // float32 [M][kChunkK / 32]
  static constexpr int kReduce = kWaves * NT * M * 16 * 4;
  static constexpr int kUse = kSums + M * (kChunkK / 32) * 4;
  static constexpr int kLds = kUse > kReduce ? kUse : kReduce;
};

// The thread's index, anew at each call: the tiles' many addresses are made of it, and a
// kernel that walks tiles would keep them all in registers from one tile to the next
// (200 bytes a lane went to memory).
__device__ __forceinline__ int own_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// What a lane holds of one step of one row tile.  SH = log2(group) for 5, 6, 7;
// 8 stands for all larger groups.  The scales and zero points of a step's groups
// are neighbours in memory and come in one or two loads.
template <int SH> struct StreamScales;
template <> struct StreamScales<5> {
  u32x4 s[2], z;
};
template <> struct StreamScales<6> {
  u32x4 s;
  u32x2 z;
};
template <> struct StreamScales<7> {
  u32x2 s;
  uint32_t z;
};
template <> struct StreamScales<8> {
  uint16_t s[4];
  uint8_t z[4];
};

template <int SH>
__device__ __forceinline__ void load_scales(StreamScales<SH>& o, const Int4Args& a, int64_t row, int64_t step) {
  if constexpr (SH == 8) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t g = row + ((step * kStep + u * kStrip) >> a.shift);
      o.s[u] = a.scale[g];
      o.z[u] = a.zero ? a.zero[g] : uint8_t(8);
    }
  } else {
    const int64_t g = row + (step << (9 - SH));
    const uint32_t eight = 0x08080808u;
    if constexpr (SH == 5) {
      o.s[0] = ld_any2<u32x4>(a.scale + g);
      o.s[1] = ld_any2<u32x4>(a.scale + g + 8);
      o.z = a.zero ? ld_any1<u32x4>(a.zero + g) : u32x4{eight, eight, eight, eight};
    } else if constexpr (SH == 6) {
      o.s = ld_any2<u32x4>(a.scale + g);
      o.z = a.zero ? ld_any1<u32x2>(a.zero + g) : u32x2{eight, eight};
    } else {
      o.s = ld_any2<u32x2>(a.scale + g);
      o.z = a.zero ? ld_any1<uint32_t>(a.zero + g) : eight;
    }
  }
}

// Scale and zero point of 32-code chunk c of strip u of the step.
template <int SH>
__device__ __forceinline__ void pick_scale(const StreamScales<SH>& o, int u, int c, float& s, float& z) {
  if constexpr (SH == 8) {
    s = bf16_to_f32(o.s[u]);
    z = float(o.z[u]);
  } else {
    constexpr uint32_t kLow = 0x01000C0Cu, kHigh = 0x03020C0Cu;  // half of a dword into the upper half
    uint32_t d;
    if constexpr (SH == 5) {
      d = (c & 2) ? o.s[u >> 1][2 * (u & 1) + 1] : o.s[u >> 1][2 * (u & 1)];
      d = __builtin_amdgcn_perm(d, d, (c & 1) ? kHigh : kLow);
      z = float((o.z[u] >> (8 * c)) & 255u);
    } else if constexpr (SH == 6) {
      d = o.s[u];
      d = __builtin_amdgcn_perm(d, d, (c & 2) ? kHigh : kLow);
      z = float(((o.z[u >> 1] >> (16 * (u & 1))) >> (4 * (c & 2))) & 255u);
    } else {
      d = (u & 1) ? o.s[u >> 1] & 0xFFFF0000u : o.s[u >> 1] << 16;
      z = float((o.z >> (8 * u)) & 255u);
    }
    s = __uint_as_float(d);
  }
}

// store(m, n, value): m < rows, n relative to the block's first row of weights; defined(m, n): the value of a result
// that is not finite.
template <int M, int NT, int WN, int WK, int SH, typename Store, typename Defined>
__device__ __forceinline__ void int4_stream_tile(char* lds, const Int4Args& a, const uint16_t* __restrict__ x, int rows,
                                                 int64_t N, int64_t K, int64_t n0, Store&& store, Defined&& defined) {
  using L = StreamLayout<M, NT, WN, WK>;
  const int thread = own_thread();
  const int lane = thread & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(thread / kWave);
  const int ln = lane & 15, quarter = lane >> 4;
  const int wn = wave / WK, wk = wave % WK;

  const uint8_t* wrow[NT];
  int64_t srow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    int64_t n = n0 + (wn * NT + i) * 16 + ln;
    n = n < N ? n : N - 1;  // rows past N re-read the last, never stored
    wrow[i] = a.w + n * a.row_bytes + quarter * 16;
    srow[i] = n * a.groups;
  }
  const int64_t steps = K / kStep;  // whole ones

  struct Step {
    u32x4 w[NT][4];
    StreamScales<SH> sc[NT];
  };
  auto fetch = [&](Step& f, int64_t step) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int u = 0; u < 4; ++u) f.w[i][u] = ldw16(wrow[i] + step * (kStep / 2) + u * (kStrip / 2));
      load_scales<SH>(f.sc[i], a, srow[i], step);
    }
  };

  float acc[NT][M];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < M; ++m) acc[i][m] = 0.f;

  // Where this lane reads x in the staged chunk; lanes of other quarters or past `rows`
  // read zeros (and a row past `rows` whatever sums: its results are not stored).
  const bool mine = (ln >> 2) == quarter && (ln & 3) < rows;
  const int xlane = L::kZeros + (ln & 3) * L::kRowBytes + 64 * quarter;
  const float* sums = reinterpret_cast<const float*>(lds + L::kSums);

  // One strip: its place in the staged x, its first 32-value chunk; scale(i, c, s, z) of row tile i, chunk c.
  auto strip = [&](int xbase, int chunk0, const u32x4 (&w)[NT], auto&& scale) {
    u32x4 xa[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) xa[t] = *reinterpret_cast<const u32x4*>(lds + xbase + t * 16);
    float xs[M];
#pragma unroll
    for (int m = 0; m < M; ++m) xs[m] = sums[m * (L::kChunkK / 32) + chunk0 + quarter];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      v4f part{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 4; ++t)
        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xa[t]),
                                                       __builtin_bit_cast(v8bf, int4x8_to_bf16x8(w[i][t])), part, 0, 0, 0);
      float s, z;
      scale(i, quarter, s, z);
#pragma unroll
      for (int m = 0; m < M; ++m) acc[i][m] = fmaf(s, fmaf(-z, xs[m], part[m]), acc[i][m]);
    }
  };

  const int64_t chunks = (K + L::kChunkK - 1) / L::kChunkK;
  for (int64_t ch = 0; ch < chunks; ++ch) {
    const int64_t kc = ch * L::kChunkK;
    const int64_t step_end = kc + L::kChunkK < K ? (kc + L::kChunkK) / kStep : steps;
    const int64_t step0 = kc / kStep;
    Step cur;
    if (step0 + wk < step_end) fetch(cur, step0 + wk);  // in flight while x is staged
    // x rows in the decoder's order, zeros past K, and the sums of 32 values.
    const int klen = int(K - kc < L::kChunkK ? (K - kc + kStrip - 1) / kStrip * kStrip : L::kChunkK);
    const int per_row = klen / 8;
    for (int idx = thread; idx < rows * per_row; idx += L::kThreads) {  // klen % 32 == 0: quads stay together
      const int m = idx / per_row, c = idx % per_row;
      const int64_t k = kc + c * 8;
      const uint16_t* p = x + m * K + k;
      const u32x4 v = decoder_order(k + 8 <= K ? ldx16(p) : ld_halves(p, int(K - k)));
      *reinterpret_cast<u32x4*>(lds + L::kZeros + m * L::kRowBytes + c * 16) = v;
      float s = dpp_add<0xB1>(sum8(v, 0.f));
      s = dpp_add<0x4E>(s);
      if ((c & 3) == 0) reinterpret_cast<float*>(lds + L::kSums)[m * (L::kChunkK / 32) + (c >> 2)] = s;
    }
    if (ch == 0)
      for (int i = thread; i < L::kZeros / 16; i += L::kThreads) *reinterpret_cast<u32x4*>(lds + i * 16) = u32x4{0u, 0u, 0u, 0u};
    wait_lds();
    block_barrier();

    for (int64_t step = step0 + wk; step < step_end; step += WK) {
      Step next;
      const bool more = step + WK < step_end;
      if (more) fetch(next, step + WK);
      const int off = int(step - step0) * kStep;
      const int xbase = mine ? xlane + off * 2 : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        u32x4 w[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) w[i] = cur.w[i][u];
        strip(xbase + u * kStrip * 2, off / 32 + u * 4, w,
              [&](int i, int c, float& s, float& z) { pick_scale<SH>(cur.sc[i], u, c, s, z); });
      }
      if (more) cur = next;
    }
    // The strips behind the last whole step, guarded, by the wave whose turn it is.
    if (ch == chunks - 1 && steps * kStep < K && wk == int(steps % WK)) {
      for (int64_t k = steps * kStep; k < K; k += kStrip) {
        const int64_t kw = k + quarter * 32;
        u32x4 w[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint8_t* p = wrow[i] + (k >> 1);
          const int64_t left = a.row_bytes - (kw >> 1);
          w[i] = left >= 16 ? ldw16(p) : ld_bytes(p, int(left));
        }
        const int off = int(k - kc);
        strip(mine ? xlane + off * 2 : 0, off / 32, w, [&](int i, int c, float& s, float& z) {
          const int64_t g = (k + 32 * c) >> a.shift;
          s = g < a.groups ? bf16_to_f32(a.scale[srow[i] + g]) : 0.f;
          z = g < a.groups ? zero_at(a, srow[i] + g) : 0.f;
        });
      }
    }
    wait_lds();
    block_barrier();  // every wave is done with this chunk of x
  }

#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      acc[i][m] += __shfl_xor(acc[i][m], 16, kWave);
      acc[i][m] += __shfl_xor(acc[i][m], 32, kWave);
    }
  if constexpr (WK > 1) {
    // red[wave][i][m][n]: the waves' sums are added in wave order.
    constexpr int kVals = M * 16;
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (quarter == 0)
#pragma unroll
        for (int m = 0; m < M; ++m) red[(wave * NT + i) * kVals + m * 16 + ln] = acc[i][m];
    wait_lds();
    block_barrier();
    for (int idx = thread; idx < WN * NT * kVals; idx += L::kThreads) {
      const int w = idx / (NT * kVals), rest = idx % (NT * kVals);
      const int i = rest / kVals, m = rest % kVals / 16, n = rest % 16;
      if (m >= rows) continue;
      float v = red[(w * WK * NT + i) * kVals + m * 16 + n];
#pragma unroll
      for (int o = 1; o < WK; ++o) v += red[((w * WK + o) * NT + i) * kVals + m * 16 + n];
      const int at = (w * NT + i) * 16 + n;
      if (__builtin_expect(!finite(v) && n0 + at < N, 0)) v = defined(m, at);
      store(m, at, v);
    }
  } else {
    float mine[NT], sum = 0.f;  // quarter m takes row m
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      mine[i] = acc[i][0];
#pragma unroll
      for (int m = 1; m < M; ++m) mine[i] = quarter == m ? acc[i][m] : mine[i];
      sum = fmaf(mine[i], 0.f, sum);
    }
    if (quarter >= rows) return;
    const int n = wn * NT * 16 + ln;
    if (__builtin_expect(__ballot(sum != sum) == 0, 1)) {
#pragma unroll
      for (int i = 0; i < NT; ++i) store(quarter, n + i * 16, mine[i]);
      return;
    }
#pragma unroll 1
    for (int i = 0; i < NT; ++i) {  // results that are not finite among them
      float v = mine[0];
#pragma unroll
      for (int j = 1; j < NT; ++j) v = i == j ? mine[j] : v;
      if (!finite(v) && n0 + n + i * 16 < N) v = defined(quarter, n + i * 16);
      store(quarter, n + i * 16, v);
    }
  }
}

template <int M, int NT, int WN, int WK, int SH>
__global__ __launch_bounds__(64 * WN * WK) void int4_stream_kernel(Int4Args a, const uint16_t* __restrict__ x,
                                                                   void* __restrict__ out, int out_bf16, int64_t rows,
                                                                   int64_t N, int64_t K, float alpha, Epilogue epi) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int64_t n0 = int64_t(blockIdx.x) * (16 * NT * WN);
  const Int4HeadPtr head = QL_INT4_HEAD();
  int4_stream_tile<M, NT, WN, WK, SH>(lds, a, x, int(rows), N, K, n0, [&](int m, int n, float v) {
    if (n0 + n < N) store_epi(out, m, n0 + n, N, v, alpha, out_bf16, epi);
  }, [=](int m, int n) { return int4_defined(head, m, n0 + n, K); });
}

// ---------------------------------------------------------------- matrix-core tile

// A block computes BM = 16 MT rows by BN = 16 NT WN columns with 16x16x32
// MFMA.  WN waves side by side share each 128-value strip of x (int4_pipe_tile), or WK
// waves split the strips between them and add their tiles at the end (int4_tile).
//
// Weights go straight into the registers of the wave that multiplies them: lane
// (n = l % 16, quarter h = l / 16) reads the 16 bytes k = 32 h .. 32 h + 31 of its
// row's strip.  For groups of 128 and more MFMA step t takes dword t of every lane, k =
// 32 h + 8 t ..; for smaller ones two half-wave swap stages first transpose the
// 4x4 dwords over the quarters, and step t covers k = 32 t + 8 h .., one group's.
// Activation: the strip [BM][128] goes through registers into LDS as it is, 16-byte
// chunks XOR-permuted by row against bank conflicts: the vector ALU is what these
// tiles run out of, so the order of k is mended where a value is decoded once for
// the whole tile (2 instructions per 8 codes) and not where x is staged.
//
// After the last step of a group: acc += scale * group.  The zero points are
// taken off by the matrix cores too: sum_groups sum_x * (zero * scale) is a
// product over the groups.  A group's sum of x (a product with ones) is in float32, 24
// bits, which are three bfloat16 cut
// from it, hi + mid + lo, and zero * scale (8 by 8 bits) is two, both exact, so six
// of a quarter's eight k slots of one MFMA hold all products of one group,
// and four groups need one instruction per 16x16 tile; on the
// vector ALU, which the decoding and the scaling fill already, they would be 16.
constexpr int kSlots = 4;  // groups per correction

template <int MT, int NT, int WN, int WK> struct Int4Tile {
  static constexpr int kBM = 16 * MT, kBN = 16 * NT * WN, kThreads = 64 * WN * WK;
  static constexpr int kStagers = 64 * WN;                 // threads that fill one activation buffer
  static constexpr int kChunks = kBM * 16 / kStagers;      // 16-byte chunks per staging thread
  static constexpr int kXBytes = kBM * kStrip * 2;
  static constexpr int kBufs = WK > 1 ? 1 : 2;             // a wave's own buffer needs no second one
  static constexpr int kSumBytes = kSlots * kBM * 16;      // [slot][BM] pieces of the sums
  static constexpr int kSums = kXBytes * kBufs;
  static constexpr int kOne = kSums + 2 * kSumBytes;
  static constexpr int kRing = kOne * WK;
  static constexpr int kReduce = WK > 1 ? WK * 64 * MT * NT * 16 : 0;
  static constexpr int kLds = kRing > kReduce ? kRing : kReduce;
  static_assert(WK == 1 || WN == 1, "either the tile or K is split over the waves");
};

__device__ __forceinline__ float cut_bf16(float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); }

// -s as (hi, mid, lo, hi, mid, lo, 0, 0), each exact in bfloat16.
__device__ __forceinline__ u32x4 sum_pieces(float s) {
  const float hi = cut_bf16(-s), rest = -s - hi, mid = cut_bf16(rest), lo = rest - mid;
  const uint32_t h = __float_as_uint(hi), m = __float_as_uint(mid), l = __float_as_uint(lo);
  return u32x4{h >> 16 | m, l >> 16 | h, m >> 16 | (l & 0xFFFF0000u), 0u};
}
// v as (hi, hi, hi, lo, lo, lo, 0, 0).
__device__ __forceinline__ u32x4 factor_pieces(float v) {
  const float hi = cut_bf16(v);
  const uint32_t h = __float_as_uint(hi), l = __float_as_uint(v - hi) & 0xFFFF0000u;
  return u32x4{h >> 16 | h, h >> 16 | l, l >> 16 | l, 0u};
}

// Buffer loads take a 32-bit lane offset and a uniform one, without address arithmetic on
// the vector ALU.  The record count is not used as a bound: every offset lies inside.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, -1, 0x00020000);
}

// GS: MFMA steps per group inside a strip (1, 2, 4; 4 also for larger groups).
// The waves share nothing until they add their tiles, so that none waits for another: this is
// the form for few rows, where a tile's time is the memory's answer.
// store(m, n, value): m and n relative to the tile; defined(m, n): the value of a result that is not finite.  Every
// thread of the block calls it; the block's LDS is free when it begins.
template <int MT, int NT, int WK, int GS, typename Store, typename Defined>
__device__ __forceinline__ void int4_tile(char* lds, const Int4Args& a, const uint16_t* __restrict__ x, int64_t rows,
                                          int64_t N, int64_t K, int64_t n0, Store&& store, Defined&& defined) {
  using L = Int4Tile<MT, NT, 1, WK>;
  constexpr int G = 4 / GS;  // groups per strip
  const int lane = threadIdx.x & (kWave - 1), wk = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int ln = lane & 15, quarter = lane >> 4;
  const int nstrips = int((K + kStrip - 1) / kStrip), nwhole = int(K / kStrip);
  char* const mem = lds + wk * L::kOne;

  // Uniform bases and 32-bit lane offsets (K < 2^23).
  const uint8_t* const wbase = a.w + n0 * a.row_bytes;
  const uint16_t* const sbase = a.scale + n0 * a.groups;
  // Without zero points the scales' bytes are read in their place and not used.
  const uint8_t* const zbase = (a.zero ? a.zero : reinterpret_cast<const uint8_t*>(a.scale)) + n0 * a.groups;
  const __amdgpu_buffer_rsrc_t wbuf = buffer_at(wbase), sbuf_ = buffer_at(sbase), zbuf = buffer_at(zbase), xbuf = buffer_at(x);
  uint32_t woff[NT], soff[NT], xoff[L::kChunks];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int n = i * 16 + ln;
    const uint32_t row = n0 + n < N ? n : uint32_t(N - 1 - n0);  // columns past N re-read the last row, never stored
    woff[i] = row * uint32_t(a.row_bytes) + quarter * 16;
    soff[i] = row * uint32_t(a.groups);
  }
#pragma unroll
  for (int j = 0; j < L::kChunks; ++j) {
    const int m = (lane + j * kWave) >> 4;
    xoff[j] = uint32_t(m < rows ? m : rows - 1) * uint32_t(K) * 2 + (lane & 15) * 16;  // rows past the end likewise
  }

  // A strip's G groups of a row are neighbours: their scales come in one load
  // and stay packed, and so do their zero points.
  u32x4 wreg[NT], xreg[L::kChunks];
  uint32_t sreg[NT][2];
  uint16_t shalf[NT];  // in place of sreg where G = 1
  uint32_t zreg[NT];

  // A whole strip: no lane branches, so that nothing waits for a load before
  // the strip after this one is staged.
  auto fetch = [&](int strip) {
    const int at = int((int64_t(strip) * kStrip) >> a.shift);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      wreg[i] = __builtin_amdgcn_raw_buffer_load_b128(wbuf, woff[i], strip * (kStrip / 2), 0);
      if constexpr (G == 4) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(sbuf_, soff[i] * 2, at * 2, 0);
        sreg[i][0] = v.x;
        sreg[i][1] = v.y;
        zreg[i] = __builtin_amdgcn_raw_buffer_load_b32(zbuf, soff[i], at, 0);
      } else if constexpr (G == 2) {
        sreg[i][0] = __builtin_amdgcn_raw_buffer_load_b32(sbuf_, soff[i] * 2, at * 2, 0);
        zreg[i] = __builtin_amdgcn_raw_buffer_load_b16(zbuf, soff[i], at, 0);
      } else {
        shalf[i] = __builtin_amdgcn_raw_buffer_load_b16(sbuf_, soff[i] * 2, at * 2, 0);
        zreg[i] = __builtin_amdgcn_raw_buffer_load_b8(zbuf, soff[i], at, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j)
      xreg[j] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, xoff[j], strip * (kStrip * 2), 0);
  };
  // The last, partial strip: zeros behind K, and groups past K are nothing,
  // whatever lies there.
  auto fetch_tail = [&](int strip) {
    const int64_t k = int64_t(strip) * kStrip, at = k >> a.shift;
    const int left = int(K - k);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int codes = left - quarter * 32;
      const uint8_t* p = wbase + (k >> 1) + woff[i];
      wreg[i] = codes >= 31 ? ldw16(p) : ld_bytes(p, (codes + 1) >> 1);
      const int groups = int(a.groups - at < G ? a.groups - at : G);
      const u32x4 v = ld_halves(sbase + at + soff[i], groups);
      sreg[i][0] = v.x;
      sreg[i][1] = v.y;
      shalf[i] = uint16_t(v.x);
      zreg[i] = ld_bytes(zbase + at + soff[i], groups).x;
    }
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j) {
      const int values = left - (lane & 15) * 8;
      const uint16_t* p = x + k + (xoff[j] >> 1);
      xreg[j] = values >= 8 ? ldx16(p) : ld_halves(p, values);
    }
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[mt][i] = v4f{0.f, 0.f, 0.f, 0.f};
  float zs[NT], due[NT];  // zero * scale of this quarter's slot: being filled, and of full slots
#pragma unroll
  for (int i = 0; i < NT; ++i) zs[i] = due[i] = 0.f;
  for (int i = lane; i < 2 * L::kSumBytes / 16; i += kWave)
    *reinterpret_cast<u32x4*>(mem + L::kSums + i * 16) = u32x4{0u, 0u, 0u, 0u};

  auto correct = [&](const char* sums) {
    v8bf zb[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) zb[i] = __builtin_bit_cast(v8bf, factor_pieces(due[i]));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const v8bf xb = *reinterpret_cast<const v8bf*>(sums + (quarter * L::kBM + mt * 16 + ln) * 16);
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, zb[i], acc[mt][i], 0, 0, 0);
    }
  };
  // Where row `row` keeps what a quarter's slots of step t hold.  A read of 64 lanes is free of
  // bank conflicts if the quarters differ in the low bits of the place, so where quarter q reads chunk
  // 4 q + t (groups of 128 and more) the two halves of the chunk's number change places.
  auto place = [&](int row, int t) { return row * (kStrip * 2) + (((t * 4 + quarter) ^ ln) << 4); };

  // slot, sbuf: the strip's first group's slot and the slots' buffer.  Sums are made while
  // their strip is multiplied, and full slots are due in the next.
  int slot = 0, sbuf = 0;
  bool full = false;
  if (wk < nwhole) fetch(wk);
  for (int strip = wk; strip < nstrips; strip += WK) {
    if (strip >= nwhole) fetch_tail(strip);
    // What is made of the loaded values is made from here on: the compiler
    // would move the first shift of a scale behind its load, where it waits for memory
    // in every strip.
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if constexpr (G == 1) asm volatile("" : "+v"(shalf[i]), "+v"(zreg[i]));
      else asm volatile("" : "+v"(sreg[i][0]), "+v"(zreg[i]));
      if constexpr (G == 4) asm volatile("" : "+v"(sreg[i][1]));
    }
    char* const xs = mem;
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j) {
      const int idx = lane + j * kWave, m = idx >> 4, c = idx & 15;
      const int p = GS == 4 ? (c & 3) * 4 + (c >> 2) : c;
      *reinterpret_cast<u32x4*>(xs + m * (kStrip * 2) + ((p ^ (m & 15)) << 4)) = xreg[j];
    }
    u32x4 w[NT];
    uint32_t sp[NT][2];
    v8bf codes[NT][GS];
    auto scale = [&](int i, int g) { return __uint_as_float((g & 1) ? sp[i][g >> 1] & 0xFFFF0000u : sp[i][g >> 1] << 16); };
    auto decode = [&](int g) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < GS; ++t) codes[i][t] = __builtin_bit_cast(v8bf, int4x8_to_bf16x8_ordered(w[i][g * GS + t]));
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      w[i] = GS == 4 ? wreg[i] : transpose_quarters(wreg[i]);
      sp[i][0] = G == 1 ? shalf[i] : sreg[i][0];
      if constexpr (G == 4) sp[i][1] = sreg[i][1];
      if (!a.zero) zreg[i] = 0x08080808u;
#pragma unroll
      for (int g = 0; g < G; ++g) zs[i] = quarter == slot + g ? scale(i, g) * float((zreg[i] >> (8 * g)) & 255u) : zs[i];
    }
    decode(0);
    if (strip + WK < nwhole) fetch(strip + WK);
    wait_lds();
    // The sums of x over the strip's groups.
    char* sums = mem + L::kSums + sbuf * L::kSumBytes;
    const v8bf ones = __builtin_bit_cast(v8bf, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
#pragma unroll
    for (int tile = 0; tile < MT; ++tile) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        v4f total{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = g * GS; t < (g + 1) * GS; ++t)
          total = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              *reinterpret_cast<const v8bf*>(xs + place(tile * 16 + ln, t)), ones, total, 0, 0, 0);
        const float mine = (ln & 2) ? ((ln & 1) ? total[3] : total[2]) : ((ln & 1) ? total[1] : total[0]);
        if (ln < 4)
          *reinterpret_cast<u32x4*>(sums + ((slot + g) * L::kBM + tile * 16 + quarter * 4 + ln) * 16) = sum_pieces(mine);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g > 0) decode(g);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        v4f part[NT];
#pragma unroll
        for (int t = 0; t < GS; ++t) {
          const v8bf xa = *reinterpret_cast<const v8bf*>(xs + place(mt * 16 + ln, g * GS + t));
#pragma unroll
          for (int i = 0; i < NT; ++i)
            part[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa, codes[i][t], t == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : part[i],
                                                              0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float s = scale(i, g);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[mt][i][r] = fmaf(s, part[i][r], acc[mt][i][r]);
        }
      }
    }
    if (full) correct(mem + L::kSums + (sbuf ^ 1) * L::kSumBytes);
    slot += G;
    full = slot == kSlots;
    if (full) {
      slot = 0;
      sbuf ^= 1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        due[i] = zs[i];
        zs[i] = 0.f;
      }
    }
  }
  wait_lds();
  if (full) {
    correct(mem + L::kSums + (sbuf ^ 1) * L::kSumBytes);
  } else if (slot > 0) {  // unfilled slots have zs = 0 and finite sums
#pragma unroll
    for (int i = 0; i < NT; ++i) due[i] = zs[i];
    correct(mem + L::kSums + sbuf * L::kSumBytes);
  }

  // Add the waves' tiles in wave order: each wave leaves its tile in LDS
  // (one 16-byte store per lane and 16x16 tile) and takes one.
  __syncthreads();
  v4f* red = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < NT; ++i) red[((wk * MT + mt) * NT + i) * 64 + lane] = acc[mt][i];
  __syncthreads();
  static_assert(MT * NT <= WK, "a 16x16 tile per wave at most");
  if (wk >= MT * NT) return;
  v4f v = red[wk * 64 + lane];
#pragma unroll
  for (int o = 1; o < WK; ++o) {
    const v4f b = red[(o * MT * NT + wk) * 64 + lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += b[r];
  }
  const int m = (wk / NT) * 16 + quarter * 4, n = (wk % NT) * 16 + ln;
  const float sum = fmaf(v[0], 0.f, fmaf(v[1], 0.f, fmaf(v[2], 0.f, v[3] * 0.f)));
  if (__builtin_expect(__ballot(sum != sum) == 0, 1)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) store(m + r, n, v[r]);
    return;
  }
#pragma unroll 1
  for (int r = 0; r < 4; ++r) {  // results that are not finite among them
    float f = r == 0 ? v[0] : r == 1 ? v[1] : r == 2 ? v[2] : v[3];
    if (!finite(f) && m + r < rows && n0 + n < N) f = defined(m + r, n);
    store(m + r, n, f);
  }
}

// A tile's way out: `out` [rows, N] from row 0, column n0 of the tile on.  Plain results
// leave through buffers whose record count ends with the last row, so that neither rows nor
// columns need a branch: a column past N gets an offset past the end, and a row past the last one has
// it.  Each 16 rows have a buffer of their own, beginning at their first row: the hardware's check takes the lane's
// offset against the count less the scalar offset, so a row in the scalar offset would be past the count
// itself, where the difference is no longer a bound.  3 instructions per value where the general
// store takes 25, which for 128x256 were 5 us.  With an epilogue, or where a tile spans 2 GiB, values go
// one by one.
struct TileOut {
  void* out;      // row 0, column 0
  int64_t rows, N, n0;
  int64_t row0;   // of the epilogue's operands and of x
  int64_t wrow0;  // of the expert among the weights
  float alpha;
  int bf16;
  Epilogue epi;
  Int4HeadPtr head;

  // acc[mt][i]: rows 16 mt .., columns wave_n + 16 i ..; K for the results that are not finite.
  template <int MT, int NT>
  __device__ __forceinline__ void write(const v4f (&acc)[MT][NT], int wave_n, int64_t K) const {
    constexpr int BM = 16 * MT;
    static_assert(MT * NT * 4 <= 64, "a bit per result of a lane");
    const int lane = threadIdx.x & (kWave - 1), ln = lane & 15, quarter = lane >> 4;
    const int64_t es = bf16 ? 2 : 4;
    const bool plain = !epi.on && int64_t(BM) * N * es < (int64_t(1) << 31);
    float sum = 0.f;  // NaN if a result is not finite
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum = fmaf(acc[mt][i][r], 0.f, sum);
    if (plain) {
      const int live = int(rows < BM ? rows : BM);
      char* const first = static_cast<char*>(out) + n0 * es;
      const uint32_t line = uint32_t(N * es), lane_at = uint32_t(quarter * 4) * line + uint32_t((wave_n + ln) * es);
      const int64_t width = N - n0 - wave_n - ln;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int m = 16 * mt;
        const uint32_t bytes = m < live ? uint32_t(live - m) * line - uint32_t(n0 * es) : 0u;
        const __amdgpu_buffer_rsrc_t buf =
            __builtin_amdgcn_make_buffer_rsrc(first + int64_t(m) * line, 0, int(bytes), 0x00020000);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint32_t at = 16 * i < width ? lane_at + uint32_t(16 * i * es) : 0x80000000u;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float f = acc[mt][i][r] * alpha;
            if (bf16)
              __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, static_cast<__bf16>(f)), buf,
                                                    at + uint32_t(r) * line, 0, 0);
            else
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f), buf, at + uint32_t(r) * line, 0, 0);
          }
        }
      }
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t row = mt * 16 + quarter * 4 + r, col = n0 + wave_n + i * 16 + ln;
            // The residual may be the output: a result that follows below is not stored before.
            if (row < rows && col < N && finite(acc[mt][i][r])) put(row, col, acc[mt][i][r]);
          }
    }
    if (__builtin_expect(__ballot(sum != sum) == 0, 1)) return;
    uint64_t lost = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) lost |= uint64_t(!finite(acc[mt][i][r])) << ((mt * NT + i) * 4 + r);
    const int again = own_thread();
    for (; lost; lost &= lost - 1) {
      const int b = __builtin_ctzll(lost), tile = b >> 2;
      const int64_t row = tile / NT * 16 + (again & 63) / 16 * 4 + (b & 3), col = n0 + wave_n + tile % NT * 16 + (again & 15);
      if (row < rows && col < N) put(row, col, int4_defined(head, row0 + row, wrow0 + col, K));
    }
  }

  __device__ __forceinline__ void put(int64_t row, int64_t col, float v) const {
    float f = v * alpha;
    if (epi.on) f = epi_apply(epi, f, row0 + row, col);
    store_out(out, row * N + col, f, 1.f, bf16);
  }
};

// The same product with every wave's work in flight at once, for tiles that use all of a
// CU's registers: while the matrix cores run strip s, the wave decodes the codes of strip
// s + 1, moves its x from registers to the other LDS buffer, and loads strip s + 2.  WN waves
// side by side along N, one barrier per strip.  (With these phases one after the other
// the 128x256 tile took 2.9 us for a strip of which the matrix cores need 1.1.)
// Bound by what the 2 waves of a SIMD issue in turn: decoding, and scaling, which grows with the groups of
// a strip, overlap little with the matrix cores' work.  128x256 with groups of 128, 64, 32: vector
// instructions (the matrix ones among them) are issued in 38, 46, 56 % of the SIMDs' cycles, the matrix cores work in
// 39, 35, 31 %, and under 5 % of the waves' cycles are waits to issue LDS instructions.
// M = 500, N = 14336, K = 4096: 82, 98 (600 TFLOP/s), 121 us, calls behind each other with the
// weights in the 256 MB cache; groups of 64, no weights there: 108.
// With four strips' loads under way the smaller tiles gained nothing (64x256 58 us for 54).
template <int MT, int NT, int WN, int GS>
__device__ __forceinline__ void int4_pipe_tile(char* lds, const Int4Args& a, const uint16_t* __restrict__ x,
                                               int64_t rows, int64_t N, int64_t K, int64_t n0, const TileOut& to) {
  using L = Int4Tile<MT, NT, WN, 1>;
  constexpr int G = 4 / GS;  // groups per strip
  const int thread = own_thread();
  const int lane = thread & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(thread / kWave);
  const int ln = lane & 15, quarter = lane >> 4;
  const int nwhole = int(K / kStrip);

  // Uniform bases and 32-bit lane offsets (K < 2^23).
  const uint8_t* const wbase = a.w + n0 * a.row_bytes;
  const uint16_t* const sbase = a.scale + n0 * a.groups;
  // Without zero points the scales' bytes are read in their place and not used.
  const uint8_t* const zbase = (a.zero ? a.zero : reinterpret_cast<const uint8_t*>(a.scale)) + n0 * a.groups;
  const __amdgpu_buffer_rsrc_t wbuf = buffer_at(wbase), scbuf = buffer_at(sbase), zbuf = buffer_at(zbase), xbuf = buffer_at(x);
  uint32_t woff[NT], soff[NT], xoff[L::kChunks];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int n = wave * 16 * NT + i * 16 + ln;
    const uint32_t row = n0 + n < N ? n : uint32_t(N - 1 - n0);  // columns past N re-read the last row, never stored
    woff[i] = row * uint32_t(a.row_bytes) + quarter * 16;
    soff[i] = row * uint32_t(a.groups);
  }
#pragma unroll
  for (int j = 0; j < L::kChunks; ++j) {
    const int m = (thread + j * L::kThreads) >> 4;
    xoff[j] = uint32_t(m < rows ? m : rows - 1) * uint32_t(K) * 2 + (thread & 15) * 16;  // rows past the end likewise
  }

  // A strip's weights as they come; its G groups' scales and zero points stay packed.
  struct Raw {
    u32x4 w[NT];
    uint32_t s[NT][2];
    uint32_t z[NT];
    uint16_t half[NT], zhalf[NT];  // in place of s where G = 1, of z where G < 4
  };
  // Decoded: MFMA operands and packed scales.
  struct Codes {
    v8bf b[NT][4];
    uint32_t s[NT][2];
    __device__ __forceinline__ float scale(int i, int g) const {
      if constexpr (G == 1) return __uint_as_float(s[i][0]);
      else return __uint_as_float((g & 1) ? s[i][g >> 1] & 0xFFFF0000u : s[i][g >> 1] << 16);
    }
  };
  u32x4 xreg[L::kChunks];
  auto fetch_w = [&](Raw& f, int strip) {
    const int at = int((int64_t(strip) * kStrip) >> a.shift);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f.w[i] = __builtin_amdgcn_raw_buffer_load_b128(wbuf, woff[i], strip * (kStrip / 2), 0);
      if constexpr (G == 4) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(scbuf, soff[i] * 2, at * 2, 0);
        f.s[i][0] = v.x;
        f.s[i][1] = v.y;
        f.z[i] = __builtin_amdgcn_raw_buffer_load_b32(zbuf, soff[i], at, 0);
      } else if constexpr (G == 2) {
        f.s[i][0] = __builtin_amdgcn_raw_buffer_load_b32(scbuf, soff[i] * 2, at * 2, 0);
        f.zhalf[i] = __builtin_amdgcn_raw_buffer_load_b16(zbuf, soff[i], at, 0);
      } else {
        f.half[i] = __builtin_amdgcn_raw_buffer_load_b16(scbuf, soff[i] * 2, at * 2, 0);
        f.zhalf[i] = __builtin_amdgcn_raw_buffer_load_b8(zbuf, soff[i], at, 0);
      }
    }
  };
  auto fetch_x = [&](int strip) {
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j)
      xreg[j] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, xoff[j], strip * (kStrip * 2), 0);
  };
  // The last, partial strip: zeros behind K, and groups past K are nothing,
  // whatever lies there.
  auto fetch_tail = [&](Raw& f, int strip) {
    const int64_t k = int64_t(strip) * kStrip, at = k >> a.shift;
    const int left = int(K - k);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int codes = left - quarter * 32;
      const uint8_t* p = wbase + (k >> 1) + woff[i];
      f.w[i] = codes >= 31 ? ldw16(p) : ld_bytes(p, (codes + 1) >> 1);
      const int groups = int(a.groups - at < G ? a.groups - at : G);
      const u32x4 v = ld_halves(sbase + at + soff[i], groups);
      f.s[i][0] = v.x;
      f.s[i][1] = v.y;
      f.half[i] = uint16_t(v.x);
      f.z[i] = ld_bytes(zbase + at + soff[i], groups).x;
      f.zhalf[i] = uint16_t(f.z[i]);
    }
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j) {
      const int values = left - (thread & 15) * 8;
      const uint16_t* p = x + k + (xoff[j] >> 1);
      xreg[j] = values >= 8 ? ldx16(p) : ld_halves(p, values);
    }
  };
  auto stage_x = [&](int buf) {
#pragma unroll
    for (int j = 0; j < L::kChunks; ++j) {
      const int idx = thread + j * L::kThreads, m = idx >> 4, c = idx & 15;
      const int p = GS == 4 ? (c & 3) * 4 + (c >> 2) : c;
      *reinterpret_cast<u32x4*>(lds + buf * L::kXBytes + m * (kStrip * 2) + ((p ^ (m & 15)) << 4)) = xreg[j];
    }
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[mt][i] = v4f{0.f, 0.f, 0.f, 0.f};
  // zero * scale of this quarter's slot: of the slots being filled, and of full ones.  The
  // sums of a strip are made while it is multiplied, so full slots are due in the next strip.
  float zs[NT], due[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) zs[i] = due[i] = 0.f;
  for (int i = thread; i < 2 * L::kSumBytes / 16; i += L::kThreads)
    *reinterpret_cast<u32x4*>(lds + L::kSums + i * 16) = u32x4{0u, 0u, 0u, 0u};
  auto correct = [&](const char* sums) {
    v8bf zb[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) zb[i] = __builtin_bit_cast(v8bf, factor_pieces(due[i]));
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const v8bf xb = *reinterpret_cast<const v8bf*>(sums + (quarter * L::kBM + mt * 16 + ln) * 16);
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[mt][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, zb[i], acc[mt][i], 0, 0, 0);
    }
  };
  // Where row `row` keeps what a quarter's slots of step t hold.  A read of 64 lanes is free of
  // bank conflicts if the quarters differ in the low bits of the place, so where quarter q reads chunk
  // 4 q + t (groups of 128 and more) the two halves of the chunk's number change places.
  auto place = [&](int row, int t) { return row * (kStrip * 2) + (((t * 4 + quarter) ^ ln) << 4); };

  // Before a strip's codes: `slot` its first group's; live: the strip exists (else nothing is noted).
  const uint32_t zkeep = a.zero ? 0xFFFFFFFFu : 0u, zset = a.zero ? 0u : 0x08080808u;
  auto begin = [&](Raw& f, Codes& c, int slot, bool live) {
    const int first = live ? slot : kSlots;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      // What is made of the loaded values is made from here on: the compiler would
      // widen a scale or a zero point behind its load, where it waits for memory.
      uint32_t z;
      if constexpr (G == 1) {
        asm volatile("v_lshlrev_b32 %0, 16, %1" : "=v"(c.s[i][0]) : "v"(f.half[i]));
      } else {
        asm volatile("" : "+v"(f.s[i][0]));
        c.s[i][0] = f.s[i][0];
      }
      if constexpr (G == 4) {
        asm volatile("" : "+v"(f.s[i][1]), "+v"(f.z[i]));
        c.s[i][1] = f.s[i][1];
        z = f.z[i];
      } else {
        asm volatile("v_mov_b32 %0, %1" : "=v"(z) : "v"(f.zhalf[i]));  // only its first G bytes are used
      }
      if constexpr (GS < 4) f.w[i] = transpose_quarters(f.w[i]);
      z = (z & zkeep) | zset;
#pragma unroll
      for (int g = 0; g < G; ++g)
        zs[i] = quarter == first + g ? c.scale(i, g) * float((z >> (8 * g)) & 255u) : zs[i];
    }
  };
  auto decode = [&](const Raw& f, Codes& c, int d) {
    c.b[d / 4][d % 4] = __builtin_bit_cast(v8bf, int4x8_to_bf16x8_ordered(f.w[d / 4][d % 4]));
  };
  // Sums of x over the groups of the strip in buffer `buf`, row tiles dealt to the waves.
  auto sum_x = [&](int buf, int set, int slot) {
    const char* xs = lds + buf * L::kXBytes;
    char* sums = lds + L::kSums + set * L::kSumBytes;
    const v8bf ones = __builtin_bit_cast(v8bf, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
#pragma unroll
    for (int q = 0; q < (MT + WN - 1) / WN; ++q) {
      const int tile = wave + q * WN;
      if (MT % WN != 0 && tile >= MT) break;  // uniform
#pragma unroll
      for (int g = 0; g < G; ++g) {
        v4f total{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = g * GS; t < (g + 1) * GS; ++t)
          total = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              *reinterpret_cast<const v8bf*>(xs + place(tile * 16 + ln, t)), ones, total, 0, 0, 0);
        const float mine = (ln & 2) ? ((ln & 1) ? total[3] : total[2]) : ((ln & 1) ? total[1] : total[0]);
        if (ln < 4)
          *reinterpret_cast<u32x4*>(sums + ((slot + g) * L::kBM + tile * 16 + quarter * 4 + ln) * 16) = sum_pieces(mine);
      }
    }
  };
  // A row tile's x is read while the one before it is multiplied; between(mt) runs after each.
  auto multiply = [&](int buf, const Codes& c, auto&& between) {
    const char* xs = lds + buf * L::kXBytes;
    v8bf xa[2][4];
    auto read = [&](int mt) {
#pragma unroll
      for (int t = 0; t < 4; ++t) xa[mt & 1][t] = *reinterpret_cast<const v8bf*>(xs + place(mt * 16 + ln, t));
    };
    read(0);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt + 1 < MT) read(mt + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        v4f part[NT];
#pragma unroll
        for (int t = 0; t < GS; ++t)
#pragma unroll
          for (int i = 0; i < NT; ++i)
            part[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xa[mt & 1][g * GS + t], c.b[i][g * GS + t],
                                                              t == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : part[i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float s = c.scale(i, g);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[mt][i][r] = fmaf(s, part[i][r], acc[mt][i][r]);
        }
      }
      between(mt);
    }
  };

  int slot = 0, set = 0;  // of the strip being multiplied
  bool ready = false;     // the other set's slots are due
  constexpr int D = NT * 4;
  auto advance = [&]() {
    slot += G;
    ready = slot == kSlots;
    if (ready) {
      slot = 0;
      set ^= 1;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        due[i] = zs[i];
        zs[i] = 0.f;
      }
    }
  };
  // One strip: r0 receives strip s + 2, r1 holds s + 1, c the codes of s; n gets those of s + 1.
  auto step = [&](int s, Raw& r0, Raw& r1, const Codes& c, Codes& n) {
    const int buf = s & 1;
    stage_x(buf ^ 1);
    const int next2 = s + 2 < nwhole ? s + 2 : nwhole - 1;  // past the end: the last one again, not used
    fetch_x(next2);
    fetch_w(r0, next2);
    if (ready) correct(lds + L::kSums + (set ^ 1) * L::kSumBytes);
    sum_x(buf, set, slot);
    advance();
    begin(r1, n, slot, s + 1 < nwhole);
    multiply(buf, c, [&](int mt) {
#pragma unroll
      for (int d = mt * D / MT; d < (mt + 1) * D / MT; ++d) decode(r1, n, d);
    });
    wait_lds();
    block_barrier();
  };
  Raw r0, r1;
  Codes c0, c1;
  if (nwhole > 0) {
    fetch_x(0);
    fetch_w(r0, 0);
    stage_x(0);
    fetch_x(nwhole > 1 ? 1 : 0);
    fetch_w(r1, nwhole > 1 ? 1 : 0);
    begin(r0, c0, 0, true);
#pragma unroll
    for (int d = 0; d < D; ++d) decode(r0, c0, d);
  }
  wait_lds();
  block_barrier();
  for (int s = 0; s < nwhole; s += 2) {
    step(s, r0, r1, c0, c1);
    if (s + 1 < nwhole) step(s + 1, r1, r0, c1, c0);
  }
  if (K % kStrip != 0) {
    if (ready) correct(lds + L::kSums + (set ^ 1) * L::kSumBytes);
    const int buf = nwhole & 1;
    fetch_tail(r0, nwhole);
    stage_x(buf);  // every wave is done with the strips before it
    begin(r0, c0, slot, true);
#pragma unroll
    for (int d = 0; d < D; ++d) decode(r0, c0, d);
    wait_lds();
    block_barrier();
    sum_x(buf, set, slot);
    advance();
    multiply(buf, c0, [](int) {});
    wait_lds();
    block_barrier();
  }
  if (ready) {
    correct(lds + L::kSums + (set ^ 1) * L::kSumBytes);
  } else if (slot > 0) {  // unfilled slots have zs = 0 and finite sums
#pragma unroll
    for (int i = 0; i < NT; ++i) due[i] = zs[i];
    correct(lds + L::kSums + set * L::kSumBytes);
  }
  to.write(acc, wave * 16 * NT, K);
}

template <int MT, int NT, int WN, int WK, int GS>
__global__ __launch_bounds__(64 * WN * WK) void int4_gemm_kernel(Int4Args a, const uint16_t* __restrict__ x,
                                                                 void* __restrict__ out, int out_bf16, int64_t M,
                                                                 int64_t N, int64_t K, float alpha, Epilogue epi) {
  using L = Int4Tile<MT, NT, WN, WK>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // Row tiles of one column tile follow each other on one XCD, whose L2 then
  // holds the column tile's weights.
  const int64_t mtiles = (M + L::kBM - 1) / L::kBM, ntiles = (N + L::kBN - 1) / L::kBN, total = mtiles * ntiles;
  const int64_t per = (total + 7) / 8;
  const int64_t tile = int64_t(blockIdx.x % 8) * per + blockIdx.x / 8;
  if (int64_t(blockIdx.x / 8) >= per || tile >= total) return;  // uniform over the block
  const int64_t m0 = tile % mtiles * L::kBM, n0 = tile / mtiles * L::kBN;
  const Int4HeadPtr head = QL_INT4_HEAD();
  if constexpr (WK == 1) {
    const TileOut to{static_cast<char*>(out) + m0 * N * (out_bf16 ? 2 : 4), M - m0, N, n0, m0, 0, alpha, out_bf16, epi, head};
    int4_pipe_tile<MT, NT, WN, GS>(lds, a, x + m0 * K, M - m0, N, K, n0, to);
  } else {
    int4_tile<MT, NT, WK, GS>(lds, a, x + m0 * K, M - m0, N, K, n0, [&](int m, int n, float v) {
      if (m0 + m < M && n0 + n < N) store_epi(out, m0 + m, n0 + n, N, v, alpha, out_bf16, epi);
    }, [=](int m, int n) { return int4_defined(head, m0 + m, n0 + n, K); });
  }
}

// Grouped: group z owns rows a_offsets[z] .. a_offsets[z + 1] - 1 (clipped to
// T) and multiplies them by expert expert_ids[z]; an id outside 0 .. E - 1
// writes zeros, an empty group nothing.  Every block builds the prefix sum of
// the groups' row tiles in LDS (cum[z] = row tiles of groups 0 .. z - 1) and walks its XCD's
// contiguous part of the (group, row tile, column tile) list.
// f(expert's operands, the expert, m0, rows from m0 to the group's end, n0).
template <int BM, int BN, int THREADS, typename F>
__device__ __forceinline__ void walk_groups(int* cum, const Int4Args& a, const uint32_t* __restrict__ a_offsets,
                                            const int32_t* __restrict__ expert_ids, void* __restrict__ out, int out_bf16,
                                            int64_t groups, int64_t T, int64_t N, int64_t E, F&& f) {
  auto span = [&](int64_t z, int64_t& start, int64_t& rows) {
    int64_t b = a_offsets[z], e = a_offsets[z + 1];
    b = b < T ? b : T;
    e = e < T ? e : T;
    start = b;
    rows = e > b ? e - b : 0;
  };
  if (threadIdx.x < kWave) count_group_tiles<BM>(cum, a_offsets, groups, T);
  __syncthreads();
  const int64_t ntiles = (N + BN - 1) / BN, work = int64_t(__builtin_amdgcn_readfirstlane(cum[groups])) * ntiles;
  const int64_t xcd = blockIdx.x % 8, per_xcd = gridDim.x / 8;  // gridDim.x is a multiple of 8
  const int64_t first = xcd * work / 8, last = (xcd + 1) * work / 8;
  for (int64_t i = first + blockIdx.x / 8; i < last; i += per_xcd) {
    const int mt = int(i / ntiles);
    const int64_t n0 = i % ntiles * BN;
    int64_t lo = 0, hi = groups;  // cum[lo] <= mt < cum[hi]
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (cum[mid] <= mt) lo = mid;
      else hi = mid;
    }
    // What was read from LDS is uniform, which the tile's scalar bases rest on.
    lo = __builtin_amdgcn_readfirstlane(int(lo));
    const int before = __builtin_amdgcn_readfirstlane(cum[lo]);
    int64_t start, rows;
    span(lo, start, rows);
    const int64_t m0 = start + int64_t(mt - before) * BM, left = start + rows - m0;
    const int64_t e = expert_ids[lo];
    if (e < 0 || e >= E) {
      for (int idx = threadIdx.x; idx < BM * BN; idx += THREADS)
        if (idx / BN < left && n0 + idx % BN < N) store_out(out, (m0 + idx / BN) * N + n0 + idx % BN, 0.f, 1.f, out_bf16);
      continue;
    }
    Int4Args b = a;
    b.w += e * N * a.row_bytes;
    b.scale += e * N * a.groups;
    if (b.zero) b.zero += e * N * a.groups;
    __syncthreads();  // the previous tile's buffers are free
    f(b, e, m0, left, n0);
  }
}

template <int MT, int NT, int WN, int GS>
__global__ __launch_bounds__(64 * WN) void int4_grouped_kernel(Int4Args a, const uint16_t* __restrict__ x,
                                                               const uint32_t* __restrict__ a_offsets,
                                                               const int32_t* __restrict__ expert_ids,
                                                               void* __restrict__ out, int out_bf16, int64_t groups,
                                                               int64_t T, int64_t N, int64_t K, int64_t E) {
  using L = Int4Tile<MT, NT, WN, 1>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Int4HeadPtr head = QL_INT4_HEAD();
  walk_groups<L::kBM, L::kBN, L::kThreads>(
      reinterpret_cast<int*>(lds + L::kLds), a, a_offsets, expert_ids, out, out_bf16, groups, T, N, E,
      [&](const Int4Args& b, int64_t e, int64_t m0, int64_t left, int64_t n0) {
        const TileOut to{static_cast<char*>(out) + m0 * N * (out_bf16 ? 2 : 4), left, N, n0, m0, e * N, 1.f, out_bf16, Epilogue{}, head};
        int4_pipe_tile<MT, NT, WN, GS>(lds, b, x + m0 * K, left, N, K, n0, to);
      });
}

// Groups of few rows: tiles of 4 rows through the streaming form, 3 waves per SIMD: with 4, 50 to
// 150 bytes of a lane's step went to memory (64 experts, N = 1536, K = 2048, groups of 128, no weights in the caches:
// 64 rows 35 us, with 3 29; 256 rows 44 and 40; with 3 and a fourth block per CU 30 and 48).
constexpr int kStreamWaves = 3;

template <int NT, int WN, int SH>
__global__ __launch_bounds__(64 * WN, kStreamWaves) void int4_grouped_stream_kernel(Int4Args a, const uint16_t* __restrict__ x,
                                                                         const uint32_t* __restrict__ a_offsets,
                                                                         const int32_t* __restrict__ expert_ids,
                                                                         void* __restrict__ out, int out_bf16,
                                                                         int64_t groups, int64_t T, int64_t N, int64_t K,
                                                                         int64_t E) {
  using L = StreamLayout<4, NT, WN, 1>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const Int4HeadPtr head = QL_INT4_HEAD();
  walk_groups<4, 16 * NT * WN, 64 * WN>(
      reinterpret_cast<int*>(lds + L::kLds), a, a_offsets, expert_ids, out, out_bf16, groups, T, N, E,
      [&](const Int4Args& b, int64_t e, int64_t m0, int64_t left, int64_t n0) {
        int4_stream_tile<4, NT, WN, 1, SH>(lds, b, x + m0 * K, int(left < 4 ? left : 4), N, K, n0, [&](int m, int n, float v) {
          if (n0 + n < N) store_out(out, (m0 + m) * N + n0 + n, v, 1.f, out_bf16);
        }, [=](int m, int n) { return int4_defined(head, m0 + m, e * N + n0 + n, K); });
      });
}

// ---------------------------------------------------------------- launch

Int4Args make_args(const uint8_t* w, const uint16_t* scale, const uint8_t* zero, int64_t K, int64_t group) {
  group = std::min(group, K);  // one group per row may be asked for with any larger value: K + group could overflow
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

template <typename F>
hipError_t by_shift(const Int4Args& a, F&& go) {
  if (a.shift == 5) return go(std::integral_constant<int, 5>{});
  if (a.shift == 6) return go(std::integral_constant<int, 6>{});
  if (a.shift == 7) return go(std::integral_constant<int, 7>{});
  return go(std::integral_constant<int, 8>{});
}

template <int M, int NT, int WN, int WK>
hipError_t stream_cfg(const Int4Args& a, const uint16_t* x, void* out, int bf16, int64_t rows, int64_t N, int64_t K,
                      float alpha, const Epilogue& epi, hipStream_t s) {
  using L = StreamLayout<M, NT, WN, WK>;
  const int64_t blocks = (N + 16 * NT * WN - 1) / (16 * NT * WN);
  if (blocks * L::kThreads >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  return by_shift(a, [&](auto sh) -> hipError_t {
    auto kernel = int4_stream_kernel<M, NT, WN, WK, decltype(sh)::value>;
    static std::atomic<uint64_t> lds_set{0};
    if (hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), L::kLds, lds_set)) return e;
    return launch(kernel, dim3(unsigned(blocks)), dim3(L::kThreads), L::kLds, s, a, x, out, bf16, rows, N, K, alpha, epi);
  });
}

// Waves along K until the card has 8 waves per CU or the steps are used up.
template <int M>
hipError_t stream_rows(const Int4Args& a, const uint16_t* x, void* out, int bf16, int64_t rows, int64_t N, int64_t K,
                       float alpha, int num_cus, const Epilogue& epi, hipStream_t s) {
  const int64_t tiles = (N + 15) / 16, want = int64_t(num_cus) * 8;
  if (tiles >= 2 * want) return stream_cfg<M, 2, 4, 1>(a, x, out, bf16, rows, N, K, alpha, epi, s);
  if (tiles >= want || K < 2 * kStep) return stream_cfg<M, 1, 4, 1>(a, x, out, bf16, rows, N, K, alpha, epi, s);
  if (tiles * 4 >= want || K < 8 * kStep) return stream_cfg<M, 1, 1, 4>(a, x, out, bf16, rows, N, K, alpha, epi, s);
  return stream_cfg<M, 1, 1, 8>(a, x, out, bf16, rows, N, K, alpha, epi, s);
}

template <int MT, int NT, int WN, int WK>
hipError_t gemm_cfg(const Int4Args& a, const uint16_t* x, void* out, int bf16, int64_t M, int64_t N, int64_t K,
                    float alpha, const Epilogue& epi, hipStream_t s) {
  using L = Int4Tile<MT, NT, WN, WK>;
  const int64_t total = ((M + L::kBM - 1) / L::kBM) * ((N + L::kBN - 1) / L::kBN);
  const int64_t blocks = (total + 7) / 8 * 8;
  if (blocks * L::kThreads >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  return by_group(a, [&](auto gs) -> hipError_t {
    auto kernel = int4_gemm_kernel<MT, NT, WN, WK, decltype(gs)::value>;
    static std::atomic<uint64_t> lds_set{0};
    if (hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), L::kLds, lds_set)) return e;
    return launch(kernel, dim3(unsigned(blocks)), dim3(L::kThreads), L::kLds, s, a, x, out, bf16, M, N, K, alpha, epi);
  });
}

constexpr int kMaxLds = 160 * 1024;

// Blocks for a walk of tiles BM x BN: as many as fit by LDS and registers (`waves` per block of
// cu_waves per CU), if there are so many tiles (at
// most ceil(T / BM) + min(G, T) row tiles exist), a multiple of 8.
int64_t walk_blocks(int64_t BM, int64_t BN, int waves, int cu_waves, int lds, int64_t G, int64_t T, int64_t N, int num_cus) {
  const int64_t upper = ((T + BM - 1) / BM + std::min(G, T)) * ((N + BN - 1) / BN);
  const int64_t per_cu = std::max<int64_t>(1, std::min<int64_t>(kMaxLds / lds, cu_waves / waves));
  return (std::min(upper, per_cu * num_cus) + 7) / 8 * 8;
}

struct GroupedCall {
  const Int4Args& a;
  const uint16_t* x;
  const uint32_t* offsets;
  const int32_t* ids;
  void* out;
  int bf16;
  int64_t G, E, T, N, K;
  int num_cus;
  hipStream_t s;

  template <typename Kernel> hipError_t go(Kernel kernel, std::atomic<uint64_t>& lds_set, int lds, int64_t BM, int64_t BN,
                                           int waves, int cu_waves) const {
    if (lds > kMaxLds) return hipErrorInvalidValue;
    if (hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(kernel), kMaxLds, lds_set)) return e;
    const int64_t blocks = walk_blocks(BM, BN, waves, cu_waves, lds, G, T, N, num_cus);
    return launch(kernel, dim3(unsigned(blocks)), dim3(64 * waves), lds, s, a, x, offsets, ids, out, bf16, G, T, N, K, E);
  }
};

template <int MT, int NT, int WN>
hipError_t grouped_cfg(const GroupedCall& c) {
  using L = Int4Tile<MT, NT, WN, 1>;
  return by_group(c.a, [&](auto gs) -> hipError_t {
    static std::atomic<uint64_t> lds_set{0};
    return c.go(int4_grouped_kernel<MT, NT, WN, decltype(gs)::value>, lds_set, int(L::kLds + 4 * (c.G + 1)), L::kBM, L::kBN,
                WN, 16);
  });
}

template <int NT, int WN>
hipError_t grouped_stream(const GroupedCall& c) {
  constexpr int kLds = StreamLayout<4, NT, WN, 1>::kLds;
  return by_shift(c.a, [&](auto sh) -> hipError_t {
    static std::atomic<uint64_t> lds_set{0};
    return c.go(int4_grouped_stream_kernel<NT, WN, decltype(sh)::value>, lds_set, int(kLds + 4 * (c.G + 1)), 4, 16 * NT * WN,
                WN, 4 * kStreamWaves);
  });
}

}  // namespace

hipError_t launch_int4_gemm(const uint8_t* w, const uint16_t* scale, const uint8_t* zero, const uint16_t* x, void* out,
                            int out_bf16, int64_t M, int64_t N, int64_t K, int64_t group, float alpha, int num_cus,
                            hipStream_t s, const Epilogue& epi) {
  const Int4Args a = make_args(w, scale, zero, K, group);
  if (M == 1) return stream_rows<1>(a, x, out, out_bf16, M, N, K, alpha, num_cus, epi, s);
  if (M == 2) return stream_rows<2>(a, x, out, out_bf16, M, N, K, alpha, num_cus, epi, s);
  if (M <= 4) return stream_rows<4>(a, x, out, out_bf16, M, N, K, alpha, num_cus, epi, s);
  // Up to 16 rows: tiles whose 4 waves split K, narrower where wide ones would leave CUs without any
  // (16 rows, K = 4096, calls behind each other, in us: N = 4096 16x16 8.5, 16x32 10.5; N = 8192 11.2, 11.0; N = 14336
  // 20.1, 17.2).
  if (M <= 16) {
    if (N <= int64_t(num_cus) * 32) return gemm_cfg<1, 1, 1, 4>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
    return gemm_cfg<1, 2, 1, 4>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
  }
  // Above, the tile with the least time for the CU that gets most of them.  A tile's time
  // hardly depends on how many other CUs have one: for K = 4096, groups of 64, calls behind each other, in us,
  //   64x128 36 (M = 500, N = 4096: 256 tiles 36; M = 200, N = 14336: 448 of them 70)
  //   32x128 28 (M = 250, N = 4096: 28; M = 500: 51), 64x256 62, 128x128 60, 128x256 97
  //   (M = 500, N = 14336: 98; with 128x128 tiles 120, 64x256 123, 64x128 138;
  //   M = 2048, N = 14336: 381, 420, 430, 503).
  // Those of 32x32 and 32x16 split K over their waves and share a CU: 11 (9) for the first, and
  // as much for each more on average (M = 64, N = 4096: 15; M = 64, N = 14336: 38).
  // Groups of 128 take 0.82 to 0.96 of these times, groups of 32 1.18 to 1.36, and K = 1024 and 14336 a third and 3.3 times:
  // the same tile is the fastest for each of them at M = 500, N = 4096 and 14336.
  struct Tile {
    int bm, bn, us;
    bool shared;
  };
  constexpr Tile kTiles[] = {{32, 16, 9, true},    {32, 32, 11, true},    {32, 128, 28, false}, {64, 128, 36, false},
                             {64, 256, 62, false}, {128, 128, 60, false}, {128, 256, 97, false}};
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < int(sizeof(kTiles) / sizeof(Tile)); ++i) {
    const Tile& t = kTiles[i];
    const int64_t tiles = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
    const double per_cu = t.shared ? std::max(1.0, double(tiles) / num_cus) : double((tiles + num_cus - 1) / num_cus);
    if (i == 0 || per_cu * t.us < least) {
      best = i;
      least = per_cu * t.us;
    }
  }
  switch (best) {
    case 0: return gemm_cfg<2, 1, 1, 4>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
    case 1: return gemm_cfg<2, 2, 1, 4>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
    case 2: return gemm_cfg<2, 1, 8, 1>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
    case 3: return gemm_cfg<4, 1, 8, 1>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
    case 4: return gemm_cfg<4, 2, 8, 1>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
    case 5: return gemm_cfg<8, 1, 8, 1>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
    default: return gemm_cfg<8, 2, 8, 1>(a, x, out, out_bf16, M, N, K, alpha, epi, s);
  }
}

hipError_t launch_int4_grouped(const uint8_t* w, const uint16_t* scale, const uint8_t* zero, const uint16_t* x,
                               const uint32_t* a_offsets, const int32_t* expert_ids, void* out, int out_bf16,
                               int64_t G, int64_t E, int64_t T, int64_t N, int64_t K, int64_t group, int num_cus,
                               hipStream_t s) {
  const Int4Args a = make_args(w, scale, zero, K, group);
  // By the rows a group has on average (64 experts, N = 1536, K = 2048, groups of 128, counts spread by Zipf 0.5, unless
  // said; calls behind each other, about half of the weights in the 256 MB cache), in us: to 6 the streaming form (64
  // rows: 23, 32x256 51; 384 rows: 41 and 51; 768 rows: 75 and 51), to 32 tiles of 32x256 (1024 rows: 51, 32x128 56,
  // 64x256 62; 2048 rows: 74, 70, 64), or of 32x128 where 32x256 would leave CUs without any (8 experts, N = K = 4096,
  // groups of 64, 96 rows: 31 and 52), above of 64x256 (4096 rows: 90, 32x256 97, 32x128 107; those 8 experts, 512 rows: 66,
  // 32x128 86, 32x256 103; 4096 rows: 318, 32x256 446).
  const bool few = ((T + 31) / 32 + std::min(G, T)) * ((N + 255) / 256) <= num_cus;
  // A block keeps the groups' prefix sums in LDS beside its tile: more groups take more launches.
  constexpr int64_t kMost = 16384;
  for (int64_t z = 0; z < G; z += kMost) {
    const int64_t groups = std::min(kMost, G - z);
    const GroupedCall c{a, x, a_offsets + z, expert_ids + z, out, out_bf16, groups, E, T, N, K, num_cus, s};
    const hipError_t e = T <= 6 * G    ? grouped_stream<1, 4>(c)
                         : T <= 32 * G ? few ? grouped_cfg<2, 1, 8>(c) : grouped_cfg<2, 2, 8>(c)
                                       : grouped_cfg<4, 2, 8>(c);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qlinear
