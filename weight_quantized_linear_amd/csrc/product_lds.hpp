// A tile of C[m, n] = sum_k A[m, k] B[n, k] on the matrix cores, with either operand stored
// along k ("rows": [M, K], bfloat16 or FP8) or across it ("turned": [K, M], bfloat16).
//
// * A block of NW waves owns BM x BN, a wave (BM / WY) x (BN / WX) of 32 x 32 MFMA blocks. K goes in strips of 64 (or 128)
//   through a ring of S LDS stages, filled by loads that write LDS directly; a strip is
//   steps of 16, and while the matrix cores work on one, the operands of the next are read.
// * Rows operands lie in LDS as 128-byte rows (FP8: 64; twice that in strips of 128) with their 16-byte pieces permuted;
// a lane
//   reads the 8 values of its row with one load (FP8: 16 values for two steps, widened exactly).
// * Turned operands lie as 64 rows of k.  The transposing LDS read hands lane l of 16 the values k .. k + 3
//   of column l from four rows: two reads give the 8 values that the MFMA wants.  Their 64-byte pieces
//   are permuted by k so that the four rows of a read lie in different banks.
// * Inside a strip, lane half h takes k = 32 t + 16 h + 8 e .. + 7 in step 2 t + e, for both operands.
// * The strips' addresses move in the buffer resource, 64 bits wide, so an operand may be larger than 4 GiB; what
//   lies past the operand's end is zero by the resource's bound, and in the last strip of a rows
//   operand what lies past K is sent past that bound.
#pragma once

#include "lds_gemm.hpp"

namespace qlinear {

constexpr int kStripK = 64;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s_t;

// Where an operand lies: rows operand: `ld` bytes a row of k; turned: `ld` bytes a row of the
// other axis, K rows.
struct Operand {
  const char* p;
  int64_t ld;
  int64_t extent;  // rows operand: its rows; turned: K
};

constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // an offset past every resource's bound

// A resource of `bytes` bytes at p, bounded so that kNowhere lies outside; none: nothing lies inside.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t strip_rsrc(const char* p, int64_t bytes, bool none) {
  return make_rsrc(p, none ? 0 : bytes < int64_t(kNowhere) ? bytes : int64_t(kNowhere));
}

// 16 bytes per lane straight into LDS, not kept in the caches.
__device__ __forceinline__ void bdma16_nt(__amdgpu_buffer_rsrc_t rsrc, char* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)lds, 16, voff, 0, 0, 2);
}

// Row r of the tile is row `first + r` of the operand.
struct PlainRows {
  int64_t first, rows;
  __device__ __forceinline__ int64_t at(int r) const { return r; }
  __device__ __forceinline__ bool in(int r) const { return first + r < rows; }
};
// Of every 64 rows of the tile 32 are gate rows and 32 the up rows of the same columns.
struct GatedRows {
  int64_t first, rows;  // of F
  __device__ __forceinline__ int64_t at(int r) const { return r / 64 * 32 + r % 32 + (r / 32 % 2 ? rows : 0); }
  __device__ __forceinline__ bool in(int r) const { return first + r / 64 * 32 + r % 32 < rows; }
};

// ROWS rows of SK values of k, EB bytes each (2: bfloat16, 1: FP8).  NT: past the caches.
template <int ROWS, int NW, int EB, class Map, int SK = kStripK, bool NT = false>
struct RowsOperand {
  using Layout = RowsOperand;
  static constexpr int kStrip = SK, kRowBytes = SK * EB, kCpr = kRowBytes / 16, kBytes = ROWS * kRowBytes;
  static constexpr int kInst = ROWS * kCpr / (64 * NW);
  static_assert(ROWS * kCpr % (64 * NW) == 0, "whole instructions");
  const char* base;
  int64_t bytes;  // from base to the operand's end
  uint32_t off[kInst], tail[kInst];

  __device__ __forceinline__ void init(const Operand& o, const Map& map, int64_t K) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    base = o.p + map.first * o.ld;
    bytes = (o.extent - map.first) * o.ld;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const int c = (q * NW + wid) * 64 + lane, r = c / kCpr, g = (c % kCpr) ^ swz<kCpr>(r);
      off[q] = map.in(r) ? uint32_t(map.at(r) * o.ld + 16 * g) : kNowhere;
      const int left = int(K % SK) * EB;  // bytes of a row in the last strip, 0: all
      tail[q] = left && 16 * g >= left ? kNowhere : off[q];
    }
  }
  __device__ __forceinline__ void fetch(char* tile, int64_t strip, bool last, bool none) const {
    const int wid = threadIdx.x >> 6;
    const int64_t at = strip * kRowBytes;
    const __amdgpu_buffer_rsrc_t r = strip_rsrc(base + at, bytes - at, none);
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      char* const to = tile + (q * NW + wid) * 1024;
      if constexpr (NT) bdma16_nt(r, to, last ? tail[q] : off[q]);
      else bdma16(r, to, last ? tail[q] : off[q], 0);
    }
  }
};

// Where row k of a turned strip of CPR 16-byte pieces a row has its pieces: exchanged in groups of four (64 bytes), so
// that a group's four rows k .. k + 3 lie in different quarters of the 64 banks.  Rows of 16 or 32 pieces all begin in
// the same quarter; rows of 24 begin in quarters 0, 2, 0, 2.
template <int CPR>
__device__ __forceinline__ int turned_swz(int k) {
  static_assert(CPR % 8 == 0 && CPR >= 16, "groups of four, in pairs");
  return CPR % 16 == 0 ? (k & 3) << 2 : (k >> 1 & 1) << 2;
}

// 64 rows of k, COLS values (bfloat16) each.
template <int COLS, int NW>
struct TurnedOperand {
  using Layout = TurnedOperand;
  static constexpr int kStrip = kStripK, kRowBytes = COLS * 2, kCpr = kRowBytes / 16, kBytes = kStripK * kRowBytes;
  static constexpr int kInst = kStripK * kCpr / (64 * NW);
  static_assert(kStripK * kCpr % (64 * NW) == 0, "whole instructions");
  const char* base;
  int64_t bytes, step;
  uint32_t off[kInst];

  __device__ __forceinline__ void init(const Operand& o, const PlainRows& map, int64_t) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    base = o.p + map.first * 2;
    bytes = o.extent * o.ld - map.first * 2;
    step = kStripK * o.ld;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const int c = (q * NW + wid) * 64 + lane, k = c / kCpr, g = (c % kCpr) ^ turned_swz<kCpr>(k);
      off[q] = uint32_t(k * o.ld + 16 * g);
    }
  }
  __device__ __forceinline__ void fetch(char* tile, int64_t strip, bool, bool none) const {
    const int wid = threadIdx.x >> 6;
    const int64_t at = strip * step;
    const __amdgpu_buffer_rsrc_t r = strip_rsrc(base + at, bytes - at, none);
#pragma unroll
    for (int q = 0; q < kInst; ++q) bdma16(r, tile + (q * NW + wid) * 1024, off[q], 0);
  }
};

// ---------------------------------------------------------------- operands at any address
//
// The same tiles through registers, for operands whose rows are not whole 16-byte pieces at aligned
// addresses: 16-byte loads at any address, held inside the operand.  A row's last values, where it does
// not end with a piece of G of them, are taken as the G values before its end, of which those that the piece before
// had are zeroed, in both operands: G = 8, or 16 beside FP8 weights, so that k means the same in both.  K >= G, and
// turned operands have 8 columns at least.

typedef u32x4 u32x4_loose1 __attribute__((aligned(1)));

// Value index of slot k of the contraction, and whether it is a repetition.
template <int G>
__device__ __forceinline__ int64_t slot_value(int64_t k, int64_t K) {
  const int64_t first = k & ~int64_t(G - 1);
  return first > K - G ? K - G + (k - first) : k;
}

// The pieces' addresses move on from strip to strip; only the last strip, where the row or the operand ends, works them
// out anew.
template <int ROWS, int NW, int EB, class Map, int G>
struct StagedRows {
  using Layout = RowsOperand<ROWS, NW, EB, Map>;
  static constexpr int kBytes = Layout::kBytes, kInst = Layout::kInst, kCpr = Layout::kCpr, kValues = 16 / EB;
  const char* at[kInst];  // of the next strip's pieces
  int64_t K;
  u32x4 held[kInst];
  static __device__ __forceinline__ int chunk(int q) { return (q * NW + (threadIdx.x >> 6)) * 64 + (threadIdx.x & 63); }
  static __device__ __forceinline__ int place(int q) { return (chunk(q) % kCpr) ^ swz<kCpr>(chunk(q) / kCpr); }
  __device__ __forceinline__ void init(const Operand& o, const Map& map, int64_t k, int64_t s0) {
    K = k;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const int r = chunk(q) / kCpr;  // rows past the end: any, not stored
      at[q] = o.p + (map.first + (map.in(r) ? map.at(r) : 0)) * o.ld + s0 * kStripK * EB + 16 * place(q);
    }
  }
  __device__ __forceinline__ void load(int64_t strip) {
    const bool ends = (strip + 1) * kStripK > K;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const char* p = at[q];
      if (ends) {
        const int64_t slot = strip * kStripK + place(q) * kValues;
        p += (slot_value<G>(slot, K) - slot) * EB;
      }
      held[q] = *reinterpret_cast<const u32x4_loose1*>(p);
      at[q] += kStripK * EB;
    }
  }
  __device__ __forceinline__ void store(char* tile, int64_t strip) {
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      if ((strip + 1) * kStripK > K) {
        const int64_t slot = strip * kStripK + place(q) * kValues, first = slot & ~int64_t(G - 1);
        const int64_t value = slot_value<G>(slot, K);
#pragma unroll
        for (int e = 0; e < kValues; ++e)
          if (value + e < first) held[q][e * EB / 4] &= ~((EB == 2 ? 0xFFFFu : 0xFFu) << (e * EB % 4 * 8));
      }
      *reinterpret_cast<u32x4*>(tile + chunk(q) * 16) = held[q];
    }
  }
};

template <int COLS, int NW, int G>
struct StagedTurned {
  using Layout = TurnedOperand<COLS, NW>;
  static constexpr int kBytes = Layout::kBytes, kInst = Layout::kInst, kCpr = Layout::kCpr;
  const char* at[kInst];
  int64_t ld, K;
  int over[kInst];  // columns of a piece past the row's end (7: all); the row's last eight are loaded then and moved in store()
  u32x4 held[kInst];
  static __device__ __forceinline__ int chunk(int q) { return (q * NW + (threadIdx.x >> 6)) * 64 + (threadIdx.x & 63); }
  __device__ __forceinline__ void init(const Operand& o, const PlainRows& map, int64_t k, int64_t s0) {
    ld = o.ld;
    K = k;
    const int64_t left = map.rows - map.first;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const int kk = chunk(q) / kCpr, col = 8 * ((chunk(q) % kCpr) ^ turned_swz<kCpr>(kk));
      const int64_t from = col < left - 8 ? col : left - 8;
      over[q] = col - from < 7 ? int(col - from) : 7;
      at[q] = o.p + (s0 * kStripK + kk) * ld + 2 * (map.first + from);
    }
  }
  __device__ __forceinline__ void load(int64_t strip) {
    const bool ends = (strip + 1) * kStripK > K;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const char* p = at[q];
      if (ends) {
        const int64_t slot = strip * kStripK + chunk(q) / kCpr;
        p += (slot_value<G>(slot, K) - slot) * ld;
      }
      held[q] = *reinterpret_cast<const u32x4_loose1*>(p);
      at[q] += kStripK * ld;
    }
  }
  __device__ __forceinline__ void store(char* tile, int64_t strip) {
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      u32x4 v = held[q];
      if (over[q]) {
        const int by = 16 * over[q];
        uint64_t lo = v.x | uint64_t(v.y) << 32;
        const uint64_t hi = v.z | uint64_t(v.w) << 32;
        lo = by >= 64 ? hi >> (by - 64) : lo >> by | hi << (64 - by);
        const uint64_t up = by >= 64 ? 0 : hi >> by;
        v = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(up), uint32_t(up >> 32)};
      }
      if ((strip + 1) * kStripK > K) {
        const int64_t slot = strip * kStripK + chunk(q) / kCpr;
        if (slot_value<G>(slot, K) < (slot & ~int64_t(G - 1))) v = u32x4{0, 0, 0, 0};
      }
      *reinterpret_cast<u32x4*>(tile + chunk(q) * 16) = v;
    }
  }
};

// The wave's fragments of NF blocks of 32 rows from `row0` on.
template <class Op, int NF> struct Fragments;

template <int ROWS, int NW, class Map, int SK, bool NT, int NF>
struct Fragments<RowsOperand<ROWS, NW, 2, Map, SK, NT>, NF> {
  static constexpr int kReads = NF;  // LDS reads of a step
  uint32_t at[SK / 16];
  __device__ __forceinline__ void init(int row0) {
    const int r = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int u = 0; u < SK / 16; ++u)
      at[u] = uint32_t((row0 + r) * SK * 2 + 16 * ((4 * (u / 2) + 2 * h + u % 2) ^ swz<SK / 8>(r)));
  }
  template <int U>
  __device__ __forceinline__ void read(const char* tile, v8bf (&f)[NF]) {
#pragma unroll
    for (int j = 0; j < NF; ++j) f[j] = __builtin_bit_cast(v8bf, lds16(tile + at[U] + j * 32 * SK * 2));
  }
};

template <int ROWS, int NW, class Map, int SK, bool NT, int NF>
struct Fragments<RowsOperand<ROWS, NW, 1, Map, SK, NT>, NF> {
  static constexpr int kReads = NF;
  uint32_t at[SK / 32];
  u32x4 raw[NF];
  __device__ __forceinline__ void init(int row0) {
    const int r = threadIdx.x & 31, h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int t = 0; t < SK / 32; ++t) at[t] = uint32_t((row0 + r) * SK + 16 * ((2 * t + h) ^ swz<SK / 16>(r)));
  }
  template <int U>
  __device__ __forceinline__ void read(const char* tile, v8bf (&f)[NF]) {
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      if constexpr (U % 2 == 0) raw[j] = lds16(tile + at[U / 2] + j * 32 * SK);
      f[j] = U % 2 == 0 ? e4m3x8_to_bf16x8(raw[j].x, raw[j].y) : e4m3x8_to_bf16x8(raw[j].z, raw[j].w);
    }
  }
};

template <int COLS, int NW, int NF>
struct Fragments<TurnedOperand<COLS, NW>, NF> {
  static constexpr int kReads = 2 * NF;
  uint32_t at[NF];
  // Lane 16 g + 4 j + c of a read supplies k row j of its half's eight (+ 4 in the second read), columns 16 (g % 2) + 4 c.
  __device__ __forceinline__ void init(int row0) {
    const int lane = threadIdx.x & 63, j = lane / 4 % 4, h = lane / 32;
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      const int byte = (row0 + 32 * n + 16 * (lane / 16 % 2) + 4 * (lane % 4)) * 2;
      at[n] = uint32_t((16 * h + j) * COLS * 2 + (byte ^ (turned_swz<COLS / 8>(j) << 4)));
    }
  }
  template <int U>
  __device__ __forceinline__ void read(const char* tile, v8bf (&f)[NF]) {
    constexpr int k = 32 * (U / 2) + 8 * (U % 2);
#pragma unroll
    for (int n = 0; n < NF; ++n) {
      char* p = const_cast<char*>(tile) + at[n] + k * COLS * 2;
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)p);
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(p + 4 * COLS * 2));
      f[n] = __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

template <class AOp, class BOp, int BM, int BN, int S, int WY, int NW>
struct ProductLayout {
  static constexpr int WX = NW / WY, FM = BM / WY / 32, FN = BN / WX / 32;
  static constexpr int kStage = AOp::kBytes + BOp::kBytes, kLds = S * kStage;
  static constexpr int kLoads = AOp::kInst + BOp::kInst;
  static constexpr int kStrip = AOp::kStrip;
  static_assert(kLds <= 160 * 1024 && (S - 1) * kLoads < 64 && S >= 2 && BOp::kStrip == kStrip, "ring");
};

// The sums of the tile whose operands `a` and `b` were set to, over the strips s0 .. s0 + nk - 1 of K (nk >= 1):
// acc[i][j][v] belongs to row
// 32 i + 8 (v / 4) + 4 h + v % 4 and column 32 j + lane % 32 of the wave's part.
template <class AOp, class BOp, int BM, int BN, int S, int WY, int NW>
__device__ __forceinline__ void product_tile(
    char* lds, const AOp& a, const BOp& b, int64_t K, int64_t s0, int64_t nk,
    v16f (&acc)[ProductLayout<AOp, BOp, BM, BN, S, WY, NW>::FM][ProductLayout<AOp, BOp, BM, BN, S, WY, NW>::FN]) {
  using L = ProductLayout<AOp, BOp, BM, BN, S, WY, NW>;
  constexpr int FM = L::FM, FN = L::FN, NM = FM * FN;
  const int wid = threadIdx.x >> 6;
  Fragments<AOp, FM> fa;
  Fragments<BOp, FN> fb;
  fa.init(wid / L::WX * (BM / WY));
  fb.init(wid % L::WX * (BN / L::WX));
  auto fetch = [&](int64_t s) {
    char* st = lds + int(s % S) * L::kStage;
    const bool last = (s0 + s + 1) * L::kStrip >= K, none = s >= nk;
    a.fetch(st, none ? 0 : s0 + s, last, none);
    b.fetch(st + AOp::kBytes, none ? 0 : s0 + s, last, none);
  };
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v16f{};
  v8bf aX[FM], aY[FM], bX[FN], bY[FN];
  auto mma = [&](const v8bf (&x)[FM], const v8bf (&y)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[i], y[j], acc[i][j], 0, 0, 0);
  };
  constexpr int kReads = Fragments<AOp, FM>::kReads + Fragments<BOp, FN>::kReads;
#pragma unroll
  for (int s = 0; s < S; ++s) fetch(s);
  wait_vm<(S - 1) * L::kLoads>();
  block_barrier();
  fa.template read<0>(lds, aX);
  fb.template read<0>(lds + AOp::kBytes, bX);
  auto inner = [&](const char* st) {
    const char* sb = st + AOp::kBytes;
    static_for<L::kStrip / 16 - 1>([&](auto uc) {
      constexpr int U = decltype(uc)::value;
      fa.template read<U + 1>(st, U % 2 ? aX : aY);
      fb.template read<U + 1>(sb, U % 2 ? bX : bY);
      mma(U % 2 ? aY : aX, U % 2 ? bY : bX);
      interleave<NM, 0, kReads, 0>();
    });
  };
  for (int64_t kt = 0; kt < nk - 1; ++kt) {
    inner(lds + int(kt % S) * L::kStage);
    // Into the next strip: it has landed for every wave after the barrier, and this one's slot is free
    // once every wave's reads of it returned.
    wait_lds();
    wait_vm<(S - 2) * L::kLoads>();
    block_barrier();
    const char* sn = lds + int((kt + 1) % S) * L::kStage;
    fa.template read<0>(sn, aX);
    fb.template read<0>(sn + AOp::kBytes, bX);
    fetch(kt + S);  // behind the reads: 3 to 5 % less time than in front of them
    mma(aY, bY);
    interleave<NM, L::kLoads, kReads, 0>();
  }
  inner(lds + int((nk - 1) % S) * L::kStage);
  mma(aY, bY);
  wait_vm<0>();  // no LDS write may land after the block ends
}

// The same with staged operands and one stage: a strip's values wait in registers while the strip before
// is multiplied.  With few registers and little LDS a block, others on its CU cover its barriers.
template <class AOp, class BOp, int BM, int BN, int WY, int NW>
__device__ __forceinline__ void staged_tile(char* lds, AOp& a, BOp& b, int64_t s0, int64_t nk,
                                            v16f (&acc)[BM / WY / 32][BN / (NW / WY) / 32]) {
  constexpr int WX = NW / WY, FM = BM / WY / 32, FN = BN / WX / 32;
  const int wid = threadIdx.x >> 6;
  Fragments<typename AOp::Layout, FM> fa;
  Fragments<typename BOp::Layout, FN> fb;
  fa.init(wid / WX * (BM / WY));
  fb.init(wid % WX * (BN / WX));
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = v16f{};
  a.load(s0);
  b.load(s0);
  for (int64_t s = 0; s < nk; ++s) {
    if (s > 0) {
      wait_lds();
      block_barrier();  // every wave has read the strip before
    }
    a.store(lds, s0 + s);
    b.store(lds + AOp::kBytes, s0 + s);
    if (s + 1 < nk) {
      a.load(s0 + s + 1);
      b.load(s0 + s + 1);
    }
    wait_lds();
    block_barrier();
    v8bf af[FM], bf[FN];
    static_for<4>([&](auto uc) {
      constexpr int U = decltype(uc)::value;
      fa.template read<U>(lds, af);
      fb.template read<U>(lds + AOp::kBytes, bf);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[i], bf[j], acc[i][j], 0, 0, 0);
    });
  }
}

}  // namespace qlinear
