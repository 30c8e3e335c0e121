// Building blocks of the tiled GEMMs whose operands go to LDS by direct loads: buffer
// resources, the strips' fetches and their slot permutation, scheduling hints, the order of
// the tiles over the XCDs and the staging of output rows.
#pragma once

#include <type_traits>
#include <utility>

#include "device.hpp"
#include "launch.hpp"

namespace qlinear {

__device__ __forceinline__ void dma4(const char* g, char* lds) {
  __builtin_amdgcn_global_load_lds((gbl_void_t*)g, (lds_void_t*)lds, 4, 0, 0);
}

// Raw buffer over `bytes` bytes at p (stride 0; the last dword is the
// gfx9-family raw-buffer format word).  Buffer loads address it with a
// 32-bit per-lane offset plus a uniform offset, so no 64-bit per-lane
// address registers are needed; a lane whose offset lies past the record
// count reads zeros without touching memory.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, int64_t bytes) {
  const uint32_t n = bytes >= int64_t(0xFFFFFFFF) ? 0xFFFFFFFFu : uint32_t(bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(n), 0x00020000);
}

// Buffer load of 16 (4) bytes per lane straight into LDS (lane i at lds + 16 i (4 i)).
__device__ __forceinline__ void bdma16(__amdgpu_buffer_rsrc_t rsrc, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void bdma4(__amdgpu_buffer_rsrc_t rsrc, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)lds, 4, voff, soff, 0, 0);
}

__device__ __forceinline__ u32x4 lds16(const char* p) { return *reinterpret_cast<const u32x4*>(p); }

// Slot permutation of a row with CPR 16-byte chunks (CPR in {2, 4, 8, 16}): rows
// r and r' of one 16-row group collide in a bank group only if they also
// agree in r / (16 / CPR), which the XOR then separates.
template <int CPR>
__device__ __forceinline__ int swz(int r) {
  return (r / (16 / CPR)) & (CPR - 1);
}

// ---------------------------------------------------------------- scheduling hints

// Items of `total` given to slot m when spread evenly over slots [lo, hi).
constexpr int share(int total, int lo, int hi, int m) {
  return (m < lo || m >= hi) ? 0 : (m - lo + 1) * total / (hi - lo) - (m - lo) * total / (hi - lo);
}

template <int NM, int NV, int ND, int NA, int M>
__device__ __forceinline__ void sched_slot() {
  // Consecutive ranges of MFMA slots for the LDS reads, the VMEM loads and
  // the VALU work, in that order; absent classes take no slots.
  constexpr int parts = (ND > 0) + (NV > 0) + (NA > 0);
  constexpr int len = parts ? NM / parts : NM;
  constexpr int d_end = ND ? (NV || NA ? len : NM) : 0;
  constexpr int v_end = NV ? (NA ? d_end + len : NM) : d_end;
  constexpr int nd = share(ND, 0, d_end, M);
  constexpr int nv = share(NV, d_end, v_end, M);
  constexpr int na = share(NA, v_end, NM, M);
  __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
  if constexpr (nd > 0) __builtin_amdgcn_sched_group_barrier(0x100, nd, 0);  // LDS reads
  if constexpr (nv > 0) __builtin_amdgcn_sched_group_barrier(0x020, nv, 0);  // VMEM loads
  if constexpr (na > 0) __builtin_amdgcn_sched_group_barrier(0x002, na, 0);  // VALU
}

template <int NM, int NV, int ND, int NA, int... Ms>
__device__ __forceinline__ void sched_region(std::integer_sequence<int, Ms...>) {
  (sched_slot<NM, NV, ND, NA, Ms>(), ...);
}

// Order the current scheduling region as NM MFMAs with ND LDS reads spread
// over the first of them, then NV VMEM loads, then NA VALU instructions (the
// weight decode, which needs the LDS reads).
template <int NM, int NV, int ND, int NA>
__device__ __forceinline__ void interleave() {
  sched_region<NM, NV, ND, NA>(std::make_integer_sequence<int, NM>{});
}

// f(std::integral_constant<int, 0>{}) .. f(std::integral_constant<int, N - 1>{}):
// a loop whose index is a compile-time constant in the body.
template <class F, int... Is>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// ---------------------------------------------------------------- strip DMA

// One strip of ROWS rows x SB bytes of a row-major operand (row stride `ld`
// bytes), rows r0 .. r0 + ROWS - 1 clipped to `rows`.  The strip's 16-byte
// chunks are split evenly over the waves; DMA instruction q of wave w covers
// chunks (q NW + w) kLanes .. +kLanes - 1 (row c / CPR, slot c % CPR).
template <int ROWS, int SB, int NW>
struct StripDma {
  static constexpr int kCpr = SB / 16;
  static constexpr int kChunks = ROWS * kCpr;
  static_assert(kChunks % NW == 0, "every wave issues the same number of DMA instructions");
  static constexpr int kPerWave = kChunks / NW;
  static constexpr int kLanes = kPerWave >= 64 ? 64 : kPerWave;  // active lanes per instruction
  static_assert(kPerWave % kLanes == 0, "whole instructions");
  static constexpr int kInst = kPerWave / kLanes;  // per wave per strip
  uint32_t off[kInst];
  __device__ __forceinline__ void init(int64_t r0, int64_t rows, int64_t ld) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const int c = (q * NW + wid) * kLanes + (lane < kLanes ? lane : 0);
      const int r = c / kCpr;
      const int g = (c % kCpr) ^ swz<kCpr>(r);
      int64_t row = r0 + r;
      if (row >= rows) row = rows - 1;
      off[q] = uint32_t(row * ld + 16 * g);
    }
  }
  // The same without clamping, for buffer fetches: rows past `rows` lie
  // past the buffer's record count and are zero-filled.
  __device__ __forceinline__ void init_open(int64_t r0, int64_t ld) {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const int c = (q * NW + wid) * kLanes + (lane < kLanes ? lane : 0);
      const int r = c / kCpr;
      const int g = (c % kCpr) ^ swz<kCpr>(r);
      off[q] = uint32_t((r0 + r) * ld + 16 * g);
    }
  }
  // base = operand start + the strip's byte offset within a row (uniform)
  __device__ __forceinline__ void fetch(char* tile, const char* base) const {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
    for (int q = 0; q < kInst; ++q)
      if (kLanes == 64 || lane < kLanes) dma16(base + off[q], tile + (q * NW + wid) * kLanes * 16);
  }
  // The same through a buffer resource; soff = the strip's byte offset.
  __device__ __forceinline__ void fetch(char* tile, __amdgpu_buffer_rsrc_t rsrc, uint32_t soff) const {
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
#pragma unroll
    for (int q = 0; q < kInst; ++q)
      if (kLanes == 64 || lane < kLanes) bdma16(rsrc, tile + (q * NW + wid) * kLanes * 16, off[q], soff);
  }
};

// Block b -> (row tile, column tile).  Blocks are dealt to the 8 XCDs round
// robin, so XCD x runs blocks x, x + 8, ...; give it a contiguous range of
// tiles, and inside the range walk 8 row tiles per column tile.
__device__ __forceinline__ void tile_of_block(int64_t b, int64_t tiles_m, int64_t tiles_n, int64_t& tm,
                                              int64_t& tn) {
#ifdef QLINEAR_FLAT_TILE_ORDER
  // Build option (QLINEAR_TILE_ORDER=flat in build.py) for measuring what the
  // order below buys: the plain row-major grid.
  tm = b / tiles_n;
  tn = b % tiles_n;
  return;
#endif
  constexpr int kXcd = 8, kGroupM = 8;
  const int64_t total = tiles_m * tiles_n;
  const int64_t q = total / kXcd, r = total % kXcd;
  const int64_t xcd = b % kXcd, local = b / kXcd;
  const int64_t t = xcd < r ? xcd * (q + 1) + local : r * (q + 1) + (xcd - r) * q + local;
  const int64_t group = kGroupM * tiles_n;
  const int64_t g = t / group;
  const int64_t first_m = g * kGroupM;
  const int64_t gm = tiles_m - first_m < kGroupM ? tiles_m - first_m : kGroupM;
  const int64_t in_group = t % group;
  tm = first_m + in_group % gm;
  tn = in_group / gm;
}

// ---------------------------------------------------------------- output staging

// OUT: 0 = float32, 1 = bfloat16 (round to nearest even; gfx950 converts in
// hardware), 2 = int32.
template <int OUT>
struct OutT {
  static constexpr int kBytes = OUT == 1 ? 2 : 4;
};

template <int OUT>
__device__ __forceinline__ void put_out(void* out, int64_t i, float v) {
  if constexpr (OUT == 1) reinterpret_cast<__bf16*>(out)[i] = static_cast<__bf16>(v);
  else reinterpret_cast<float*>(out)[i] = v;
}

// ROWS rows of a wave's output part (ROWS x 32 FN elements) staged in LDS
// so that they leave as 16-byte row segments.  Row stride: the two lane
// halves of one ds_write (rows 4 apart) hit disjoint banks.
template <int OUT, int FN, int ROWS>
struct Slab {
  static constexpr int kEs = OutT<OUT>::kBytes;
  static constexpr int kCols = 32 * FN;
  static constexpr int kStride = kEs * kCols + (kEs == 2 ? 16 : 32);
  static constexpr int kBytes = ROWS * kStride;
  static constexpr int kLanesPerRow = kCols * kEs / 16;
  static constexpr int kChunks = ROWS * kLanesPerRow;  // 16-byte pieces
  static constexpr int kInst = (kChunks + 63) / 64;
  static_assert(kLanesPerRow <= 64, "slab row layout");

  char* base;
  int lane;  // 0 .. 63
  __device__ __forceinline__ char* at(int row, int col) const { return base + row * kStride + col * kEs; }
  __device__ __forceinline__ void put_f(int row, int col, float x) const {
    if constexpr (OUT == 1) *reinterpret_cast<__bf16*>(at(row, col)) = static_cast<__bf16>(x);
    else *reinterpret_cast<float*>(at(row, col)) = x;
  }
  __device__ __forceinline__ void put_i(int row, int col, int32_t x) const {
    *reinterpret_cast<int32_t*>(at(row, col)) = x;
  }
  // Copy the slab to out rows row0 .. row0 + ROWS - 1, columns col0 ..
  // (row-major, leading dimension N elements, 16-byte aligned rows).  LDS
  // accesses of one wave complete in order, so the reads see the writes;
  // the asm barriers keep the compiler from reordering them.
  __device__ __forceinline__ void flush(void* out, int64_t N, int64_t row0, int64_t col0) const {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < kInst; ++q) {
      const int idx = q * 64 + lane;
      if (kChunks % 64 == 0 || idx < kChunks) {
        const int row = idx / kLanesPerRow, cb = (idx % kLanesPerRow) * 16;
        const u32x4 d = lds16(base + row * kStride + cb);
        *reinterpret_cast<u32x4*>(reinterpret_cast<char*>(out) + ((row0 + row) * N + col0) * kEs + cb) = d;
      }
    }
    asm volatile("" ::: "memory");
  }
};

// Raise the kernel's dynamic LDS limit once per kernel, then launch.
template <auto Kernel, class... Args>
hipError_t launch_big_lds(int lds_bytes, int64_t blocks, int threads, hipStream_t s, Args... args) {
  static std::atomic<uint64_t> lds_set{0};  // per kernel, one bit per device
  if (hipError_t e = raise_lds_limit(reinterpret_cast<const void*>(Kernel), lds_bytes, lds_set)) return e;
  return launch(Kernel, dim3(blocks), dim3(threads), lds_bytes, s, args...);
}

}  // namespace qlinear
