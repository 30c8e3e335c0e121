// The mixture-of-experts operators around the grouped products: the top-k
// softmax router and its gradient, the stable sort of token slots by expert,
// the gather of token rows into expert order, the weighted way back and its
// gradient, and the experts' gated activation with its gradient.
#include "device.hpp"
#include "launch.hpp"

namespace qlinear {

namespace {

// 16 bytes at any 2-byte (4-byte) aligned address: global accesses of gfx950
// need no more, so rows of odd lengths take the same wide accesses.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ u32x4 ld16_any(const void* p) { return *reinterpret_cast<const u32x4_any*>(p); }
__device__ __forceinline__ void st16_any(void* p, u32x4 v) { *reinterpret_cast<u32x4_any*>(p) = v; }
// NT: past the caches, for calls that move more than these hold (kNtBytes).
template <bool NT> __device__ __forceinline__ u32x4 ld16_at(const void* p) {
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  else return ld16_any(p);
}
template <bool NT> __device__ __forceinline__ void st16_at(void* p, u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  else st16_any(p, v);
}

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

// ---------------------------------------------------------------- wave helpers

// Kernels whose waves take independent items (a token, a slot, a piece of a
// row) walk them with a stride, so any number of items fits the grid.
__device__ __forceinline__ int64_t first_item() {
  return int64_t(blockIdx.x) * (blockDim.x / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
}
__device__ __forceinline__ int64_t item_stride() { return int64_t(gridDim.x) * (blockDim.x / kWave); }
constexpr int64_t kMaxBlocks = int64_t(1) << 20;

// A logit as an unsigned key of the same order; 0 marks what is never chosen
// (-inf and NaN).  -0 and +0 share a key.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  const uint32_t k = (u >> 31) ? ~u : (u | 0x80000000u);
  return f > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

// ---------------------------------------------------------------- router

// L lanes per token (16, 32 or 64: the fewest that hold its E logits with at
// most 16 each), so a wave takes up to 4 tokens; lane l of a token holds the R
// logits e = l R .. l R + R - 1.  The kernel is bound by its vector instructions (87 % of the SIMDs' cycles), and
// a pick costs the same ones however many tokens the wave holds: T = 16384, E = 256,
// top 8, bfloat16 takes 9.0 us, 15.8 with one token per wave.

// Reductions over the L lanes of a token; every lane gets the result.
template <int L, typename F>
__device__ __forceinline__ uint32_t token_reduce(uint32_t v, F&& f) {
  auto step = [&](uint32_t o) { v = f(v, o); };
  step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));
  step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));
  step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, false)));
  step(uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xF, 0xF, false)));
  if constexpr (L >= 32) {
    const auto h = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(h[0], h[1]);
  }
  if constexpr (L >= 64) {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(h[0], h[1]);
  }
  return v;
}
template <int L> __device__ __forceinline__ uint32_t token_max(uint32_t v) {
  return token_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L> __device__ __forceinline__ uint32_t token_min(uint32_t v) {
  return token_reduce<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int L> __device__ __forceinline__ float token_sum(float v) {
  return __uint_as_float(token_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// The R logits of lane l of token t; -inf behind E and for t >= T.
template <int BF16, int R>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int64_t T, int E, int l, float (&v)[R]) {
  using El = Elem<BF16>;
  const typename El::T* row = reinterpret_cast<const typename El::T*>(logits) + (t < T ? t : T - 1) * E;
  constexpr int P = El::kPer16;
  if constexpr (R % P == 0) {
    if (l * R + R <= E) {
#pragma unroll
      for (int c = 0; c < R / P; ++c) {
        float f[P];
        El::unpack(ld16_any(row + l * R + c * P), f);
#pragma unroll
        for (int i = 0; i < P; ++i) v[c * P + i] = f[i];
      }
      return;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = l * R + r < E ? El::get(row[l * R + r]) : -INFINITY;
}

// Each of the top_k picks is the largest key of the token and among equal ones the
// lowest index.  A bfloat16 logit's key (16 bits) and its index make one 26-bit
// number, so one maximum finds both, and "smaller than the last pick" replaces the
// taking away: key - last wraps to the top for every key below it.  A float32
// key fills the 32 bits; there the index comes from a second reduction.
// Slot j waits in LDS for the weights.  Softmax in float32 from the
// first pick.
constexpr int kRouteThreads = 256;

template <int BF16, int L, int R>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const void* __restrict__ logits,
                                                              int32_t* __restrict__ ids, float* __restrict__ weights,
                                                              int64_t T, int E, int top_k, int renorm) {
  constexpr int kTokens = kRouteThreads / L;
  __shared__ int32_t pick_id[kTokens][64];
  __shared__ float pick_logit[kTokens][64];
  const int l = threadIdx.x % L, tok = threadIdx.x / L;
  for (int64_t t0 = int64_t(blockIdx.x) * kTokens; t0 < T; t0 += int64_t(gridDim.x) * kTokens) {
    const int64_t t = t0 + tok;
    float v[R];
    load_logits<BF16>(logits, t, T, E, l, v);
    uint32_t key[R];
    bool nan = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t k = order_key(v[r]);
      key[r] = BF16 ? (k >> 16 ? (k >> 16) << 10 | uint32_t(1023 - (l * R + r)) : 0u) : k;
      nan |= v[r] != v[r];
    }
    float top = 0.f;
    uint32_t last = 1u << 30;  // above every bfloat16 key
    for (int j = 0; j < top_k; ++j) {
      int32_t id;
      float logit;
      bool any;
      if constexpr (BF16) {
        uint32_t best = key[0] - last;
#pragma unroll
        for (int r = 1; r < R; ++r) best = max(best, key[r] - last);
        const uint32_t m = token_max<L>(best) + last;
        any = m - 1u < last - 1u;  // 0 < m < last
        if (!any) {  // nothing is left of this token
          id = -1;
          logit = -INFINITY;
        } else {
          id = 1023 - int(m & 1023u);
          logit = __uint_as_float(__float_as_uint(key_value((m >> 10) << 16)) & 0xFFFF0000u);
          last = m;
        }
      } else {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int r = 1; r < R; ++r)
          if (key[r] > best) {
            best = key[r];
            at = r;
          }
        const uint32_t m = token_max<L>(best);
        const uint32_t e = token_min<L>(best == m ? uint32_t(l * R + at) : 0xFFFFFFFFu);
        any = m != 0;
        id = any ? int32_t(e) : -1;
        logit = any ? key_value(m) : -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r) key[r] = uint32_t(l * R + r) == e ? 0u : key[r];
      }
      if (j == 0 && any) top = logit;
      if (l == 0) {
        pick_id[tok][j] = id;
        pick_logit[tok][j] = logit;
      }
    }
    const bool any_nan = token_max<L>(nan ? 1u : 0u) != 0;
    wait_lds();  // the token's lanes are in one wave
    float part = 0.f;
    if (renorm) {
      for (int j = l; j < top_k; j += L) part += pick_id[tok][j] >= 0 ? expf(pick_logit[tok][j] - top) : 0.f;
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) part += v[r] > -INFINITY ? expf(v[r] - top) : 0.f;
    }
    const float total = token_sum<L>(part);
    if (t < T)
      for (int j = l; j < top_k; j += L) {
        const int32_t id = pick_id[tok][j];
        const float p = id >= 0 ? expf(pick_logit[tok][j] - top) : 0.f;
        ids[t * top_k + j] = id;
        // A row of which nothing is left has total 0 and weights 0.
        weights[t * top_k + j] = any_nan ? NAN : total != 0.f ? p / total : 0.f;
      }
    wait_lds();
  }
}

// dl_e = p_e (a_e - mean): a_e the gradient of the weight of a chosen expert
// (0 otherwise), p_e its softmax value, mean = sum of p a over the chosen.
// With renormalised weights the softmax runs over the chosen ones only, so only their logits
// are read, and every other gradient is 0.  Lane layout of the router; a row (the
// chosen experts' gradients, or with renormalised weights the result) lies in LDS,
// where the chosen lanes put what belongs to their experts.  T = 16384, E = 256, bfloat16:
// 7.8 us, 2.2 TB/s; bound by the vector instructions of the softmax, which fill 69 % of the SIMDs'
// cycles while their CUs have work (the router's 87 %).
template <int BF16, int L, int R>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(const void* __restrict__ logits,
                                                                       const int32_t* __restrict__ ids,
                                                                       const float* __restrict__ dw,
                                                                       void* __restrict__ dlogits, int64_t T, int E,
                                                                       int top_k, int renorm) {
  using El = Elem<BF16>;
  constexpr int kTokens = kRouteThreads / L;
  __shared__ __attribute__((aligned(16))) float rows[kTokens][L * R];
  const int l = threadIdx.x % L, tok = threadIdx.x / L;
  float* row = rows[tok];
  for (int64_t t0 = int64_t(blockIdx.x) * kTokens; t0 < T; t0 += int64_t(gridDim.x) * kTokens) {
    const int64_t t = t0 + tok;
    const int64_t tc = t < T ? t : T - 1;
    float v[R];
    if (!renorm) load_logits<BF16>(logits, t, T, E, l, v);
#pragma unroll
    for (int r = 0; r < R; ++r) row[l * R + r] = 0.f;
    wait_lds();
    float top = -INFINITY, part = 0.f, dot = 0.f;
    if (renorm) {
      const typename El::T* lg = reinterpret_cast<const typename El::T*>(logits) + tc * E;
      for (int j = l; j < top_k; j += L) {
        const int id = ids[tc * top_k + j];
        if (id >= 0 && id < E) top = fmaxf(top, El::get(lg[id]));
      }
      const uint32_t m = token_max<L>(order_key(top));
      top = m ? key_value(m) : 0.f;
      for (int j = l; j < top_k; j += L) {
        const int id = ids[tc * top_k + j];
        if (id < 0 || id >= E) continue;
        const float x = El::get(lg[id]), p = x == -INFINITY ? 0.f : expf(x - top);
        part += p;
        dot = fmaf(p, dw[tc * top_k + j], dot);
      }
      const float total = token_sum<L>(part), inv = total != 0.f ? 1.f / total : 0.f;
      const float mean = token_sum<L>(dot) * inv;
      for (int j = l; j < top_k; j += L) {
        const int id = ids[tc * top_k + j];
        if (id < 0 || id >= E) continue;
        const float x = El::get(lg[id]), p = x == -INFINITY ? 0.f : expf(x - top);
        if (p != 0.f) atomicAdd(&row[id], p * inv * (dw[tc * top_k + j] - mean));  // one per expert: no order
      }
      wait_lds();
#pragma unroll
      for (int r = 0; r < R; ++r) v[r] = row[l * R + r];
    } else {
      for (int j = l; j < top_k; j += L) {
        const int id = ids[tc * top_k + j];
        if (id >= 0 && id < E) atomicAdd(&row[id], dw[tc * top_k + j]);
      }
      uint32_t best = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) best = max(best, order_key(v[r]));
      const uint32_t m = token_max<L>(best);
      top = m ? key_value(m) : 0.f;
      wait_lds();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v[r] = v[r] == -INFINITY ? 0.f : expf(v[r] - top);
        part += v[r];
        dot = fmaf(v[r], row[l * R + r], dot);
      }
      const float total = token_sum<L>(part), inv = total != 0.f ? 1.f / total : 0.f;
      const float mean = token_sum<L>(dot) * inv;
#pragma unroll
      for (int r = 0; r < R; ++r) v[r] = v[r] != 0.f ? v[r] * inv * (row[l * R + r] - mean) : 0.f;
    }
    if (t < T) {
      typename El::T* out = reinterpret_cast<typename El::T*>(dlogits) + t * E + l * R;
      constexpr int P = El::kPer16;
      bool done = false;
      if constexpr (R % P == 0) {
        if (l * R + R <= E) {
#pragma unroll
          for (int c = 0; c < R / P; ++c) {
            float f[P];
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = v[c * P + i];
            st16_any(out + c * P, El::pack(f));
          }
          done = true;
        }
      }
      if (!done)
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (l * R + r < E) out[r] = El::put(v[r]);
    }
    wait_lds();
  }
}

// ---------------------------------------------------------------- sort

// Stable counting sort of the slots s = token * top_k + choice by expert id;
// ids outside 0 .. E-1 go last (bin E).  Blocks take contiguous pieces of
// slots and, inside a block, waves contiguous pieces of those, so a row is
//   start of its bin + the bin's slots in earlier pieces + its rank in the
//   wave's piece,
// with no atomic whose order could matter: counts come from LDS atomics
// (sums only), ranks from ballots.  Bound by latency, the way from the ids over the counts to
// the places: 64 slots 4.8 us (one launch), 131072 slots of 256 experts 4.9 to count
// and 9.3 to place.
constexpr int kSortWaves = 8;
constexpr int kSortThreads = kSortWaves * kWave;
constexpr int kSortMaxBins = 1025;

__device__ __forceinline__ int sort_bin(const int32_t* ids, int64_t s, int E) {
  const int id = ids[s];
  return id >= 0 && id < E ? id : E;
}

// Counts of each wave's piece: cnt[w * bins + b].  Ends with a barrier.
__device__ __forceinline__ void sort_count(int* cnt, const int32_t* __restrict__ ids, int64_t lo, int64_t hi, int E) {
  const int bins = E + 1, wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  for (int i = threadIdx.x; i < kSortWaves * bins; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  for (int64_t s = lo + lane; s < hi; s += kWave) atomicAdd(&cnt[wave * bins + sort_bin(ids, s, E)], 1);
  __syncthreads();
}

// The wave's slots [lo, hi) of a block's piece of `per` slots from `first`.
__device__ __forceinline__ void sort_span(int64_t first, int64_t per, int64_t S, int64_t& lo, int64_t& hi) {
  const int wave = threadIdx.x / kWave;
  const int64_t pw = (per + kSortWaves - 1) / kSortWaves;
  const int64_t end = first + per < S ? first + per : S;
  lo = first + wave * pw;
  hi = lo + pw < end ? lo + pw : end;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int32_t* __restrict__ ids,
                                                                  int32_t* __restrict__ hist, int64_t S, int E,
                                                                  int64_t per) {
  __shared__ int cnt[kSortWaves * kSortMaxBins];
  const int bins = E + 1;
  int64_t lo, hi;
  sort_span(int64_t(blockIdx.x) * per, per, S, lo, hi);
  sort_count(cnt, ids, lo, hi, E);
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    int n = 0;
    for (int w = 0; w < kSortWaves; ++w) n += cnt[w * bins + b];
    hist[int64_t(b) * gridDim.x + blockIdx.x] = n;  // a bin's counts side by side
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int32_t* __restrict__ ids,
                                                                  const int32_t* __restrict__ hist,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ row_slot,
                                                                  int32_t* __restrict__ slot_row, int64_t S, int E,
                                                                  int64_t per) {
  __shared__ int cnt[kSortWaves * kSortMaxBins];  // becomes the next row of each (wave, bin)
  __shared__ int wave_total[kSortWaves];
  const int bins = E + 1, wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int blocks = gridDim.x;
  int64_t lo, hi;
  sort_span(int64_t(blockIdx.x) * per, per, S, lo, hi);
  sort_count(cnt, ids, lo, hi, E);
  int carry = 0;  // rows of the bins before this pass
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int b = b0 + int(threadIdx.x);
    int total = 0, before = 0;  // the bin's slots in all blocks, and in earlier ones
    if (b < bins) {
      if (blocks > 1) {
        const int32_t* h = hist + int64_t(b) * blocks;
#pragma unroll 16
        for (int k = 0; k < blocks; ++k) {  // loads in flight together
          const int n = h[k];
          total += n;
          before += k < int(blockIdx.x) ? n : 0;
        }
      } else {
        for (int w = 0; w < kSortWaves; ++w) total += cnt[w * bins + b];
      }
    }
    int incl = total;  // prefix sum over the bins: the wave's, then the waves'
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(incl, d, kWave);
      if (lane >= d) incl += o;
    }
    if (lane == kWave - 1) wave_total[wave] = incl;
    __syncthreads();
    int base = carry, all = 0;
    for (int w = 0; w < kSortWaves; ++w) {
      base += w < wave ? wave_total[w] : 0;
      all += wave_total[w];
    }
    carry += all;
    if (b < bins) {
      const int start = base + incl - total;
      if (blockIdx.x == 0) offsets[b] = start;
      int next = start + before;
      for (int w = 0; w < kSortWaves; ++w) {
        const int n = cnt[w * bins + b];
        cnt[w * bins + b] = next;
        next += n;
      }
    }
    __syncthreads();
  }
  volatile int* next = cnt + wave * bins;  // this wave's own counters from here on
  const int bits = 32 - __builtin_clz(E);
  for (int64_t s0 = lo; s0 < hi; s0 += kWave) {
    const int64_t s = s0 + lane;
    const bool on = s < hi;
    const int bin = on ? sort_bin(ids, s, E) : 0;
    uint64_t peers = __ballot(on);  // lanes of this step with the same bin
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((bin >> b) & 1);
      peers &= ((bin >> b) & 1) ? m : ~m;
    }
    const int rank = __popcll(peers & ((uint64_t(1) << lane) - 1));
    const int row = on ? next[bin] + rank : 0;
    __builtin_amdgcn_wave_barrier();
    if (on && rank == 0) next[bin] = row + __popcll(peers);
    __builtin_amdgcn_wave_barrier();
    if (on) {
      const bool live = bin < E;
      row_slot[row] = live ? int32_t(s) : ~int32_t(s);
      slot_row[s] = live ? row : ~row;
    }
  }
}

// ---------------------------------------------------------------- gather and combine

// These move rows and are bound by HBM.  What they need is many loads in flight: the
// slots of a token (or the pieces of a row) are taken a handful at a time, first their
// places, then all their bytes, and a wave that has more to do reads its
// next places while the bytes are on their way.
constexpr int kBatch = 8;

// Waves walk (token, piece of 64 x 16 bytes of its row); 2^split waves of a block share a
// token.  f(t, h): h = the lane's first element.
template <int P, typename F>
__device__ __forceinline__ void walk_tokens(int64_t T, int64_t H, int split, F&& f) {
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int per_block = 4 >> split, span = kWave * P;
  for (int64_t t = int64_t(blockIdx.x) * per_block + (wave >> split); t < T; t += int64_t(gridDim.x) * per_block)
    for (int64_t h = int64_t(wave & ((1 << split) - 1)) * span; h < H; h += int64_t(span) << split) f(t, h + lane * P);
}

// The place and weight of up to kBatch slots from p on; row -1 for those that are
// dropped, foreign or behind `left`.  Uniform over the wave: scalar loads and registers.
struct Slots {
  int32_t row[kBatch];
  float w[kBatch];
};
__device__ __forceinline__ Slots load_slots(const int32_t* p, const float* w, int left, int64_t count) {
  Slots s;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int j = i < left ? i : 0;
    const int32_t q = __builtin_amdgcn_readfirstlane(p[j]);
    s.row[i] = i < left && q < count ? q : -1;
    s.w[i] = w ? __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(w[j]))) : 1.f;
  }
  return s;
}

// The token's bytes are read once and stored to each of its top_k rows; a
// dropped slot (~row) clears the row it pads.  16384 tokens of 2048 bfloat16, top 8: 120 us, 5.0 TB/s
// read and written, the rate of a copy.
template <int BF16, bool NT>
__global__ __launch_bounds__(256) void gather_kernel(const void* __restrict__ x, const int32_t* __restrict__ slot_row,
                                                     void* __restrict__ out, int64_t T, int top_k, int64_t H,
                                                     int split) {
  using El = Elem<BF16>;
  using V = typename El::T;
  const int64_t S = T * top_k;
  walk_tokens<El::kPer16>(T, H, split, [&](int64_t t, int64_t h) {
    const V* src = reinterpret_cast<const V*>(x) + t * H + h;
    V* dst = reinterpret_cast<V*>(out) + h;
    if (h + El::kPer16 <= H) {
      const u32x4 v = ld16_any(src);
#pragma unroll 4
      for (int j = 0; j < top_k; ++j) {
        const int32_t q = slot_row[t * top_k + j];
        const int64_t row = q < 0 ? ~q : q;
        if (row < S) st16_at<NT>(dst + row * H, q < 0 ? u32x4{0u, 0u, 0u, 0u} : v);
      }
    } else if (h < H) {
      for (int j = 0; j < top_k; ++j) {
        const int32_t q = slot_row[t * top_k + j];
        const int64_t row = q < 0 ? ~q : q;
        if (row >= S) continue;
        for (int i = 0; h + i < H; ++i) dst[row * H + i] = q < 0 ? V(0) : src[i];
      }
    }
  });
}

// out[t] = sum over the token's live slots, in slot order, of weight x row,
// in float32, rounded once.  The same sizes: 114 us, 5.3 TB/s.
template <int BF16, int OBF16, bool NT>
__global__ __launch_bounds__(256, 6) void combine_kernel(const void* __restrict__ rows,
                                                         const int32_t* __restrict__ slot_row,
                                                         const float* __restrict__ weights, void* __restrict__ out,
                                                         int64_t T, int top_k, int64_t H, int split) {
  using El = Elem<BF16>;
  using V = typename El::T;
  using O = typename Elem<OBF16>::T;
  constexpr int P = El::kPer16;
  const int64_t S = T * top_k;
  walk_tokens<P>(T, H, split, [&](int64_t t, int64_t h) {
    const V* src = reinterpret_cast<const V*>(rows) + h;
    O* dst = reinterpret_cast<O*>(out) + t * H + h;
    const int32_t* place = slot_row + t * top_k;
    const float* weight = weights ? weights + t * top_k : nullptr;
    float acc[P];
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] = 0.f;
    if (h + P <= H) {
      Slots s = load_slots(place, weight, top_k, S);
      for (int j0 = 0; j0 < top_k; j0 += kBatch) {
        u32x4 b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (s.row[i] >= 0) b[i] = ld16_at<NT>(src + int64_t(s.row[i]) * H);  // uniform
        Slots next;
        if (j0 + kBatch < top_k)
          next = load_slots(place + j0 + kBatch, weight ? weight + j0 + kBatch : nullptr, top_k - j0 - kBatch, S);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (s.row[i] < 0) continue;  // a dropped slot's weight is not used, whatever it is
          float f[P];
          El::unpack(b[i], f);
#pragma unroll
          for (int c = 0; c < P; ++c) acc[c] = fmaf(s.w[i], f[c], acc[c]);
        }
        s = next;
      }
      if constexpr (BF16 == OBF16) {
        st16_any(dst, El::pack(acc));
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) dst[i] = Elem<OBF16>::put(acc[i]);
      }
    } else {
      for (int i = 0; h + i < H; ++i) {
        float a = 0.f;
        for (int j = 0; j < top_k; ++j) {
          const int32_t q = place[j];
          if (q >= 0 && q < S) a = fmaf(weight ? weight[j] : 1.f, El::get(src[int64_t(q) * H + i]), a);
        }
        dst[i] = Elem<OBF16>::put(a);
      }
    }
  });
}

// Gradients of the weighted sum: grad_rows[row] = w dy[t] and
// grad_weights[t, j] = <dy[t], rows[row]>.  One wave per slot, four pieces of the row
// in flight; the slots of a token run next to each other, so dy comes from the
// caches after the first.  4099 tokens of 4096 bfloat16, top 6: 86 us for 437 MB, 5.1 TB/s.
template <int BF16, bool NT>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const void* __restrict__ dy, const void* __restrict__ rows, const int32_t* __restrict__ slot_row,
    const float* __restrict__ weights, void* __restrict__ drows, float* __restrict__ dweights, int64_t S, int top_k,
    int64_t H) {
  using El = Elem<BF16>;
  using V = typename El::T;
  constexpr int P = El::kPer16, U = 4;
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t s = first_item(); s < S; s += item_stride()) {  // uniform per wave
    const int64_t t = s / top_k;
    const int32_t q = slot_row[s];
    const int64_t row = q < 0 ? ~q : q;
    if (row >= S) {
      if (lane == 0) dweights[s] = 0.f;
      continue;
    }
    const float w = weights[s];
    const V* g = reinterpret_cast<const V*>(dy) + t * H;
    const V* r = reinterpret_cast<const V*>(rows) + row * H;
    V* d = reinterpret_cast<V*>(drows) + row * H;
    float dot = 0.f;
    const int64_t whole = H / P * P;
    for (int64_t h0 = int64_t(lane) * P; h0 < whole; h0 += U * kWave * P) {
      u32x4 a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t h = h0 + u * kWave * P;
        a[u] = b[u] = u32x4{0u, 0u, 0u, 0u};
        if (h < whole && q >= 0) {
          a[u] = ld16_any(g + h);
          b[u] = ld16_at<NT>(r + h);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t h = h0 + u * kWave * P;
        float fa[P], fb[P];
        El::unpack(a[u], fa);
        El::unpack(b[u], fb);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          dot = fmaf(fa[i], fb[i], dot);
          fa[i] *= w;
        }
        if (h < whole) st16_at<NT>(d + h, q < 0 ? u32x4{0u, 0u, 0u, 0u} : El::pack(fa));
      }
    }
    if (whole + lane < H) {
      const int64_t h = whole + lane;
      const float a = q < 0 ? 0.f : El::get(g[h]);
      if (q >= 0) dot = fmaf(a, El::get(r[h]), dot);
      d[h] = q < 0 ? V(0) : El::put(a * w);
    }
    dot = wave_sum(dot);
    if (lane == 0) dweights[s] = q < 0 ? 0.f : dot;
  }
}

// ---------------------------------------------------------------- gated activation

// What sigmoid(g) and sigmoid(-g) are made of, from h = exp(-|g| / 2): near = 1 / (1 + h^2) =
// sigmoid(|g|); half = 1 for g >= 0, else h, so that sigmoid(g) = half^2 near; rest = sigmoid(-g).  Nothing
// overflows or cancels.  A negative gate's two halves go to different factors of a
// product: h^2 leaves float32's normal range below g = -87 (and the exponential instruction gives 0
// there), where its product with u or dy need not, and h only below g = -174.
// Good to a few float32 roundings (u = 2^-24): |g| log2(e) / 2 is taken with the
// rounding error of its product, so h is off by 3 u (the instruction itself by 2) and h^2 by 7, 1 + h^2
// adds one, and a Newton step leaves one of the reciprocal.  Beyond |g| = 256 nothing changes (h = 0).
// The library's expf and division would be twice the instructions, and the forward pass over
// bfloat16 was bound by them.
__device__ __forceinline__ void sigmoids(float g, float& near, float& half, float& rest) {
  constexpr float kHi = 0.5f * 1.44269502f, kLo = 0.5f * 1.92596299e-8f;  // log2(e) / 2
  const float a = fminf(fabsf(g), 256.f);
  const float t = -a * kHi;
  const float r = fmaf(-a, kLo, fmaf(-a, kHi, -t));
  float h = __builtin_amdgcn_exp2f(t);
  h = fmaf(h, r * 0.693147182f, h);
  const float d = fmaf(h, h, 1.f), y = __builtin_amdgcn_rcpf(d);
  near = fmaf(y, fmaf(-d, y, 1.f), y);
  half = g >= 0.f ? 1.f : h;
  rest = g >= 0.f ? h * h * near : near;
}

__device__ __forceinline__ float swiglu_one(float g, float u) {
  float near, half, rest;
  sigmoids(g, near, half, rest);
  return (g * near * half) * (u * half);
}

// dgate = dy u sig (1 + g (1 - sig)), dup = dy g sig, with sigmoid(-g) for 1 - sig.  dy u alone
// could overflow where the gradient does not.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dy, float& dg, float& du) {
  float near, half, rest;
  sigmoids(g, near, half, rest);
  const float dh = dy * half;
  dg = dh * (u * half) * (near * fmaf(g, rest, 1.f));
  du = dh * (g * near * half);
}

// n / d for n < 2^31 as a product: m = floor(2^(31 + l) / d) + 1 with l = ceil(log2 d) is
// off by less than 2^-31 of itself, so n m / 2^(31 + l) by less than 1 / d.
struct Divisor {
  uint32_t d, m;
  int l;
  explicit Divisor(uint32_t v) : d(v), m(0), l(0) {
    while ((uint64_t(1) << l) < v) ++l;
    m = uint32_t((uint64_t(1) << (31 + l)) / v + 1);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const {
    return l == 0 ? n : uint32_t((uint64_t(n) * m) >> 31) >> l;
  }
};

// x: [M, 2F], gate columns first.  Thread item = 16 bytes of one row's half.  Bound by HBM: 32768 x 1536,
// bfloat16, 47 us, 6.4 TB/s; the gradient of 4100 x 1535 in float32 22 us, 5.7 TB/s.
template <int BF16, bool BACK, bool NT>
__global__ __launch_bounds__(256) void swiglu_kernel(const void* __restrict__ x, const void* __restrict__ dy,
                                                     void* __restrict__ out, uint32_t items, int64_t F,
                                                     Divisor per_row) {
  using El = Elem<BF16>;
  using V = typename El::T;
  constexpr int P = El::kPer16;
  const uint32_t item = blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= items) return;
  const uint32_t row = per_row.of(item);
  const int64_t m = row;
  const int64_t f = int64_t(item - row * per_row.d) * P;
  const V* gp = reinterpret_cast<const V*>(x) + m * 2 * F + f;
  const V* up = gp + F;
  const V* dp = BACK ? reinterpret_cast<const V*>(dy) + m * F + f : nullptr;
  V* op = reinterpret_cast<V*>(out) + (BACK ? m * 2 * F : m * F) + f;
  if (f + P <= F) {
    float g[P], u[P];
    const u32x4 gv = ld16_at<NT>(gp), uv = ld16_at<NT>(up);
    El::unpack(gv, g);
    El::unpack(uv, u);
    if constexpr (BACK) {
      float d[P];
      El::unpack(ld16_at<NT>(dp), d);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float a, b;
        swiglu_grad(g[i], u[i], d[i], a, b);
        g[i] = a;
        u[i] = b;
      }
      st16_at<NT>(op, El::pack(g));
      st16_at<NT>(op + F, El::pack(u));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) g[i] = swiglu_one(g[i], u[i]);
      st16_at<NT>(op, El::pack(g));
    }
  } else {
    for (int i = 0; f + i < F; ++i) {
      const float g = El::get(gp[i]), u = El::get(up[i]);
      if constexpr (BACK) {
        float a, b;
        swiglu_grad(g, u, El::get(dp[i]), a, b);
        op[i] = El::put(a);
        op[F + i] = El::put(b);
      } else {
        op[i] = El::put(swiglu_one(g, u));
      }
    }
  }
}

// Calls that move more than this go past the caches.  Above it: sort, gather and combine of 16384
// tokens (604 MB each way) 231 us, 266 through the caches; a combine and its gradients (672 MB) 125 and 141; the
// activation of 302 MB 46.5 and 50.7.  Below it the next operator finds the rows in the 256 MB cache (a
// gradient of 126 MB: 20.4 us, 22.6 past it).
constexpr int64_t kNtBytes = int64_t(160) << 20;

template <typename F> hipError_t by_size(int64_t bytes, F&& go) {
  return bytes > kNtBytes ? go(std::integral_constant<bool, true>{}) : go(std::integral_constant<bool, false>{});
}

// Lanes per token and logits per lane.
template <int L_, int R_> struct RouteWidth {
  static constexpr int L = L_, R = R_;
};
template <typename F>
hipError_t route_by_width(int E, F&& go) {
  if (E <= 16) return go(RouteWidth<16, 1>{});
  if (E <= 64) return go(RouteWidth<16, 4>{});
  if (E <= 128) return go(RouteWidth<16, 8>{});
  if (E <= 256) return go(RouteWidth<16, 16>{});
  if (E <= 512) return go(RouteWidth<32, 16>{});
  return go(RouteWidth<64, 16>{});
}

dim3 blocks_for(int64_t items, int per_block) {
  const int64_t b = (items + per_block - 1) / per_block;
  return dim3(unsigned(b < kMaxBlocks ? b : kMaxBlocks));
}

int64_t sort_blocks(int64_t S, int64_t* per) {
  // One block up to 4096 slots; beyond, pieces of 2048, growing so that at
  // most 128 blocks read each other's counts.
  if (S <= 4096) {
    *per = S;
    return 1;
  }
  *per = (S + 127) / 128;
  if (*per < 2048) *per = 2048;
  return (S + *per - 1) / *per;
}

}  // namespace

hipError_t launch_moe_route(const void* logits, int bf16, int32_t* ids, float* weights, int64_t T, int64_t E,
                            int64_t top_k, int renorm, hipStream_t s) {
  return route_by_width(int(E), [&](auto w) {
    const dim3 grid = blocks_for(T, kRouteThreads / w.L), block(kRouteThreads);
    auto go = [&](auto kernel) {
      return launch(kernel, grid, block, 0, s, logits, ids, weights, T, int(E), int(top_k), renorm);
    };
    return bf16 ? go(route_kernel<1, w.L, w.R>) : go(route_kernel<0, w.L, w.R>);
  });
}

hipError_t launch_moe_route_backward(const void* logits, int bf16, const int32_t* ids, const float* dw, void* dlogits,
                                     int64_t T, int64_t E, int64_t top_k, int renorm, hipStream_t s) {
  return route_by_width(int(E), [&](auto w) {
    const dim3 grid = blocks_for(T, kRouteThreads / w.L), block(kRouteThreads);
    auto go = [&](auto kernel) {
      return launch(kernel, grid, block, 0, s, logits, ids, dw, dlogits, T, int(E), int(top_k), renorm);
    };
    return bf16 ? go(route_backward_kernel<1, w.L, w.R>) : go(route_backward_kernel<0, w.L, w.R>);
  });
}

size_t moe_sort_ws_bytes(int64_t S, int64_t E) {
  if (S <= 0) return 0;
  int64_t per;
  const int64_t blocks = sort_blocks(S, &per);
  return blocks > 1 ? size_t(blocks) * size_t(E + 1) * 4 : 0;
}

hipError_t launch_moe_sort(const int32_t* ids, int32_t* offsets, int32_t* row_slot, int32_t* slot_row, int64_t S,
                           int64_t E, int32_t* ws, hipStream_t s) {
  int64_t per;
  const int64_t blocks = sort_blocks(S, &per);
  if (blocks > 1) {
    if (hipError_t e = launch(sort_count_kernel, dim3(blocks), dim3(kSortThreads), 0, s, ids, ws, S, int(E), per))
      return e;
  }
  return launch(sort_place_kernel, dim3(blocks), dim3(kSortThreads), 0, s, ids, ws, offsets, row_slot, slot_row, S,
                int(E), per);
}

// Waves of a block per token: as many as the row has pieces, 4 at most.
int token_split(int64_t H, int bf16) {
  const int64_t span = kWave * (bf16 ? 8 : 4);
  return H <= span ? 0 : H <= 2 * span ? 1 : 2;
}

hipError_t launch_moe_gather(const void* x, const int32_t* slot_row, void* out, int bf16, int64_t T, int64_t top_k,
                             int64_t H, hipStream_t s) {
  const int split = token_split(H, bf16);
  const dim3 grid = blocks_for(T, 4 >> split), block(256);
  return by_size(T * (top_k + 1) * H * (bf16 ? 2 : 4), [&](auto nt) {
    if (bf16) return launch(gather_kernel<1, nt.value>, grid, block, 0, s, x, slot_row, out, T, int(top_k), H, split);
    return launch(gather_kernel<0, nt.value>, grid, block, 0, s, x, slot_row, out, T, int(top_k), H, split);
  });
}

hipError_t launch_moe_combine(const void* rows, int bf16, const int32_t* slot_row, const float* weights, void* out,
                              int out_bf16, int64_t T, int64_t top_k, int64_t H, hipStream_t s) {
  const int split = token_split(H, bf16);
  const dim3 grid = blocks_for(T, 4 >> split), block(256);
  return by_size(T * (top_k + 1) * H * (bf16 ? 2 : 4), [&](auto nt) {
    constexpr bool NT = nt.value;
    auto go = [&](auto kernel) {
      return launch(kernel, grid, block, 0, s, rows, slot_row, weights, out, T, int(top_k), H, split);
    };
    if (bf16) return out_bf16 ? go(combine_kernel<1, 1, NT>) : go(combine_kernel<1, 0, NT>);
    return out_bf16 ? go(combine_kernel<0, 1, NT>) : go(combine_kernel<0, 0, NT>);
  });
}

hipError_t launch_moe_combine_backward(const void* dy, const void* rows, int bf16, const int32_t* slot_row,
                                       const float* weights, void* drows, float* dweights, int64_t T, int64_t top_k,
                                       int64_t H, hipStream_t s) {
  const int64_t S = T * top_k;
  const dim3 grid = blocks_for(S, 4), block(256);
  return by_size((2 * S + T) * H * (bf16 ? 2 : 4), [&](auto nt) {
    auto go = [&](auto kernel) {
      return launch(kernel, grid, block, 0, s, dy, rows, slot_row, weights, drows, dweights, S, int(top_k), H);
    };
    return bf16 ? go(combine_backward_kernel<1, nt.value>) : go(combine_backward_kernel<0, nt.value>);
  });
}

hipError_t launch_swiglu(const void* x, const void* dy, void* out, int bf16, int64_t M, int64_t F, hipStream_t s) {
  const int64_t es = bf16 ? 2 : 4, per_row = (F * es + 15) / 16, most = (int64_t(1) << 31) - 1;
  if (per_row > most) return hipErrorInvalidValue;
  // Items are counted in 31 bits: more rows take more launches.
  for (int64_t m0 = 0; m0 < M; m0 += most / per_row) {
    const int64_t rows = M - m0 < most / per_row ? M - m0 : most / per_row, items = rows * per_row;
    const char* px = static_cast<const char*>(x) + m0 * 2 * F * es;
    const char* pd = dy ? static_cast<const char*>(dy) + m0 * F * es : nullptr;
    char* po = static_cast<char*>(out) + m0 * F * es * (dy ? 2 : 1);
    const dim3 grid(unsigned((items + 255) / 256)), block(256);
    const hipError_t e = by_size(rows * F * es * (dy ? 5 : 3), [&](auto nt) {
      constexpr bool NT = nt.value;
      auto go = [&](auto kernel) {
        return launch(kernel, grid, block, 0, s, px, pd, po, uint32_t(items), F, Divisor(uint32_t(per_row)));
      };
      if (dy) return bf16 ? go(swiglu_kernel<1, true, NT>) : go(swiglu_kernel<0, true, NT>);
      return bf16 ? go(swiglu_kernel<1, false, NT>) : go(swiglu_kernel<0, false, NT>);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qlinear
