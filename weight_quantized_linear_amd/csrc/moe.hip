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
struct __attribute__((packed, aligned(2))) Unaligned16 {
  u32x4 v;
};
__device__ __forceinline__ u32x4 ld16_any(const void* p) { return reinterpret_cast<const Unaligned16*>(p)->v; }
__device__ __forceinline__ void st16_any(void* p, u32x4 v) { reinterpret_cast<Unaligned16*>(p)->v = v; }

template <int BF16> struct Elem;
template <> struct Elem<1> {
  using T = uint16_t;
  static constexpr int kPer16 = 8;
  static __device__ __forceinline__ float get(T v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ T put(float v) { return f32_to_bf16(v); }
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
    for (int i = 0; i < 4; ++i) v[i] = uint32_t(f32_to_bf16(f[2 * i])) | uint32_t(f32_to_bf16(f[2 * i + 1])) << 16;
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

template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROW_MASK, 0xF, false));
  return v > o ? v : o;
}

// Largest unsigned value over the wave, in every lane (the steps of wave_sum).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  v = dpp_max<0x140>(v);
  v = dpp_max<0x142, 0xA>(v);
  v = dpp_max<0x143, 0xC>(v);
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

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

template <int BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t i) {
  return Elem<BF16>::get(reinterpret_cast<const typename Elem<BF16>::T*>(logits)[i]);
}

// ---------------------------------------------------------------- router

// One wave per token; lane l holds the R logits e = l R .. l R + R - 1, so of
// equal logits the lowest lane's first one has the lowest index.  Each of the
// k picks is a wave maximum over the lanes' best keys; the winning lane drops
// its key.  Lane j keeps pick j.  Softmax in float32 from the row's maximum
// (the first pick).
template <int BF16, int R>
__global__ __launch_bounds__(256) void route_kernel(const void* __restrict__ logits, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights, int64_t T, int E, int top_k,
                                                    int renorm) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t t = first_item(); t < T; t += item_stride()) {  // uniform per wave
    float v[R];
    uint32_t key[R];
    bool nan = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = lane * R + r;
      v[r] = e < E ? load_logit<BF16>(logits, t * E + e) : -INFINITY;
      key[r] = order_key(v[r]);
      nan |= v[r] != v[r];
    }
    const bool any_nan = __ballot(nan) != 0;
    int my_id = -1;
    float my_logit = -INFINITY;
    float top = 0.f;
    for (int j = 0; j < top_k; ++j) {
      uint32_t best = key[0];
      int at = 0;
#pragma unroll
      for (int r = 1; r < R; ++r)
        if (key[r] > best) {
          best = key[r];
          at = r;
        }
      const uint32_t m = wave_max(best);
      if (m == 0) break;  // nothing is left to choose
      const int src = __builtin_ctzll(__ballot(best == m));
      const int e = __builtin_amdgcn_readlane(lane * R + at, src);
      if (j == 0) top = key_value(m);
      if (lane == j) {
        my_id = e;
        my_logit = key_value(m);
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (lane == src && r == at) key[r] = 0;
    }
    const float p = my_id >= 0 ? expf(my_logit - top) : 0.f;
    float total;
    if (renorm) {
      total = wave_sum(p);
    } else {
      float part = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) part += v[r] > -INFINITY ? expf(v[r] - top) : 0.f;
      total = wave_sum(part);
    }
    if (lane < top_k) {
      const int64_t i = t * top_k + lane;
      ids[i] = my_id;
      // A row of which nothing is left has total 0 and weights 0.
      weights[i] = any_nan ? NAN : total != 0.f ? p / total : 0.f;
    }
  }
}

// dl_e = p_e (a_e - mean): a_e the gradient of the weight of a chosen expert
// (0 otherwise), p_e its softmax value, mean = sum of p a over the chosen.
// With renormalised weights the softmax runs over the chosen ones only and
// every other gradient is 0.  One wave per token, lane layout of the router.
template <int BF16, int R>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ dw, void* __restrict__ dlogits,
                                                             int64_t T, int E, int top_k, int renorm) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t t = first_item(); t < T; t += item_stride()) {  // uniform per wave
    int id = -1;
    float g = 0.f;
    if (lane < top_k) {
      id = ids[t * top_k + lane];
      g = dw[t * top_k + lane];
      if (id < 0 || id >= E) id = -1;
    }
    float v[R], a[R];
    bool chosen[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = lane * R + r;
      v[r] = e < E ? load_logit<BF16>(logits, t * E + e) : -INFINITY;
      a[r] = 0.f;
      chosen[r] = false;
    }
    for (int j = 0; j < top_k; ++j) {
      const int e = __builtin_amdgcn_readlane(id, j);
      const float ge = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), j));
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (lane * R + r == e) {
          a[r] += ge;
          chosen[r] = true;
        }
    }
    uint32_t best = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t k = (chosen[r] || !renorm) ? order_key(v[r]) : 0u;
      best = k > best ? k : best;
    }
    const uint32_t m = wave_max(best);
    const float top = m ? key_value(m) : 0.f;
    float part = 0.f, dot = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = chosen[r] || !renorm;
      const float p = in && !(v[r] == -INFINITY) ? expf(v[r] - top) : 0.f;
      v[r] = p;
      part += p;
      dot += chosen[r] ? p * a[r] : 0.f;
    }
    const float total = wave_sum(part);
    const float inv = total != 0.f ? 1.f / total : 0.f;
    const float mean = wave_sum(dot) * inv;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = lane * R + r;
      const float d = v[r] != 0.f ? v[r] * inv * (a[r] - mean) : 0.f;
      if (e < E) reinterpret_cast<typename Elem<BF16>::T*>(dlogits)[t * E + e] = Elem<BF16>::put(d);
    }
  }
}

// ---------------------------------------------------------------- sort

// Stable counting sort of the slots s = token * top_k + choice by expert id;
// ids outside 0 .. E-1 go last (bin E).  Blocks take contiguous pieces of
// slots and, inside a block, waves contiguous pieces of those, so a row is
//   start of its bin + the bin's slots in earlier pieces + its rank in the
//   wave's piece,
// with no atomic whose order could matter: counts come from LDS atomics
// (sums only), ranks from ballots.
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
    hist[int64_t(blockIdx.x) * bins + b] = n;
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
        for (int k = 0; k < blocks; ++k) {
          const int n = hist[int64_t(k) * bins + b];
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

// Work item (token, piece of 64 x 16 bytes of its row) per wave: the token's
// bytes are read once and stored to each of its top_k rows; a dropped slot
// (~row) clears the row it pads.
template <int BF16>
__global__ __launch_bounds__(256) void gather_kernel(const void* __restrict__ x, const int32_t* __restrict__ slot_row,
                                                     void* __restrict__ out, int64_t T, int top_k, int64_t H,
                                                     int64_t pieces) {
  using El = Elem<BF16>;
  using V = typename El::T;
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t item = first_item(); item < T * pieces; item += item_stride()) {  // uniform per wave
    const int64_t t = item / pieces;
    const int64_t h = ((item - t * pieces) * kWave + lane) * El::kPer16;
    if (h >= H) continue;
    const int64_t S = T * top_k;
    const V* src = reinterpret_cast<const V*>(x) + t * H + h;
    V* dst = reinterpret_cast<V*>(out) + h;
    if (h + El::kPer16 <= H) {
      const u32x4 v = ld16_any(src);
      for (int j = 0; j < top_k; ++j) {
        const int32_t q = slot_row[t * top_k + j];
        const int64_t row = q < 0 ? ~q : q;
        if (row < S) st16_any(dst + row * H, q < 0 ? u32x4{0u, 0u, 0u, 0u} : v);
      }
    } else {
      for (int j = 0; j < top_k; ++j) {
        const int32_t q = slot_row[t * top_k + j];
        const int64_t row = q < 0 ? ~q : q;
        if (row >= S) continue;
        for (int i = 0; h + i < H; ++i) dst[row * H + i] = q < 0 ? V(0) : src[i];
      }
    }
  }
}

// out[t] = sum over the token's live slots, in slot order, of weight x row,
// in float32, rounded once.  Work items as in gather_kernel.
template <int BF16, int OBF16>
__global__ __launch_bounds__(256) void combine_kernel(const void* __restrict__ rows,
                                                      const int32_t* __restrict__ slot_row,
                                                      const float* __restrict__ weights, void* __restrict__ out,
                                                      int64_t T, int top_k, int64_t H, int64_t pieces) {
  using El = Elem<BF16>;
  using V = typename El::T;
  using O = typename Elem<OBF16>::T;
  constexpr int P = El::kPer16;
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t item = first_item(); item < T * pieces; item += item_stride()) {  // uniform per wave
    const int64_t t = item / pieces;
    const int64_t h = ((item - t * pieces) * kWave + lane) * P;
    if (h >= H) continue;
    const int64_t S = T * top_k;
    const V* src = reinterpret_cast<const V*>(rows) + h;
    O* dst = reinterpret_cast<O*>(out) + t * H + h;
    float acc[P];
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] = 0.f;
    const bool whole = h + P <= H;
    for (int j = 0; j < top_k; ++j) {
      const int64_t row = slot_row[t * top_k + j];
      if (row < 0 || row >= S) continue;  // uniform per wave
      const float w = weights ? weights[t * top_k + j] : 1.f;
      float f[P];
      if (whole) {
        El::unpack(ld16_any(src + row * H), f);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = h + i < H ? El::get(src[row * H + i]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] = fmaf(w, f[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (h + i < H) dst[i] = Elem<OBF16>::put(acc[i]);
  }
}

// Gradients of the weighted sum: grad_rows[row] = w dy[t] and
// grad_weights[t, j] = <dy[t], rows[row]>.  One wave per slot; the slots of a
// token run next to each other, so dy comes from the caches after the first.
template <int BF16>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const void* __restrict__ dy, const void* __restrict__ rows, const int32_t* __restrict__ slot_row,
    const float* __restrict__ weights, void* __restrict__ drows, float* __restrict__ dweights, int64_t S, int top_k,
    int64_t H) {
  using El = Elem<BF16>;
  using V = typename El::T;
  constexpr int P = El::kPer16;
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
    for (int64_t h = int64_t(lane) * P; h < H; h += kWave * P) {
      if (h + P <= H) {
        if (q < 0) {
          st16_any(d + h, u32x4{0u, 0u, 0u, 0u});
          continue;
        }
        float a[P], b[P];
        El::unpack(ld16_any(g + h), a);
        El::unpack(ld16_any(r + h), b);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          dot = fmaf(a[i], b[i], dot);
          a[i] *= w;
        }
        st16_any(d + h, El::pack(a));
      } else {
        for (int i = 0; h + i < H; ++i) {
          const float a = q < 0 ? 0.f : El::get(g[h + i]);
          if (q >= 0) dot = fmaf(a, El::get(r[h + i]), dot);
          d[h + i] = q < 0 ? V(0) : El::put(a * w);
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) dweights[s] = q < 0 ? 0.f : dot;
  }
}

// ---------------------------------------------------------------- gated activation

__device__ __forceinline__ float swiglu_one(float g, float u) { return mul_sigmoid(g, g) * u; }

// dgate = dy u sig (1 + g (1 - sig)), dup = dy g sig, with 1 - sig taken as
// the other branch of the same exponential, so that neither tail cancels.
__device__ __forceinline__ void swiglu_grad(float g, float u, float dy, float& dg, float& du) {
  const float e = expf(-fabsf(g));
  const float near = 1.f / (1.f + e), far = e * near;  // sigmoid of |g| and of -|g|
  const float sig = g >= 0.f ? near : far, rest = g >= 0.f ? far : near;
  dg = dy * u * sig * (1.f + g * rest);
  du = dy * g * sig;
}

// x: [M, 2F], gate columns first.  Thread item = 16 bytes of one row's half.
template <int BF16, bool BACK>
__global__ __launch_bounds__(256) void swiglu_kernel(const void* __restrict__ x, const void* __restrict__ dy,
                                                     void* __restrict__ out, int64_t M, int64_t F, int64_t per_row) {
  using El = Elem<BF16>;
  using V = typename El::T;
  constexpr int P = El::kPer16;
  const int64_t stride = int64_t(gridDim.x) * blockDim.x;
  for (int64_t item = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; item < M * per_row; item += stride) {
    const int64_t m = item / per_row;
    const int64_t f = (item - m * per_row) * P;
    const V* gp = reinterpret_cast<const V*>(x) + m * 2 * F + f;
    const V* up = gp + F;
    const V* dp = BACK ? reinterpret_cast<const V*>(dy) + m * F + f : nullptr;
    V* op = reinterpret_cast<V*>(out) + (BACK ? m * 2 * F : m * F) + f;
    if (f + P <= F) {
      float g[P], u[P];
      El::unpack(ld16_any(gp), g);
      El::unpack(ld16_any(up), u);
      if constexpr (BACK) {
        float d[P];
        El::unpack(ld16_any(dp), d);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float a, b;
          swiglu_grad(g[i], u[i], d[i], a, b);
          g[i] = a;
          u[i] = b;
        }
        st16_any(op, El::pack(g));
        st16_any(op + F, El::pack(u));
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) g[i] = swiglu_one(g[i], u[i]);
        st16_any(op, El::pack(g));
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
}

template <typename F>
hipError_t route_by_width(int E, F&& go) {
  if (E <= 64) return go(std::integral_constant<int, 1>{});
  if (E <= 128) return go(std::integral_constant<int, 2>{});
  if (E <= 256) return go(std::integral_constant<int, 4>{});
  if (E <= 512) return go(std::integral_constant<int, 8>{});
  return go(std::integral_constant<int, 16>{});
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
  const dim3 grid = blocks_for(T, 4), block(256);
  if (bf16)
    return route_by_width(int(E), [&](auto r) {
      return launch(route_kernel<1, decltype(r)::value>, grid, block, 0, s, logits, ids, weights, T, int(E),
                    int(top_k), renorm);
    });
  return route_by_width(int(E), [&](auto r) {
    return launch(route_kernel<0, decltype(r)::value>, grid, block, 0, s, logits, ids, weights, T, int(E), int(top_k),
                  renorm);
  });
}

hipError_t launch_moe_route_backward(const void* logits, int bf16, const int32_t* ids, const float* dw, void* dlogits,
                                     int64_t T, int64_t E, int64_t top_k, int renorm, hipStream_t s) {
  const dim3 grid = blocks_for(T, 4), block(256);
  if (bf16)
    return route_by_width(int(E), [&](auto r) {
      return launch(route_backward_kernel<1, decltype(r)::value>, grid, block, 0, s, logits, ids, dw, dlogits, T,
                    int(E), int(top_k), renorm);
    });
  return route_by_width(int(E), [&](auto r) {
    return launch(route_backward_kernel<0, decltype(r)::value>, grid, block, 0, s, logits, ids, dw, dlogits, T, int(E),
                  int(top_k), renorm);
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

hipError_t launch_moe_gather(const void* x, const int32_t* slot_row, void* out, int bf16, int64_t T, int64_t top_k,
                             int64_t H, hipStream_t s) {
  const int64_t span = kWave * (bf16 ? 8 : 4), pieces = (H + span - 1) / span;
  const dim3 grid = blocks_for(T * pieces, 4), block(256);
  if (bf16) return launch(gather_kernel<1>, grid, block, 0, s, x, slot_row, out, T, int(top_k), H, pieces);
  return launch(gather_kernel<0>, grid, block, 0, s, x, slot_row, out, T, int(top_k), H, pieces);
}

hipError_t launch_moe_combine(const void* rows, int bf16, const int32_t* slot_row, const float* weights, void* out,
                              int out_bf16, int64_t T, int64_t top_k, int64_t H, hipStream_t s) {
  const int64_t span = kWave * (bf16 ? 8 : 4), pieces = (H + span - 1) / span;
  const dim3 grid = blocks_for(T * pieces, 4), block(256);
  auto go = [&](auto kernel) {
    return launch(kernel, grid, block, 0, s, rows, slot_row, weights, out, T, int(top_k), H, pieces);
  };
  if (bf16) return out_bf16 ? go(combine_kernel<1, 1>) : go(combine_kernel<1, 0>);
  return out_bf16 ? go(combine_kernel<0, 1>) : go(combine_kernel<0, 0>);
}

hipError_t launch_moe_combine_backward(const void* dy, const void* rows, int bf16, const int32_t* slot_row,
                                       const float* weights, void* drows, float* dweights, int64_t T, int64_t top_k,
                                       int64_t H, hipStream_t s) {
  const int64_t S = T * top_k;
  const dim3 grid = blocks_for(S, 4), block(256);
  if (bf16)
    return launch(combine_backward_kernel<1>, grid, block, 0, s, dy, rows, slot_row, weights, drows, dweights, S,
                  int(top_k), H);
  return launch(combine_backward_kernel<0>, grid, block, 0, s, dy, rows, slot_row, weights, drows, dweights, S,
                int(top_k), H);
}

hipError_t launch_swiglu(const void* x, const void* dy, void* out, int bf16, int64_t M, int64_t F, hipStream_t s) {
  const int64_t per_row = (F + (bf16 ? 7 : 3)) / (bf16 ? 8 : 4);
  const dim3 grid = blocks_for(M * per_row, 256), block(256);
  auto go = [&](auto kernel) { return launch(kernel, grid, block, 0, s, x, dy, out, M, F, per_row); };
  if (dy) return bf16 ? go(swiglu_kernel<1, true>) : go(swiglu_kernel<0, true>);
  return bf16 ? go(swiglu_kernel<1, false>) : go(swiglu_kernel<0, false>);
}

}  // namespace qlinear
