// The norm behind a block with its gate and residual scale, fused with the norm in front of
// the next block, and the gradients of both:
//   p  = o * w_o / sqrt(mean o^2 + eps)            (or p = o without a norm behind the block)
//   r' = a r + gate * p,                           stored in r's type
//   y  = r' * w / sqrt(mean r'^2 + eps),           from r' as stored
// Backward, with D the whole gradient of r', v = 1 / sqrt(mean r'^2 + eps), n = r' v and
// v_o, n_o alike for o:
//   D    = dr' + v (dy w - n mean(dy w n)),        dr = a D,     dw = sum_t dy n
//   b    = D gate w_o,  do = v_o (b - n_o mean(b n_o)),          dw_o = sum_t D gate n_o
//   dgate = sum over the gate's rows of D p        (without a norm: do = D gate)
// All of it bound by HBM: every row is read once into registers, both sums over it are
// taken there, and it is written once.
//
// A row belongs to TPR threads (64 .. 512, whole waves), V values each in pieces of 8
// (V / 8 16-byte loads of bfloat16, twice as many of float32), so a wave's load covers
// 1 KiB of the row.  Rows of up to 64 * 8 values are one wave's and take no barrier.
#include <type_traits>

#include "device.hpp"
#include "elem.hpp"
#include "launch.hpp"

namespace qlinear {

namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 8;  // values of a thread that lie together

// N sums over the TPR threads of a row; every thread gets the results.  `part`: LDS of its own for two calls in
// a row, so that a call's one barrier also lies between the reads of one and the writes of the next but one.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if constexpr (TPR > kWave) {
    constexpr int W = TPR / kWave;
    const int wid = threadIdx.x / kWave;
    if (threadIdx.x % kWave == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) part[wid][n] = v[n];
    __syncthreads();
    const int first = wid / W * W;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) v[n] += part[first + i][n];
    }
  }
}

struct NormArgs {
  const void *res, *block, *w, *wo, *gate;  // block, wo, gate: null where there is none
  void *y, *res_out;
  int64_t T, H, per;  // per: rows of a gate
  float scale, eps;
};

// R, IO, P: element types of the residual, of block output and y, of the parameters.  TAIL: H % 8 != 0.
// NT: results past the caches.  Bound by HBM: 16384 x 4096, float32
// residual, 146 us, 5.5 TB/s; 16384 x 2048 in bfloat16 46 to 48 us, 5.7 (here and below: the kernel alone, no operand in a
// cache, if nothing else is said); a 1 GiB copy reaches 5.0.  8 x 4096: 4.7 us, the
// launch and one way to memory and back.
template <int R, int IO, int P, int TPR, int V, bool TAIL, bool NT>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void norm_kernel(NormArgs a) {
  constexpr int THREADS = TPR > kThreads ? TPR : kThreads, ROWS = THREADS / TPR, C = V / kPiece;
  __shared__ float part[4][THREADS / kWave][1];
  const int lane = threadIdx.x % TPR, mine = threadIdx.x / TPR;
  const float inv_h = 1.f / float(a.H);
  int turn = 0;
  // Whole blocks of rows, so that every thread meets the barriers; rows past the end repeat the last.
  for (int64_t t0 = int64_t(blockIdx.x) * ROWS; t0 < a.T; t0 += int64_t(gridDim.x) * ROWS, turn ^= 2) {
    const bool live = t0 + mine < a.T;
    const int64_t t = live ? t0 + mine : a.T - 1, at = t * a.H;
    const int64_t grow = a.gate ? t / a.per * a.H : 0;
    Eight<R> r8[C];
    Eight<IO> o8[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t i = int64_t(c * TPR + lane) * kPiece;
      r8[c].template load<TAIL>(a.res, at + i, a.H - i);
      if (a.block) o8[c].template load<TAIL>(a.block, at + i, a.H - i);
    }
    auto parameter = [&](const void* p, int64_t from, int64_t i, float (&f)[8]) {
      Eight<P> v;
      v.template load<TAIL>(p, from + i, a.H - i);
      v.get(f);
    };
    float r[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) r8[c].get(r[c]);
    if (a.block) {
      float o[C][8];
      float inv = 1.f;
#pragma unroll
      for (int c = 0; c < C; ++c) o8[c].get(o[c]);
      if (a.wo) {
        float s[1] = {0.f};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(o[c][e], o[c][e], s[0]);
        row_sums<TPR>(s, part[turn]);
        inv = rsqrtf(s[0] * inv_h + a.eps);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t i = int64_t(c * TPR + lane) * kPiece;
        if (a.wo) {
          float w[8];
          parameter(a.wo, 0, i, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[c][e] = o[c][e] * inv * w[e];
        }
        if (a.gate) {
          float g[8];
          parameter(a.gate, grow, i, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[c][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] = fmaf(a.scale, r[c][e], o[c][e]);
        r8[c].put(r[c]);
        r8[c].get(r[c]);  // as it is stored
        if (live) r8[c].template store<TAIL, NT>(a.res_out, at + i, a.H - i);
      }
    }
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = fmaf(r[c][e], r[c][e], s[0]);
    row_sums<TPR>(s, part[turn + 1]);
    const float inv = rsqrtf(s[0] * inv_h + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t i = int64_t(c * TPR + lane) * kPiece;
      float w[8];
      parameter(a.w, 0, i, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = r[c][e] * inv * w[e];
      Eight<IO> y;
      y.put(w);
      if (live) y.template store<TAIL, NT>(a.y, at + i, a.H - i);
    }
  }
}

struct NormGradArgs {
  const void *dy, *dres_in, *res, *w, *block, *wo, *gate;  // dres_in, block, wo, gate: null where there is none
  void *dres, *dblock, *dgate;
  float *part_w, *part_wo, *part_gate;  // [workers, H], [workers, H], [workers, 2, H]
  int64_t T, H, per, rows;  // rows of a worker
  float scale, eps;
};

// A worker is the TPR threads of a row.  It takes `rows` rows one after the other and keeps the columns'
// sums in registers; the workers' sums are added afterwards in their order.  Gates of no more rows than a
// worker's lie whole in one (rows is a multiple of theirs) and are finished by it; of others it leaves parts:
// [0] of the gate that its range begins in the middle of, [1] of the one that begins in its range.
// With V = 8 the parameters stay in registers and the next row is on its way while one is worked on; wider
// rows have no registers for that.  Both means come from sums over the row as it was read, so that a row meets
// one barrier.  Bound by HBM: 8192 x 2048 in bfloat16 with the residual's gradient coming in 45 us, 4.4 TB/s, without
// 37, 4.5;
// 16384 x 4096 159 us, 4.2; results past the caches changed neither.  4096 rows of H = 5120 79 us, 2.7 TB/s (a thread's
// second eight values lie past the row's end for three threads of four), of 8192 95, 3.5, of 16384 861, 0.8: 32 values a
// thread take 540 to 730 bytes of scratch a lane, 16 none or, with float32 parameters where H % 8 != 0, 8 to 16.  256 or 1024 blocks take 1.5 and 1.1 times as long
// at 8192 x 2048.
template <int R, int IO, int P, int TPR, int V, bool TAIL>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void norm_grad_kernel(NormGradArgs a) {
  constexpr int THREADS = TPR > kThreads ? TPR : kThreads, WORKERS = THREADS / TPR, C = V / kPiece;
  constexpr bool kAhead = V == 8;
  __shared__ float part[2][THREADS / kWave][6];
  const int lane = threadIdx.x % TPR;
  const float inv_h = 1.f / float(a.H);
  const int64_t worker = int64_t(blockIdx.x) * WORKERS + threadIdx.x / TPR;
  const int64_t begin = worker * a.rows, end = begin + a.rows < a.T ? begin + a.rows : a.T;
  const bool with_o = a.wo || a.gate;
  auto piece = [&](int c) { return int64_t(c * TPR + lane) * kPiece; };

  struct Row {
    Eight<R> r[C], dr[C];
    Eight<IO> dy[C], o[C];
  };
  auto row_of = [&](int64_t n) { return begin + n < a.T ? begin + n : a.T - 1; };
  auto load = [&](Row& row, int64_t t) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t i = piece(c), at = t * a.H + i;
      row.r[c].template load<TAIL>(a.res, at, a.H - i);
      row.dy[c].template load<TAIL>(a.dy, at, a.H - i);
      if (a.dres_in) row.dr[c].template load<TAIL>(a.dres_in, at, a.H - i);
      if (with_o) row.o[c].template load<TAIL>(a.block, at, a.H - i);
    }
  };
  auto parameter = [&](const void* p, int64_t at, int c, float (&f)[8]) {
    Eight<P> v;
    v.template load<TAIL>(p, at + piece(c), a.H - piece(c));
    v.get(f);
  };
  float w[C][8], wo[C][8], g[C][8];
  if (kAhead) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      parameter(a.w, 0, c, w[c]);
      if (a.wo) parameter(a.wo, 0, c, wo[c]);
    }
  }
  int64_t held = -1;  // the gate in g
  float sw[C][8], swo[C][8], sg[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) sw[c][e] = swo[c][e] = sg[c][e] = 0.f;
  Row cur, next;
  load(cur, row_of(0));
  for (int64_t n = 0; n < a.rows; ++n) {  // as many turns for every worker of the block: barriers
    const bool live = begin + n < end;
    const int64_t t = row_of(n), at = t * a.H;
    if (kAhead) load(next, row_of(n + 1 < a.rows ? n + 1 : n));
    const int64_t gate = a.gate ? t / a.per : 0;
    if (a.gate && (!kAhead || gate != held)) {
#pragma unroll
      for (int c = 0; c < C; ++c) parameter(a.gate, gate * a.H, c, g[c]);
      held = gate;
    }
    // All sums over the row at once: of r^2, dy w r, o^2, and with q = gate w_o o those of dr' q, dy w q, r q, of
    // which sum(b o) = sum(D q) is made.
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float r[8], dy[8];
      cur.r[c].get(r);
      cur.dy[c].get(dy);
      if (!kAhead) parameter(a.w, 0, c, w[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dy[e] *= w[c][e];
        s[0] = fmaf(r[e], r[e], s[0]);
        s[1] = fmaf(dy[e], r[e], s[1]);
      }
      if (a.wo) {
        float o[8], in[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        cur.o[c].get(o);
        if (a.dres_in) cur.dr[c].get(in);
        if (!kAhead) parameter(a.wo, 0, c, wo[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[2] = fmaf(o[e], o[e], s[2]);
          const float q = a.gate ? o[e] * wo[c][e] * g[c][e] : o[e] * wo[c][e];
          s[3] = fmaf(in[e], q, s[3]);
          s[4] = fmaf(dy[e], q, s[4]);
          s[5] = fmaf(r[e], q, s[5]);
        }
      }
    }
    row_sums<TPR>(s, part[n & 1]);
    const float inv = rsqrtf(s[0] * inv_h + a.eps), mean = s[1] * inv * inv_h;
    const float inv_o = a.wo ? rsqrtf(s[2] * inv_h + a.eps) : 1.f;
    const float mean_o = (s[3] + inv * (s[4] - inv * mean * s[5])) * inv_o * inv_h;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float r[8], d[8], out[8], in[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      cur.r[c].get(r);
      cur.dy[c].get(d);
      if (a.dres_in) cur.dr[c].get(in);
      if (!kAhead) parameter(a.w, 0, c, w[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r[e] *= inv;
        if (live) sw[c][e] = fmaf(d[e], r[e], sw[c][e]);
        d[e] = fmaf(inv, fmaf(-r[e], mean, d[e] * w[c][e]), in[e]);
        out[e] = a.scale * d[e];
      }
      Eight<R> dres;
      dres.put(out);
      if (live) dres.template store<TAIL>(a.dres, at + piece(c), a.H - piece(c));
      if (!a.block) continue;
      float o[8];
      if (with_o) cur.o[c].get(o);
      if (!kAhead && a.wo) parameter(a.wo, 0, c, wo[c]);
      if (!kAhead && a.gate) parameter(a.gate, gate * a.H, c, g[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (a.wo) o[e] *= inv_o;
        if (a.gate) {
          if (live) sg[c][e] = fmaf(d[e], a.wo ? o[e] * wo[c][e] : o[e], sg[c][e]);
          d[e] *= g[c][e];
        }
        if (a.wo) {
          if (live) swo[c][e] = fmaf(d[e], o[e], swo[c][e]);
          d[e] = inv_o * fmaf(-o[e], mean_o, d[e] * wo[c][e]);
        }
      }
      Eight<IO> dblock;
      dblock.put(d);
      if (live) dblock.template store<TAIL>(a.dblock, at + piece(c), a.H - piece(c));
    }
    if (a.block) {
      // The gate's last row of this range: its sum leaves.
      if (a.gate && live && (t + 1 == end || (t + 1) % a.per == 0)) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (a.per <= a.rows) {
            Eight<P> out;
            out.put(sg[c]);
            out.template store<TAIL>(a.dgate, gate * a.H + piece(c), a.H - piece(c));
          } else {
            Eight<0> out;
            out.put(sg[c]);
            out.template store<TAIL>(a.part_gate, (2 * worker + (gate * a.per >= begin)) * a.H + piece(c), a.H - piece(c));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) sg[c][e] = 0.f;
        }
      }
    }
    if (kAhead) cur = next;
    else if (n + 1 < a.rows) load(cur, row_of(n + 1));
  }
  if (begin >= a.T) return;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    Eight<0> out;
    out.put(sw[c]);
    out.template store<TAIL>(a.part_w, worker * a.H + piece(c), a.H - piece(c));
    if (a.wo) {
      out.put(swo[c]);
      out.template store<TAIL>(a.part_wo, worker * a.H + piece(c), a.H - piece(c));
    }
  }
}

// Adds the workers' sums in their order: 64 columns a block, each of its 16 waves every sixteenth worker.
// blockIdx.y: 0 dw, 1 dw_o, from 2 on the gates, where they have more rows than a worker.
struct NormJoinArgs {
  const float *part_w, *part_wo, *part_gate;
  void *dw, *dwo, *dgate;
  int64_t T, H, per, rows, workers;
  int p_bf16;
};
constexpr int kJoinWaves = 16;

__global__ __launch_bounds__(kJoinWaves* kWave) void norm_join_kernel(NormJoinArgs a) {
  __shared__ float part[kJoinWaves][kWave];
  const int lane = threadIdx.x % kWave, wid = threadIdx.x / kWave;
  const int64_t col = int64_t(blockIdx.x) * kWave + lane;
  const bool live = col < a.H;
  const float* src = blockIdx.y ? a.part_wo : a.part_w;  // term n: the first at first_at, then next_at + (n - 1) stride
  void* out = blockIdx.y ? a.dwo : a.dw;
  int64_t count = a.workers, stride = a.H, first_at = 0, next_at = a.H, at = 0;
  if (blockIdx.y >= 2) {
    const int64_t g = blockIdx.y - 2, w0 = g * a.per / a.rows, w1 = ((g + 1) * a.per - 1) / a.rows;  // its workers
    src = a.part_gate;
    out = a.dgate;
    stride = 2 * a.H;
    first_at = (2 * w0 + 1) * a.H;  // the gate begins in the first worker's range, and the others begin in it
    next_at = 2 * (w0 + 1) * a.H;
    count = w1 - w0 + 1;
    at = g * a.H;
  }
  if (!out) return;
  float s = 0.f;
  if (live) {
    int64_t n = wid;
    for (; n + 7 * kJoinWaves < count; n += 8 * kJoinWaves) {  // eight loads on their way at once
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t m = n + e * kJoinWaves;
        v[e] = src[(m ? next_at + (m - 1) * stride : first_at) + col];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e];
    }
    for (; n < count; n += kJoinWaves) s += src[(n ? next_at + (n - 1) * stride : first_at) + col];
  }
  part[wid][lane] = s;
  __syncthreads();
  if (wid || !live) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinWaves; ++i) s += part[i][lane];
  if (a.p_bf16) reinterpret_cast<uint16_t*>(out)[at + col] = Elem<1>::put(s);
  else reinterpret_cast<float*>(out)[at + col] = s;
}

template <int TPR_, int V_> struct RowShape {
  static constexpr int kTpr = TPR_, kV = V_;
  static constexpr int kRows = TPR_ > kThreads ? 1 : kThreads / TPR_;
};
template <typename F>
auto by_width(int64_t H, F&& go) {
  if (H <= 512) return go(RowShape<64, 8>{});
  if (H <= 1024) return go(RowShape<128, 8>{});
  if (H <= 2048) return go(RowShape<256, 8>{});
  if (H <= 4096) return go(RowShape<512, 8>{});
  if (H <= 8192) return go(RowShape<512, 16>{});
  return go(RowShape<512, 32>{});
}

template <int R_, int IO_, int P_, bool TAIL_> struct RowTypes {
  static constexpr int R = R_, IO = IO_, P = P_;
  static constexpr bool TAIL = TAIL_;
};
template <typename F>
hipError_t by_types(int r, int io, int p, bool tail, F&& go) {
  auto with = [&](auto tail_) {
    constexpr bool TAIL = decltype(tail_)::value;
    if (r) return p ? go(RowTypes<1, 1, 1, TAIL>{}) : go(RowTypes<1, 1, 0, TAIL>{});
    if (io) return p ? go(RowTypes<0, 1, 1, TAIL>{}) : go(RowTypes<0, 1, 0, TAIL>{});
    return p ? go(RowTypes<0, 0, 1, TAIL>{}) : go(RowTypes<0, 0, 0, TAIL>{});
  };
  return tail ? with(std::true_type{}) : with(std::false_type{});
}

// Calls that move more leave their results past the caches, as calls among others, which find part of their operands
// there: 16384 x 2048 in bfloat16 (268 MB) 43 us, 55 through them; 4096 x 4096 (134 MB) 23.5 us either way, and the next
// operator finds the rows.
constexpr int64_t kNtBytes = int64_t(160) << 20;

// Workers of the backward pass: two blocks per CU of a 256 CU card, a row each at least.  Not the current device's CUs:
// the workspace's size is a function of the sizes alone, asked for before there is a device.  Where a gate's
// rows are fewer than a worker's, these are a multiple of them.
constexpr int64_t kGradBlocks = 512;
void grad_split(int64_t T, int64_t per, int rows_per_block, int64_t* rows, int64_t* workers) {
  const int64_t most = kGradBlocks * rows_per_block;
  *rows = (T + most - 1) / most;
  if (per < *rows) *rows = (*rows + per - 1) / per * per;
  *workers = (T + *rows - 1) / *rows;
}

}  // namespace

hipError_t launch_block_norm(const void* res, int r_bf16, const void* w, int p_bf16, const void* block, int io_bf16,
                             const void* wo, const void* gate, int64_t gates, void* res_out, void* y, int64_t T,
                             int64_t H, float scale, float eps, hipStream_t s) {
  const NormArgs a{res, block, w, wo, gate, y, res_out, T, H, gates ? T / gates : T, scale, eps};
  return by_types(r_bf16, io_bf16, p_bf16, H % kPiece != 0, [&](auto ty) {
    using Ty = decltype(ty);
    return by_width(H, [&](auto shape) {
      using S = decltype(shape);
      const int64_t blocks = (T + S::kRows - 1) / S::kRows;
      auto go = [&](auto kernel) {
        return launch(kernel, dim3(unsigned(blocks < 65536 ? blocks : 65536)),
                      dim3(S::kTpr > kThreads ? S::kTpr : kThreads), 0, s, a);
      };
      const int64_t bytes = T * H * ((block ? 2 : 1) * (r_bf16 ? 2 : 4) + (block ? 2 : 1) * (io_bf16 ? 2 : 4));
      return bytes > kNtBytes ? go(norm_kernel<Ty::R, Ty::IO, Ty::P, S::kTpr, S::kV, Ty::TAIL, true>)
                              : go(norm_kernel<Ty::R, Ty::IO, Ty::P, S::kTpr, S::kV, Ty::TAIL, false>);
    });
  });
}

size_t block_norm_grad_ws_bytes(int64_t T, int64_t H, bool post, bool gate) {
  if (T <= 0) return 0;
  return by_width(H, [&](auto shape) {
    int64_t rows, workers;
    grad_split(T, T, decltype(shape)::kRows, &rows, &workers);  // the most workers that any gate leaves
    return size_t(workers) * size_t(H) * 4 * (1 + (post ? 1 : 0) + (gate ? 2 : 0));
  });
}

hipError_t launch_block_norm_grad(const void* dy, int io_bf16, const void* dres_in, const void* res, int r_bf16,
                                  const void* w, int p_bf16, const void* block, const void* wo, const void* gate,
                                  int64_t gates, void* dres, void* dblock, void* dw, void* dwo, void* dgate, int64_t T,
                                  int64_t H, float scale, float eps, float* ws, hipStream_t s) {
  int64_t rows = 0, workers = 0;
  NormGradArgs a{dy, dres_in, res, w, block, wo, gate, dres, dblock, dgate, ws, nullptr, nullptr, T, H,
                 gates ? T / gates : T, 0, scale, eps};
  const hipError_t e = by_types(r_bf16, io_bf16, p_bf16, H % kPiece != 0, [&](auto ty) {
    using Ty = decltype(ty);
    return by_width(H, [&](auto shape) {
      using S = decltype(shape);
      grad_split(T, a.per, S::kRows, &rows, &workers);
      a.rows = rows;
      a.part_wo = a.part_w + workers * H;
      a.part_gate = a.part_wo + (wo ? workers * H : 0);
      return launch(norm_grad_kernel<Ty::R, Ty::IO, Ty::P, S::kTpr, S::kV, Ty::TAIL>,
                    dim3(unsigned((workers + S::kRows - 1) / S::kRows)),
                    dim3(S::kTpr > kThreads ? S::kTpr : kThreads), 0, s, a);
    });
  });
  if (e != hipSuccess) return e;
  const NormJoinArgs j{a.part_w, a.part_wo, a.part_gate, dw, wo ? dwo : nullptr, dgate, T, H, a.per, rows, workers, p_bf16};
  const unsigned joins = gate && a.per > rows ? unsigned(2 + gates) : wo ? 2u : 1u;  // such gates are fewer than the workers
  return launch(norm_join_kernel, dim3(unsigned((H + kWave - 1) / kWave), joins), dim3(kJoinWaves * kWave), 0, s, j);
}

}  // namespace qlinear
