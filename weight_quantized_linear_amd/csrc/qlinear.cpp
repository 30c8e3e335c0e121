// The C ABI of libqlinear: argument validation, the gfx950 device check and
// the choice of kernel.  Declarations and the contract of every call are in
// include/qlinear.h.
#include "qlinear.h"

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>
#include <limits>
#include <mutex>

#include "launch.hpp"
#include "gated_out.hpp"

namespace {

using namespace qlinear;

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  std::atomic<int> state{0};  // 0 unknown, 1 gfx950, 2 other arch, 3 query failed
  int num_cus = 0;
};
DeviceInfo g_devices[kMaxDevices];
std::mutex g_device_mutex;

// Status of the current device, cached per device index; fills num_cus.
int current_device(int* num_cus) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return QLINEAR_ERR_DEVICE;
  DeviceInfo& d = g_devices[dev];
  int st = d.state.load(std::memory_order_acquire);
  if (st == 0) {
    std::lock_guard<std::mutex> lock(g_device_mutex);
    st = d.state.load(std::memory_order_relaxed);
    if (st == 0) {
      hipDeviceProp_t prop;
      if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
        st = 3;
      } else {
        st = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        d.num_cus = prop.multiProcessorCount;
      }
      d.state.store(st, std::memory_order_release);
    }
  }
  if (st == 3) return QLINEAR_ERR_DEVICE;
  if (st == 2) return QLINEAR_ERR_UNSUPPORTED;
  *num_cus = d.num_cus > 0 ? d.num_cus : 256;
  return QLINEAR_OK;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// n1 * n2 (* n3) must stay addressable; all factors are already > 0.
bool fits(int64_t a, int64_t b, int64_t c = 1) {
  const int64_t lim = std::numeric_limits<int64_t>::max() / 8;
  if (a > lim / b) return false;
  const int64_t ab = a * b;
  return ab <= lim / c;
}

int float_out_ok(int out_dtype) { return out_dtype == QLINEAR_F32 || out_dtype == QLINEAR_BF16; }

size_t out_size(int out_dtype) { return out_dtype == QLINEAR_BF16 ? 2 : 4; }

int finish(hipError_t e) { return e == hipSuccess ? QLINEAR_OK : QLINEAR_ERR_LAUNCH; }

// Validates a caller's epilogue for an [M, N] output and converts it (null:
// no epilogue).  The residual may be the output itself (same type, ld = N).
int to_epilogue(const qlinear_epilogue* e, int64_t M, int64_t N, Epilogue* out) {
  *out = Epilogue{};
  if (!e) return QLINEAR_OK;
  if (e->activation < QLINEAR_ACT_NONE || e->activation > QLINEAR_ACT_GELU_TANH) return QLINEAR_ERR_INVALID_ARG;
  if ((e->row_scale && !aligned(e->row_scale, 4)) || (e->col_scale && !aligned(e->col_scale, 4)) ||
      (e->bias && !aligned(e->bias, 2)))
    return QLINEAR_ERR_INVALID_ARG;
  if (e->residual) {
    if (e->residual_dtype != QLINEAR_F32 && e->residual_dtype != QLINEAR_BF16) return QLINEAR_ERR_INVALID_ARG;
    if (e->residual_ld < N || !aligned(e->residual, out_size(e->residual_dtype)) || !fits(M, e->residual_ld))
      return QLINEAR_ERR_INVALID_ARG;
  }
  out->row_scale = e->row_scale;
  out->col_scale = e->col_scale;
  out->bias = static_cast<const uint16_t*>(e->bias);
  out->residual = e->residual;
  out->ld = e->residual ? e->residual_ld : 0;
  out->act = e->activation;
  out->res_bf16 = e->residual_dtype == QLINEAR_BF16;
  out->on = e->row_scale || e->col_scale || e->bias || e->residual || e->activation != QLINEAR_ACT_NONE;
  return QLINEAR_OK;
}

// A caller's split-K workspace: NULL (with 0 bytes) for none, else at least
// 16-byte aligned device memory of workspace_bytes >= 0 bytes.
int check_workspace(const void* ws, int64_t ws_bytes) {
  if (ws_bytes < 0 || (!ws && ws_bytes != 0) || (ws && !aligned(ws, 16))) return QLINEAR_ERR_INVALID_ARG;
  return QLINEAR_OK;
}

// Sizes and choices of the feed-forward block's operators.
constexpr int64_t kMaxLoraGroups = 4096, kMaxAdapters = 4096, kMaxRank = 256, kMaxLoraWidth = int64_t(1) << 20;
constexpr int64_t kMaxNormWidth = 16384;

bool gated_act_ok(int act) { return act >= QLINEAR_ACT_RELU && act <= QLINEAR_ACT_GELU_TANH; }
bool gated_sizes_ok(int64_t M, int64_t F) { return F > 0 && fits(M > 0 ? M : 1, F, 2); }

bool linear_grad_ok(const void* dout, const void* other, const void* grad, int dtype, int64_t M, int64_t N, int64_t K) {
  return dout && other && grad && M >= 0 && N > 0 && K > 0 && fits(M ? M : 1, N) && fits(M ? M : 1, K) && fits(N, K) &&
         float_out_ok(dtype) && aligned(dout, 2) && aligned(other, 2) && aligned(grad, out_size(dtype));
}

bool lora_sizes_ok(int64_t G, int64_t L, int64_t T, int64_t N, int64_t K, int64_t R) {
  return G > 0 && G <= kMaxLoraGroups && L > 0 && L <= kMaxAdapters && T >= 0 && T <= (int64_t(1) << 30) && N > 0 &&
         N <= kMaxLoraWidth && K > 0 && K <= kMaxLoraWidth && R > 0 && R <= kMaxRank;
}

bool norm_ok(int res_dtype, int dtype, int param_dtype, const void* block, const void* block_weight, const void* gate,
             int64_t gates, int64_t T, int64_t H, float eps) {
  if (!float_out_ok(res_dtype) || !float_out_ok(dtype) || !float_out_ok(param_dtype)) return false;
  if (res_dtype == QLINEAR_BF16 && dtype == QLINEAR_F32) return false;
  if (T < 0 || H <= 0 || H > kMaxNormWidth || !fits(T ? T : 1, H) || !(eps > 0.f)) return false;
  if (!block && (block_weight || gate)) return false;
  return gate ? gates > 0 && T % gates == 0 && fits(gates, H) : gates == 0;
}

// The FP8 kernel family that a call takes: `path` if forced, else the
// automatic choice, which depends on the shape, the operands' alignment and
// whether a workspace of at least `ws_need` bytes is given (and on nothing
// else, so that a call is reproducible from its arguments).
int fp8_choose(int path, int64_t M, int64_t N, int64_t K, bool wide, bool splitk_ok) {
  if (path != QLINEAR_PATH_AUTO) return path;
  // Measured on the decode shapes: the vector-ALU GEMV wins for M <= 2
  // below 65536 output features and for M <= 4 on small weights; the
  // matrix-core skinny kernels win above that (for 3 <= M <= 4 from 8192
  // output features or a K of 8192 when the activation-in-LDS kernel
  // applies, and for M = 4 from 4096 output features where the streaming
  // kernel takes the shape) and for 5 <= M <= 16; beyond 16 rows the
  // LDS-tiled GEMM.
  const bool big = N >= 65536 || (M >= 3 && (N >= 8192 || K >= 8192) && fp8_skinny_xlds_supported(M, N, K)) ||
                   (M == 4 && fp8_skinny_stream_wins(M, N, K) && (K == 1024 || K == 2048 || K == 3072 || K == 4096));
  // Split-K needs the caller's workspace.  Where K is made of 2048-value
  // slices (K >= 8192) and there are fewer than 65536 output features, its
  // streaming form wins from M = 3 (N = 4096, K = 14336: M = 4 14.8 against
  // 17.2 us for the 4x4x4 skinny kernel, M = 8 15.4 against 18.5; N = K =
  // 14336, M = 8: 40.1 against 51.7) and at M = 2 from 8192 output features
  // (N = K = 14336: 37.2 against 47.2 us for the GEMV; at N = 4096 the GEMV
  // keeps 12.6 against 14.3); for 9 <= M <= 16 the split-K skinny kernel also
  // wins at other long K (M = 16, N = 4096, K = 14336: 19.2 against 23.1 us).
  const bool split_long = splitk_ok && wide && K >= 8192 && N < 65536;
  if (M == 1) return QLINEAR_PATH_GEMV;
  if (M <= 4) {
    if ((M >= 3 || N >= 8192) && split_long && K % 2048 == 0) return QLINEAR_PATH_SPLITK;
    return (wide && big) ? QLINEAR_PATH_SKINNY : QLINEAR_PATH_GEMV;
  }
  if (M <= 16 && wide)
    return (split_long && (K % 2048 == 0 || (M > 8 && K % 64 == 0))) ? QLINEAR_PATH_SPLITK : QLINEAR_PATH_SKINNY;
  return QLINEAR_PATH_TILED;
}

int nvfp4_choose(int path, int64_t M) {
  if (path != QLINEAR_PATH_AUTO) return path;
  return M <= 4 ? QLINEAR_PATH_GEMV : QLINEAR_PATH_TILED;
}

int bf16_choose(int path, int64_t M, bool wide) {
  if (path != QLINEAR_PATH_AUTO) return path;
  if (M <= 4) return QLINEAR_PATH_GEMV;
  if (M <= 16 && wide) return QLINEAR_PATH_SKINNY;
  return QLINEAR_PATH_TILED;
}

}  // namespace

namespace qlinear {

int fp8_gemm_impl(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                  float alpha, int path, void* ws, int64_t ws_bytes, void* stream,
                  const qlinear_epilogue* epilogue = nullptr) {
  if (!w || !x || !out) return QLINEAR_ERR_INVALID_ARG;
  if (M <= 0 || N <= 0 || K <= 0 || !fits(N, K) || !fits(M, K) || !fits(M, N))
    return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype)) return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(out, out_size(out_dtype))) return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(ws, ws_bytes)) return st;
  const bool wide = K % 16 == 0 && aligned(w, 16) && aligned(x, 16);
  switch (path) {
    case QLINEAR_PATH_AUTO:
    case QLINEAR_PATH_TILED:
      break;
    case QLINEAR_PATH_GEMV:
      if (M > 4) return QLINEAR_ERR_INVALID_ARG;
      break;
    case QLINEAR_PATH_SKINNY:
      if (M > 16 || !wide) return QLINEAR_ERR_INVALID_ARG;
      break;
    case QLINEAR_PATH_SPLITK:
      if (M > 16 || !wide || K % 64 != 0) return QLINEAR_ERR_INVALID_ARG;
      break;
    default:
      return QLINEAR_ERR_INVALID_ARG;
  }
  Epilogue epi;
  if (int st = to_epilogue(epilogue, M, N, &epi)) return st;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  const size_t splitk_need = fp8_skinny_splitk_ws_bytes(M, N, K, num_cus);
  const bool splitk_ok = ws && splitk_need > 0 && splitk_need <= size_t(ws_bytes);
  path = fp8_choose(path, M, N, K, wide, splitk_ok);
  // Forced split-K with fewer than two K slices or planes beyond the workspace.
  if (path == QLINEAR_PATH_SPLITK && !splitk_ok) return QLINEAR_ERR_UNSUPPORTED;
  auto s = static_cast<hipStream_t>(stream);
  auto* wp = static_cast<const uint8_t*>(w);
  auto* xp = static_cast<const uint16_t*>(x);
  auto* wsp = static_cast<float*>(ws);
  const int bf16 = out_dtype == QLINEAR_BF16;
  if (path == QLINEAR_PATH_SPLITK)
    return finish(launch_fp8_skinny_splitk(wp, xp, out, bf16, M, N, K, alpha, num_cus, wsp, size_t(ws_bytes), s, epi));
  if (path == QLINEAR_PATH_GEMV)
    return finish(launch_fp8_gemv(wp, xp, out, bf16, M, N, K, alpha, num_cus, s, epi));
  if (path == QLINEAR_PATH_SKINNY)
    return finish(launch_fp8_skinny(wp, xp, out, bf16, M, N, K, alpha, num_cus, s, epi));
  return finish(launch_fp8_tiled(wp, xp, out, bf16, M, N, K, alpha, num_cus, wsp, size_t(ws_bytes), s, epi));
}

int fp8_gemm_ws_need(int path, int64_t M, int64_t N, int64_t K, int num_cus, int64_t* bytes) {
  *bytes = 0;
  if (M <= 0 || N <= 0 || K <= 0 || !fits(N, K) || !fits(M, K) || !fits(M, N)) return QLINEAR_ERR_INVALID_ARG;
  const size_t splitk = fp8_skinny_splitk_ws_bytes(M, N, K, num_cus);
  path = fp8_choose(path, M, N, K, K % 16 == 0, splitk > 0);
  if (path == QLINEAR_PATH_SPLITK) *bytes = int64_t(splitk);
  else if (path == QLINEAR_PATH_TILED && K % 64 == 0) *bytes = int64_t(fp8_gemm_lds_ws_bytes(M, N, K, num_cus));
  return QLINEAR_OK;
}

}  // namespace qlinear

namespace {

int nvfp4_gemm_impl(const void* wp, const void* wsc, const void* x, void* out, int out_dtype, int64_t M, int64_t N,
                    int64_t K, float alpha, int path, void* ws, int64_t ws_bytes, void* stream,
                    const qlinear_epilogue* epilogue = nullptr) {
  if (!wp || !wsc || !x || !out) return QLINEAR_ERR_INVALID_ARG;
  if (M <= 0 || N <= 0 || K <= 0 || K % 16 != 0 || !fits(N, K) || !fits(M, K) || !fits(M, N))
    return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype) || !aligned(x, 2) || !aligned(out, out_size(out_dtype)))
    return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(ws, ws_bytes)) return st;
  path = nvfp4_choose(path, M);
  if (path == QLINEAR_PATH_GEMV) {
    if (M > 4) return QLINEAR_ERR_INVALID_ARG;
  } else if (path != QLINEAR_PATH_TILED) {
    return QLINEAR_ERR_INVALID_ARG;
  }
  Epilogue epi;
  if (int st = to_epilogue(epilogue, M, N, &epi)) return st;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  auto s = static_cast<hipStream_t>(stream);
  auto* p = static_cast<const uint8_t*>(wp);
  auto* sc = static_cast<const uint8_t*>(wsc);
  auto* xp = static_cast<const uint16_t*>(x);
  const int bf16 = out_dtype == QLINEAR_BF16;
  if (path == QLINEAR_PATH_GEMV)
    return finish(launch_nvfp4_gemv(p, sc, xp, out, bf16, M, N, K, alpha, num_cus, s, epi));
  return finish(launch_nvfp4_tiled(p, sc, xp, out, bf16, M, N, K, alpha, num_cus, static_cast<float*>(ws),
                                   size_t(ws_bytes), s, epi));
}

int bf16_gemm_impl(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                   float alpha, int path, void* ws, int64_t ws_bytes, void* stream,
                   const qlinear_epilogue* epilogue = nullptr) {
  if (!w || !x || !out) return QLINEAR_ERR_INVALID_ARG;
  if (M <= 0 || N <= 0 || K <= 0 || !fits(N, K) || !fits(M, K) || !fits(M, N))
    return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype)) return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(w, 2) || !aligned(x, 2) || !aligned(out, out_size(out_dtype))) return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(ws, ws_bytes)) return st;
  const bool wide = bf16_wide(w, x, K);
  path = bf16_choose(path, M, wide);
  switch (path) {
    case QLINEAR_PATH_GEMV:
      if (M > 4) return QLINEAR_ERR_INVALID_ARG;
      break;
    case QLINEAR_PATH_SKINNY:
      if (M > 16 || !wide) return QLINEAR_ERR_INVALID_ARG;
      break;
    case QLINEAR_PATH_TILED:
      break;
    default:
      return QLINEAR_ERR_INVALID_ARG;
  }
  Epilogue epi;
  if (int st = to_epilogue(epilogue, M, N, &epi)) return st;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  auto s = static_cast<hipStream_t>(stream);
  auto* wp = static_cast<const uint16_t*>(w);
  auto* xp = static_cast<const uint16_t*>(x);
  const int bf16 = out_dtype == QLINEAR_BF16;
  if (path == QLINEAR_PATH_GEMV)
    return finish(launch_bf16_gemv(wp, xp, out, bf16, M, N, K, alpha, num_cus, s, epi));
  if (path == QLINEAR_PATH_SKINNY)
    return finish(launch_bf16_skinny(wp, xp, out, bf16, M, N, K, alpha, num_cus, s, epi));
  return finish(launch_bf16_tiled(wp, xp, out, bf16, M, N, K, alpha, num_cus, static_cast<float*>(ws),
                                  size_t(ws_bytes), s, epi));
}

// int4 groups: a power of two >= 32, or one group per row.  The kernels take
// 32-bit offsets inside a tile of rows.
bool int4_group_ok(int64_t g, int64_t K) { return K < (int64_t(1) << 23) && (g >= K || (g >= 32 && (g & (g - 1)) == 0)); }

// Limits of the expert calls: the router keeps a token's logits in one wave's
// registers and its picks in 64 places of LDS; slots and rows are int32.
constexpr int64_t kMaxRouted = 1024, kMaxTopK = 64, kMaxSlots = std::numeric_limits<int32_t>::max();

bool permute_sizes_ok(int64_t T, int64_t top_k, int64_t H) {
  return T >= 0 && top_k >= 1 && top_k <= kMaxTopK && T <= kMaxSlots / top_k && H > 0 && fits(T ? T : 1, top_k, H);
}

bool route_sizes_ok(int64_t T, int64_t E, int64_t top_k) {
  return E >= 1 && E <= kMaxRouted && top_k <= E && permute_sizes_ok(T, top_k, E);
}

}  // namespace

extern "C" {

int qlinear_abi_version(void) { return QLINEAR_ABI_VERSION; }

const char* qlinear_status_string(int status) {
  switch (status) {
    case QLINEAR_OK: return "ok";
    case QLINEAR_ERR_INVALID_ARG: return "invalid argument";
    case QLINEAR_ERR_UNSUPPORTED: return "unsupported device or configuration";
    case QLINEAR_ERR_DEVICE: return "no usable HIP device";
    case QLINEAR_ERR_LAUNCH: return "kernel launch failed";
    case QLINEAR_ERR_SCRATCH_LIMIT: return "shape needs more split-K scratch than the library's fixed buffer";
    default: return "unknown status";
  }
}

int qlinear_fp8_gemv(const void* w, const void* x, void* out, int out_dtype, int64_t N, int64_t K,
                     float alpha, void* stream) {
  return fp8_gemm_impl(w, x, out, out_dtype, 1, N, K, alpha, QLINEAR_PATH_GEMV, nullptr, 0, stream);
}

int qlinear_fp8_gemm(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N,
                     int64_t K, float alpha, void* stream) {
  return fp8_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, QLINEAR_PATH_AUTO, nullptr, 0, stream);
}

int qlinear_fp8_gemm_path(const void* w, const void* x, void* out, int out_dtype, int64_t M,
                          int64_t N, int64_t K, float alpha, int path, void* stream) {
  return fp8_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, path, nullptr, 0, stream);
}

int qlinear_fp8_materialize(const void* w, void* out, int out_dtype, int64_t N, int64_t K,
                            void* stream) {
  if (!w || !out || N <= 0 || K <= 0 || !fits(N, K) || !float_out_ok(out_dtype))
    return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(out, out_size(out_dtype))) return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_fp8_materialize(static_cast<const uint8_t*>(w), out,
                                       out_dtype == QLINEAR_BF16, N * K,
                                       static_cast<hipStream_t>(stream)));
}

int qlinear_fp8_grouped_gemm(const void* w, const void* x, const uint32_t* a_offsets,
                             const int32_t* expert_ids, void* out, int out_dtype, int64_t num_groups,
                             int64_t max_tokens_per_group, int64_t num_experts, int64_t T, int64_t N,
                             int64_t K, void* stream) {
  return qlinear_fp8_grouped_gemm_scaled(w, x, a_offsets, expert_ids, nullptr, out, out_dtype, num_groups,
                                         max_tokens_per_group, num_experts, T, N, K, stream);
}

int qlinear_fp8_grouped_gemm_scaled(const void* w, const void* x, const uint32_t* a_offsets,
                                    const int32_t* expert_ids, const float* expert_scale, void* out, int out_dtype,
                                    int64_t num_groups, int64_t max_tokens_per_group, int64_t num_experts, int64_t T,
                                    int64_t N, int64_t K, void* stream) {
  if (!w || !x || !a_offsets || !expert_ids || !out) return QLINEAR_ERR_INVALID_ARG;
  if (expert_scale && !aligned(expert_scale, 4)) return QLINEAR_ERR_INVALID_ARG;
  if (num_groups <= 0 || num_groups > 65535 || max_tokens_per_group < 0 || num_experts <= 0 || T <= 0 ||
      N <= 0 || K <= 0)
    return QLINEAR_ERR_INVALID_ARG;
  if (!fits(num_experts, N, K) || !fits(T, K) || !fits(T, N)) return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype) || !aligned(x, 2) || !aligned(out, out_size(out_dtype)) ||
      !aligned(a_offsets, 4) || !aligned(expert_ids, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_fp8_grouped(static_cast<const uint8_t*>(w), static_cast<const uint16_t*>(x),
                                   a_offsets, expert_ids, out, out_dtype == QLINEAR_BF16, num_groups,
                                   max_tokens_per_group, num_experts, T, N, K, num_cus,
                                   static_cast<hipStream_t>(stream), expert_scale));
}

int qlinear_fp8_quantize_act(const void* x, void* q, float input_scale, int64_t M, int64_t K, void* stream) {
  if (!x || !q || M <= 0 || K <= 0 || !fits(M, K) || !aligned(x, 2)) return QLINEAR_ERR_INVALID_ARG;
  if (!(input_scale > 0.f) || !(input_scale <= std::numeric_limits<float>::max())) return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_fp8_quantize_act(static_cast<const uint16_t*>(x), static_cast<uint8_t*>(q), input_scale, M, K,
                                        num_cus, static_cast<hipStream_t>(stream)));
}

int qlinear_fp8_w8a8_gemm(const void* xq, const void* w, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                          float alpha, void* stream) {
  if (!xq || !w || !out || M <= 0 || N <= 0 || K <= 0 || !fits(M, K) || !fits(N, K) || !fits(M, N))
    return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype) || !aligned(out, out_size(out_dtype))) return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_fp8_w8a8_gemm(static_cast<const uint8_t*>(xq), static_cast<const uint8_t*>(w), out,
                                     out_dtype == QLINEAR_BF16, M, N, K, alpha, num_cus,
                                     static_cast<hipStream_t>(stream)));
}

int qlinear_nvfp4_grouped_gemm(const void* w_packed, const void* w_scale, const void* x, const uint32_t* a_offsets,
                               const int32_t* expert_ids, void* out, int out_dtype, int64_t num_groups,
                               int64_t max_tokens_per_group, int64_t num_experts, int64_t T, int64_t N, int64_t K,
                               void* stream) {
  return qlinear_nvfp4_grouped_gemm_scaled(w_packed, w_scale, x, a_offsets, expert_ids, nullptr, out, out_dtype,
                                           num_groups, max_tokens_per_group, num_experts, T, N, K, stream);
}

int qlinear_nvfp4_grouped_gemm_scaled(const void* w_packed, const void* w_scale, const void* x,
                                      const uint32_t* a_offsets, const int32_t* expert_ids, const float* expert_scale,
                                      void* out, int out_dtype, int64_t num_groups, int64_t max_tokens_per_group,
                                      int64_t num_experts, int64_t T, int64_t N, int64_t K, void* stream) {
  if (!w_packed || !w_scale || !x || !a_offsets || !expert_ids || !out) return QLINEAR_ERR_INVALID_ARG;
  if (expert_scale && !aligned(expert_scale, 4)) return QLINEAR_ERR_INVALID_ARG;
  if (num_groups <= 0 || num_groups > 65535 || max_tokens_per_group < 0 || num_experts <= 0 || T <= 0 ||
      N <= 0 || K <= 0 || K % 16 != 0)
    return QLINEAR_ERR_INVALID_ARG;
  if (!fits(num_experts, N, K) || !fits(T, K) || !fits(T, N)) return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype) || !aligned(x, 2) || !aligned(out, out_size(out_dtype)) ||
      !aligned(a_offsets, 4) || !aligned(expert_ids, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_nvfp4_grouped(static_cast<const uint8_t*>(w_packed), static_cast<const uint8_t*>(w_scale),
                                     static_cast<const uint16_t*>(x), a_offsets, expert_ids, out,
                                     out_dtype == QLINEAR_BF16, num_groups, max_tokens_per_group, num_experts, T,
                                     N, K, num_cus, static_cast<hipStream_t>(stream), expert_scale));
}

int qlinear_nvfp4_gemm(const void* w_packed, const void* w_scale, const void* x, void* out, int out_dtype,
                       int64_t M, int64_t N, int64_t K, float alpha, void* stream) {
  return nvfp4_gemm_impl(w_packed, w_scale, x, out, out_dtype, M, N, K, alpha, QLINEAR_PATH_AUTO, nullptr, 0, stream);
}

int qlinear_nvfp4_gemm_path(const void* w_packed, const void* w_scale, const void* x, void* out,
                            int out_dtype, int64_t M, int64_t N, int64_t K, float alpha, int path,
                            void* stream) {
  return nvfp4_gemm_impl(w_packed, w_scale, x, out, out_dtype, M, N, K, alpha, path, nullptr, 0, stream);
}

int qlinear_nvfp4_dequant(const void* w_packed, const void* w_scale, void* out, int out_dtype, int64_t N,
                          int64_t K, void* stream) {
  if (!w_packed || !w_scale || !out || N <= 0 || K <= 0 || K % 16 != 0 || !fits(N, K) ||
      !float_out_ok(out_dtype) || !aligned(out, out_size(out_dtype)))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_nvfp4_dequant(static_cast<const uint8_t*>(w_packed), static_cast<const uint8_t*>(w_scale),
                                     out, out_dtype == QLINEAR_BF16, N, K, static_cast<hipStream_t>(stream)));
}

int qlinear_int8_quantize_act(const void* x, void* q, float* a_scale, int64_t M, int64_t K, void* stream) {
  if (!x || !q || !a_scale || M <= 0 || K <= 0 || !fits(M, K) || !aligned(x, 2) || !aligned(a_scale, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_int8_quantize(static_cast<const uint16_t*>(x), static_cast<int8_t*>(q), a_scale, M, K,
                                     static_cast<hipStream_t>(stream)));
}

int qlinear_int8_gemm(const void* a, const void* b, const float* a_scale, const float* b_scale,
                      const void* bias, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                      void* stream) {
  if (!a || !b || !out || M <= 0 || N <= 0 || K <= 0 || K > 133144) return QLINEAR_ERR_INVALID_ARG;
  if (!fits(M, K) || !fits(N, K) || !fits(M, N)) return QLINEAR_ERR_INVALID_ARG;
  int mode;
  if (out_dtype == QLINEAR_F32) mode = 0;
  else if (out_dtype == QLINEAR_BF16) mode = 1;
  else if (out_dtype == QLINEAR_I32) mode = 2;
  else return QLINEAR_ERR_INVALID_ARG;
  if (mode != 2 && (!a_scale || !b_scale || !aligned(a_scale, 4) || !aligned(b_scale, 4)))
    return QLINEAR_ERR_INVALID_ARG;
  if (mode != 2 && bias && !aligned(bias, 2)) return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(out, mode == 1 ? 2 : 4)) return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_int8_gemm(static_cast<const int8_t*>(a), static_cast<const int8_t*>(b), a_scale, b_scale,
                                 mode == 2 ? nullptr : static_cast<const uint16_t*>(bias), out, mode, M, N, K,
                                 num_cus, static_cast<hipStream_t>(stream)));
}

int qlinear_bf16_gemm(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                      float alpha, void* stream) {
  return bf16_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, QLINEAR_PATH_AUTO, nullptr, 0, stream);
}

int qlinear_bf16_gemm_path(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                           float alpha, int path, void* stream) {
  return bf16_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, path, nullptr, 0, stream);
}

int qlinear_fp8_gemm_epilogue(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N,
                              int64_t K, float alpha, const qlinear_epilogue* epilogue, void* stream) {
  return fp8_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, QLINEAR_PATH_AUTO, nullptr, 0, stream, epilogue);
}

int qlinear_fp8_gemm_epilogue_path(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N,
                                   int64_t K, float alpha, const qlinear_epilogue* epilogue, int path, void* stream) {
  return fp8_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, path, nullptr, 0, stream, epilogue);
}

int qlinear_nvfp4_gemm_epilogue(const void* w_packed, const void* w_scale, const void* x, void* out, int out_dtype,
                                int64_t M, int64_t N, int64_t K, float alpha, const qlinear_epilogue* epilogue,
                                void* stream) {
  return nvfp4_gemm_impl(w_packed, w_scale, x, out, out_dtype, M, N, K, alpha, QLINEAR_PATH_AUTO, nullptr, 0, stream, epilogue);
}

int qlinear_bf16_gemm_epilogue(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N,
                               int64_t K, float alpha, const qlinear_epilogue* epilogue, void* stream) {
  return bf16_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, QLINEAR_PATH_AUTO, nullptr, 0, stream, epilogue);
}

int qlinear_int8_grouped_gemm(const void* a, const void* b, const float* a_scale, const float* b_scale,
                              const void* bias, const uint32_t* a_offsets, const int32_t* expert_ids, void* out,
                              int out_dtype, int64_t num_groups, int64_t max_tokens_per_group, int64_t num_experts,
                              int64_t T, int64_t N, int64_t K, void* stream) {
  if (!a || !b || !a_offsets || !expert_ids || !out) return QLINEAR_ERR_INVALID_ARG;
  if (num_groups <= 0 || num_groups > 65535 || max_tokens_per_group < 0 || num_experts <= 0 || T <= 0 ||
      N <= 0 || K <= 0 || K > 133144)
    return QLINEAR_ERR_INVALID_ARG;
  if (!fits(num_experts, N, K) || !fits(T, K) || !fits(T, N)) return QLINEAR_ERR_INVALID_ARG;
  int mode;
  if (out_dtype == QLINEAR_F32) mode = 0;
  else if (out_dtype == QLINEAR_BF16) mode = 1;
  else if (out_dtype == QLINEAR_I32) mode = 2;
  else return QLINEAR_ERR_INVALID_ARG;
  if (mode != 2 && (!a_scale || !b_scale || !aligned(a_scale, 4) || !aligned(b_scale, 4)))
    return QLINEAR_ERR_INVALID_ARG;
  if (mode != 2 && bias && !aligned(bias, 2)) return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(out, mode == 1 ? 2 : 4) || !aligned(a_offsets, 4) || !aligned(expert_ids, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_int8_grouped(static_cast<const int8_t*>(a), static_cast<const int8_t*>(b),
                                    mode == 2 ? nullptr : a_scale, mode == 2 ? nullptr : b_scale,
                                    mode == 2 ? nullptr : static_cast<const uint16_t*>(bias), a_offsets, expert_ids,
                                    out, mode, num_groups, max_tokens_per_group, num_experts, T, N, K, num_cus,
                                    static_cast<hipStream_t>(stream)));
}

int qlinear_gemm_workspace_size(int weight_format, int path, int64_t M, int64_t N, int64_t K, int64_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARG;
  *bytes = 0;
  if (M <= 0 || N <= 0 || K <= 0 || !fits(N, K) || !fits(M, K) || !fits(M, N)) return QLINEAR_ERR_INVALID_ARG;
  if (path < QLINEAR_PATH_AUTO || path > QLINEAR_PATH_SPLITK) return QLINEAR_ERR_INVALID_ARG;
  if (weight_format < QLINEAR_WEIGHT_FP8 || weight_format > QLINEAR_WEIGHT_BF16) return QLINEAR_ERR_INVALID_ARG;
  if (weight_format == QLINEAR_WEIGHT_NVFP4 && K % 16 != 0) return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  switch (weight_format) {
    case QLINEAR_WEIGHT_FP8:
      return fp8_gemm_ws_need(path, M, N, K, num_cus, bytes);
    case QLINEAR_WEIGHT_NVFP4:
      if (nvfp4_choose(path, M) == QLINEAR_PATH_TILED && K % 64 == 0)
        *bytes = int64_t(nvfp4_gemm_lds_ws_bytes(M, N, K, num_cus));
      return QLINEAR_OK;
    case QLINEAR_WEIGHT_BF16:
      if (bf16_choose(path, M, K % 8 == 0) == QLINEAR_PATH_TILED && K % 64 == 0)
        *bytes = int64_t(bf16_gemm_lds_ws_bytes(M, N, K, num_cus));
      return QLINEAR_OK;
    default:
      return QLINEAR_ERR_INVALID_ARG;
  }
}

int qlinear_fp8_gemm_ws(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                        float alpha, const qlinear_epilogue* epilogue, int path, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  return fp8_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, path, workspace, workspace_bytes, stream, epilogue);
}

int qlinear_nvfp4_gemm_ws(const void* w_packed, const void* w_scale, const void* x, void* out, int out_dtype,
                          int64_t M, int64_t N, int64_t K, float alpha, const qlinear_epilogue* epilogue, int path,
                          void* workspace, int64_t workspace_bytes, void* stream) {
  return nvfp4_gemm_impl(w_packed, w_scale, x, out, out_dtype, M, N, K, alpha, path, workspace, workspace_bytes,
                         stream, epilogue);
}

int qlinear_bf16_gemm_ws(const void* w, const void* x, void* out, int out_dtype, int64_t M, int64_t N, int64_t K,
                         float alpha, const qlinear_epilogue* epilogue, int path, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  return bf16_gemm_impl(w, x, out, out_dtype, M, N, K, alpha, path, workspace, workspace_bytes, stream, epilogue);
}

int qlinear_int4_gemm(const void* w_packed, const void* w_scale, const void* w_zero, const void* x, void* out,
                      int out_dtype, int64_t M, int64_t N, int64_t K, int64_t group_size, float alpha,
                      const qlinear_epilogue* epilogue, void* stream) {
  if (!w_packed || !w_scale || !x || !out) return QLINEAR_ERR_INVALID_ARG;
  if (M < 0 || N <= 0 || K <= 0 || !int4_group_ok(group_size, K) || !fits(N, K) || !fits(M ? M : 1, K) ||
      !fits(M ? M : 1, N))
    return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype) || !aligned(x, 2) || !aligned(w_scale, 2) || !aligned(out, out_size(out_dtype)))
    return QLINEAR_ERR_INVALID_ARG;
  Epilogue epi;
  if (int st = to_epilogue(epilogue, M ? M : 1, N, &epi)) return st;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (M == 0) return QLINEAR_OK;
  return finish(launch_int4_gemm(static_cast<const uint8_t*>(w_packed), static_cast<const uint16_t*>(w_scale),
                                 static_cast<const uint8_t*>(w_zero), static_cast<const uint16_t*>(x), out,
                                 out_dtype == QLINEAR_BF16, M, N, K, group_size, alpha, num_cus,
                                 static_cast<hipStream_t>(stream), epi));
}

int qlinear_int4_grouped_gemm(const void* w_packed, const void* w_scale, const void* w_zero, const void* x,
                              const uint32_t* a_offsets, const int32_t* expert_ids, void* out, int out_dtype,
                              int64_t num_groups, int64_t max_tokens_per_group, int64_t num_experts, int64_t T,
                              int64_t N, int64_t K, int64_t group_size, void* stream) {
  if (!w_packed || !w_scale || !x || !a_offsets || !expert_ids || !out) return QLINEAR_ERR_INVALID_ARG;
  // The kernel counts row tiles (at most T + num_groups, whatever the offsets) in int32.
  if (num_groups <= 0 || num_groups > 65535 || max_tokens_per_group < 0 || num_experts <= 0 || T < 0 ||
      T > (int64_t(1) << 30) || N <= 0 || K <= 0 || !int4_group_ok(group_size, K))
    return QLINEAR_ERR_INVALID_ARG;
  if (!fits(num_experts, N, K) || !fits(T ? T : 1, K) || !fits(T ? T : 1, N)) return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype) || !aligned(x, 2) || !aligned(w_scale, 2) || !aligned(out, out_size(out_dtype)) ||
      !aligned(a_offsets, 4) || !aligned(expert_ids, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_int4_grouped(static_cast<const uint8_t*>(w_packed), static_cast<const uint16_t*>(w_scale),
                                    static_cast<const uint8_t*>(w_zero), static_cast<const uint16_t*>(x), a_offsets,
                                    expert_ids, out, out_dtype == QLINEAR_BF16, num_groups, num_experts, T, N, K,
                                    group_size, num_cus, static_cast<hipStream_t>(stream)));
}

int qlinear_moe_route(const void* logits, int logits_dtype, int32_t* expert_ids, float* weights, int64_t T, int64_t E,
                      int64_t top_k, int renormalize, void* stream) {
  if (!logits || !expert_ids || !weights || !route_sizes_ok(T, E, top_k) || !float_out_ok(logits_dtype))
    return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(logits, out_size(logits_dtype)) || !aligned(expert_ids, 4) || !aligned(weights, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_moe_route(logits, logits_dtype == QLINEAR_BF16, expert_ids, weights, T, E, top_k,
                                 renormalize != 0, static_cast<hipStream_t>(stream)));
}

int qlinear_moe_route_backward(const void* logits, int logits_dtype, const int32_t* expert_ids,
                               const float* grad_weights, void* grad_logits, int64_t T, int64_t E, int64_t top_k,
                               int renormalize, void* stream) {
  if (!logits || !expert_ids || !grad_weights || !grad_logits || !route_sizes_ok(T, E, top_k) ||
      !float_out_ok(logits_dtype))
    return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(logits, out_size(logits_dtype)) || !aligned(grad_logits, out_size(logits_dtype)) ||
      !aligned(expert_ids, 4) || !aligned(grad_weights, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_moe_route_backward(logits, logits_dtype == QLINEAR_BF16, expert_ids, grad_weights, grad_logits,
                                          T, E, top_k, renormalize != 0, static_cast<hipStream_t>(stream)));
}

int qlinear_moe_sort_workspace_size(int64_t slots, int64_t num_experts, int64_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARG;
  *bytes = 0;
  if (slots < 0 || slots > kMaxSlots || num_experts <= 0 || num_experts > kMaxRouted) return QLINEAR_ERR_INVALID_ARG;
  *bytes = int64_t(moe_sort_ws_bytes(slots, num_experts));
  return QLINEAR_OK;
}

int qlinear_moe_sort(const int32_t* expert_ids, uint32_t* a_offsets, int32_t* row_slot, int32_t* slot_row,
                     int64_t slots, int64_t num_experts, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!expert_ids || !a_offsets || !row_slot || !slot_row) return QLINEAR_ERR_INVALID_ARG;
  int64_t need = 0;
  if (int st = qlinear_moe_sort_workspace_size(slots, num_experts, &need)) return st;
  if (int st = check_workspace(workspace, workspace_bytes)) return st;
  if (workspace_bytes < need || !aligned(expert_ids, 4) || !aligned(a_offsets, 4) || !aligned(row_slot, 4) ||
      !aligned(slot_row, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  return finish(launch_moe_sort(expert_ids, reinterpret_cast<int32_t*>(a_offsets), row_slot, slot_row, slots,
                                num_experts, static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)));
}

int qlinear_moe_gather(const void* x, const int32_t* slot_row, void* out, int dtype, int64_t T, int64_t top_k,
                       int64_t H, void* stream) {
  if (!x || !slot_row || !out || !permute_sizes_ok(T, top_k, H) || !float_out_ok(dtype))
    return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(x, out_size(dtype)) || !aligned(out, out_size(dtype)) || !aligned(slot_row, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_moe_gather(x, slot_row, out, dtype == QLINEAR_BF16, T, top_k, H,
                                  static_cast<hipStream_t>(stream)));
}

int qlinear_moe_combine(const void* rows, int rows_dtype, const int32_t* slot_row, const float* weights, void* out,
                        int out_dtype, int64_t T, int64_t top_k, int64_t H, void* stream) {
  if (!rows || !slot_row || !out || !permute_sizes_ok(T, top_k, H) || !float_out_ok(rows_dtype) ||
      !float_out_ok(out_dtype))
    return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(rows, out_size(rows_dtype)) || !aligned(out, out_size(out_dtype)) || !aligned(slot_row, 4) ||
      (weights && !aligned(weights, 4)))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_moe_combine(rows, rows_dtype == QLINEAR_BF16, slot_row, weights, out,
                                   out_dtype == QLINEAR_BF16, T, top_k, H, static_cast<hipStream_t>(stream)));
}

int qlinear_moe_combine_backward(const void* grad_out, const void* rows, int dtype, const int32_t* slot_row,
                                 const float* weights, void* grad_rows, float* grad_weights, int64_t T, int64_t top_k,
                                 int64_t H, void* stream) {
  if (!grad_out || !rows || !slot_row || !weights || !grad_rows || !grad_weights || !permute_sizes_ok(T, top_k, H) ||
      !float_out_ok(dtype))
    return QLINEAR_ERR_INVALID_ARG;
  const size_t es = out_size(dtype);
  if (!aligned(grad_out, es) || !aligned(rows, es) || !aligned(grad_rows, es) || !aligned(slot_row, 4) ||
      !aligned(weights, 4) || !aligned(grad_weights, 4))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_moe_combine_backward(grad_out, rows, dtype == QLINEAR_BF16, slot_row, weights, grad_rows,
                                            grad_weights, T, top_k, H, static_cast<hipStream_t>(stream)));
}

int qlinear_swiglu(const void* x, void* y, int dtype, int64_t M, int64_t F, void* stream) {
  if (!x || !y || M < 0 || F <= 0 || !fits(M ? M : 1, F) || !float_out_ok(dtype)) return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(x, out_size(dtype)) || !aligned(y, out_size(dtype))) return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (M == 0) return QLINEAR_OK;
  return finish(launch_swiglu(x, nullptr, y, dtype == QLINEAR_BF16, M, F, static_cast<hipStream_t>(stream)));
}

int qlinear_swiglu_backward(const void* grad_y, const void* x, void* grad_x, int dtype, int64_t M, int64_t F,
                            void* stream) {
  if (!grad_y || !x || !grad_x || M < 0 || F <= 0 || !fits(M ? M : 1, F) || !float_out_ok(dtype))
    return QLINEAR_ERR_INVALID_ARG;
  const size_t es = out_size(dtype);
  if (!aligned(grad_y, es) || !aligned(x, es) || !aligned(grad_x, es)) return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (M == 0) return QLINEAR_OK;
  return finish(launch_swiglu(x, grad_y, grad_x, dtype == QLINEAR_BF16, M, F, static_cast<hipStream_t>(stream)));
}

int qlinear_gated_gemm(const void* w, int weight_format, const void* x, const void* addend, int addend_dtype, void* out,
                       int out_dtype, void* pre, int pre_dtype, int64_t M, int64_t F, int64_t K, float alpha,
                       float alpha_up, int activation, void* stream) {
  if (!w || !x || !out || M < 0 || !gated_sizes_ok(M, F) || K <= 0 || !fits(2, F, K) || !fits(M ? M : 1, K) ||
      !gated_act_ok(activation))
    return QLINEAR_ERR_INVALID_ARG;
  if (weight_format != QLINEAR_WEIGHT_BF16 && weight_format != QLINEAR_WEIGHT_FP8) return QLINEAR_ERR_INVALID_ARG;
  if (!float_out_ok(out_dtype) || (addend && !float_out_ok(addend_dtype)) || (pre && !float_out_ok(pre_dtype)))
    return QLINEAR_ERR_INVALID_ARG;
  const bool fp8 = weight_format == QLINEAR_WEIGHT_FP8;
  if (!aligned(x, 2) || (!fp8 && !aligned(w, 2)) || !aligned(out, out_size(out_dtype)) ||
      (addend && !aligned(addend, out_size(addend_dtype))) || (pre && !aligned(pre, out_size(pre_dtype))))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (M == 0) return QLINEAR_OK;
  const GatedOut o{addend, out, pre, alpha, alpha_up, activation, out_dtype == QLINEAR_BF16,
                   addend_dtype == QLINEAR_BF16, pre_dtype == QLINEAR_BF16};
  return finish(launch_gated_gemm(w, fp8, static_cast<const uint16_t*>(x), o, M, F, K, num_cus,
                                  static_cast<hipStream_t>(stream)));
}

int qlinear_gated_backward(const void* grad_out, int grad_dtype, const void* pre, int pre_dtype, void* grad_pre, int64_t M,
                           int64_t F, int activation, void* stream) {
  if (!grad_out || !pre || !grad_pre || M < 0 || !gated_sizes_ok(M, F) || !gated_act_ok(activation) ||
      !float_out_ok(grad_dtype) || !float_out_ok(pre_dtype))
    return QLINEAR_ERR_INVALID_ARG;
  if (!aligned(grad_out, out_size(grad_dtype)) || !aligned(pre, out_size(pre_dtype)) || !aligned(grad_pre, 2))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (M == 0) return QLINEAR_OK;
  return finish(launch_gated_grad(grad_out, grad_dtype == QLINEAR_BF16, pre, pre_dtype == QLINEAR_BF16,
                                  static_cast<uint16_t*>(grad_pre), activation, M, F, static_cast<hipStream_t>(stream)));
}

int qlinear_bf16_gemm_grad_workspace_size(int64_t M, int64_t N, int64_t K, int64_t* x_bytes, int64_t* w_bytes) {
  if (x_bytes) *x_bytes = 0;
  if (w_bytes) *w_bytes = 0;
  if ((!x_bytes && !w_bytes) || M < 0 || N <= 0 || K <= 0 || !fits(M ? M : 1, N) || !fits(M ? M : 1, K) || !fits(N, K))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (x_bytes && M) *x_bytes = int64_t(bf16_product_ws_bytes(M, K, N, num_cus));
  if (w_bytes && M) *w_bytes = int64_t(bf16_product_ws_bytes(N, K, M, num_cus));
  return QLINEAR_OK;
}

int qlinear_bf16_gemm_grad_x(const void* grad_out, const void* w, void* grad_x, int dtype, int64_t M, int64_t N, int64_t K,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  if (!linear_grad_ok(grad_out, w, grad_x, dtype, M, N, K)) return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(workspace, workspace_bytes)) return st;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (M == 0) return QLINEAR_OK;
  return finish(launch_bf16_grad_x(static_cast<const uint16_t*>(grad_out), static_cast<const uint16_t*>(w), grad_x,
                                   dtype == QLINEAR_BF16, M, N, K, num_cus, static_cast<float*>(workspace),
                                   size_t(workspace_bytes), static_cast<hipStream_t>(stream)));
}

int qlinear_bf16_gemm_grad_w(const void* grad_out, const void* x, void* grad_w, int dtype, int64_t M, int64_t N, int64_t K,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  if (!linear_grad_ok(grad_out, x, grad_w, dtype, M, N, K)) return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(workspace, workspace_bytes)) return st;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (M == 0) return finish(launch_clear(grad_w, N * K * int64_t(out_size(dtype)), static_cast<hipStream_t>(stream)));
  return finish(launch_bf16_grad_w(static_cast<const uint16_t*>(grad_out), static_cast<const uint16_t*>(x), grad_w,
                                   dtype == QLINEAR_BF16, M, N, K, num_cus, static_cast<float*>(workspace),
                                   size_t(workspace_bytes), static_cast<hipStream_t>(stream)));
}

int qlinear_lora_workspace_size(int64_t num_groups, int64_t T, int64_t K, int64_t R, int64_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARG;
  *bytes = 0;
  if (!lora_sizes_ok(num_groups, 1, T, 1, K, R)) return QLINEAR_ERR_INVALID_ARG;
  *bytes = int64_t(lora_ws_bytes(T, num_groups, K, R));
  return QLINEAR_OK;
}

int qlinear_lora_gemm(const void* x, const void* a, const void* b, const uint32_t* a_offsets, const int32_t* adapter_ids,
                      const float* scale, const void* base, void* out, int out_dtype, float* z, int64_t num_groups,
                      int64_t num_adapters, int64_t T, int64_t N, int64_t K, int64_t R, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  if (!x || !a || !b || !a_offsets || !adapter_ids || !out || !float_out_ok(out_dtype) ||
      !lora_sizes_ok(num_groups, num_adapters, T, N, K, R))
    return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(workspace, workspace_bytes)) return st;
  if (workspace_bytes < int64_t(lora_ws_bytes(T, num_groups, K, R))) return QLINEAR_ERR_INVALID_ARG;
  const size_t es = out_size(out_dtype);
  if (!aligned(x, 2) || !aligned(a, 2) || !aligned(b, 2) || !aligned(a_offsets, 4) || !aligned(adapter_ids, 4) ||
      !aligned(scale, 4) || !aligned(base, es) || !aligned(out, es) || !aligned(z, 16))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_lora(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(a),
                            static_cast<const uint16_t*>(b), a_offsets, adapter_ids, scale, base, out,
                            out_dtype == QLINEAR_BF16, z, num_groups, num_adapters, T, N, K, R,
                            static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

int qlinear_lora_backward_workspace_size(int64_t num_groups, int64_t num_adapters, int64_t T, int64_t N, int64_t K,
                                         int64_t R, int64_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARG;
  *bytes = 0;
  if (!lora_sizes_ok(num_groups, num_adapters, T, N, K, R)) return QLINEAR_ERR_INVALID_ARG;
  *bytes = int64_t(lora_grad_ws_bytes(T, num_groups, num_adapters, N, K, R));
  return QLINEAR_OK;
}

int qlinear_lora_gemm_backward(const void* grad_out, const void* x, const float* z, const void* a, const void* b,
                               const uint32_t* a_offsets, const int32_t* adapter_ids, const float* scale, const void* base,
                               void* grad_x, int x_dtype, void* grad_a, void* grad_b, int param_dtype, int64_t num_groups,
                               int64_t num_adapters, int64_t T, int64_t N, int64_t K, int64_t R, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  if (!grad_out || !x || !z || !a || !b || !a_offsets || !adapter_ids || !grad_x || !grad_a || !grad_b ||
      !float_out_ok(x_dtype) || !float_out_ok(param_dtype) || !lora_sizes_ok(num_groups, num_adapters, T, N, K, R))
    return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(workspace, workspace_bytes)) return st;
  if (workspace_bytes < int64_t(lora_grad_ws_bytes(T, num_groups, num_adapters, N, K, R))) return QLINEAR_ERR_INVALID_ARG;
  const size_t xs = out_size(x_dtype), ps = out_size(param_dtype);
  if (!aligned(grad_out, 2) || !aligned(x, 2) || !aligned(z, 4) || !aligned(a, 2) || !aligned(b, 2) ||
      !aligned(a_offsets, 4) || !aligned(adapter_ids, 4) || !aligned(scale, 4) || !aligned(base, xs) ||
      !aligned(grad_x, xs) || !aligned(grad_a, ps) || !aligned(grad_b, ps))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  const auto s = static_cast<hipStream_t>(stream);
  if (T == 0) {
    if (int st = finish(launch_clear(grad_a, num_adapters * R * K * int64_t(ps), s))) return st;
    return finish(launch_clear(grad_b, num_adapters * R * N * int64_t(ps), s));
  }
  return finish(launch_lora_grad(static_cast<const uint16_t*>(grad_out), static_cast<const uint16_t*>(x), z,
                                 static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b), a_offsets, adapter_ids,
                                 scale, base, grad_x, x_dtype == QLINEAR_BF16, grad_a, grad_b,
                                 param_dtype == QLINEAR_BF16, num_groups, num_adapters, T, N, K, R,
                                 static_cast<char*>(workspace), s));
}

int qlinear_block_norm(const void* residual, int residual_dtype, const void* weight, int param_dtype, const void* block,
                       int dtype, const void* block_weight, const void* gate, int64_t gates, void* residual_out,
                       void* out, int64_t T, int64_t H, float residual_scale, float eps, void* stream) {
  if (!residual || !weight || !out || !norm_ok(residual_dtype, dtype, param_dtype, block, block_weight, gate, gates, T, H, eps) ||
      (block != nullptr) != (residual_out != nullptr))
    return QLINEAR_ERR_INVALID_ARG;
  const size_t rs = out_size(residual_dtype), es = out_size(dtype), ps = out_size(param_dtype);
  if (!aligned(residual, rs) || !aligned(residual_out, rs) || !aligned(block, es) || !aligned(out, es) ||
      !aligned(weight, ps) || !aligned(block_weight, ps) || !aligned(gate, ps))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  if (T == 0) return QLINEAR_OK;
  return finish(launch_block_norm(residual, residual_dtype == QLINEAR_BF16, weight, param_dtype == QLINEAR_BF16, block,
                                  dtype == QLINEAR_BF16, block_weight, gate, gates, residual_out, out, T, H,
                                  residual_scale, eps, static_cast<hipStream_t>(stream)));
}

int qlinear_block_norm_backward_workspace_size(int64_t T, int64_t H, int post, int gated, int64_t* bytes) {
  if (!bytes) return QLINEAR_ERR_INVALID_ARG;
  *bytes = 0;
  if (T < 0 || H <= 0 || H > kMaxNormWidth || !fits(T ? T : 1, H)) return QLINEAR_ERR_INVALID_ARG;
  *bytes = int64_t(block_norm_grad_ws_bytes(T, H, post != 0, gated != 0));
  return QLINEAR_OK;
}

int qlinear_block_norm_backward(const void* grad_out, int dtype, const void* grad_residual_out, const void* residual_out,
                                int residual_dtype, const void* weight, int param_dtype, const void* block,
                                const void* block_weight, const void* gate, int64_t gates, void* grad_residual,
                                void* grad_block, void* grad_weight, void* grad_block_weight, void* grad_gate, int64_t T,
                                int64_t H, float residual_scale, float eps, void* workspace, int64_t workspace_bytes,
                                void* stream) {
  if (!grad_out || !residual_out || !weight || !grad_residual || !grad_weight ||
      !norm_ok(residual_dtype, dtype, param_dtype, block, block_weight, gate, gates, T, H, eps) ||
      (block != nullptr) != (grad_block != nullptr) || (block_weight != nullptr) != (grad_block_weight != nullptr) ||
      (gate != nullptr) != (grad_gate != nullptr))
    return QLINEAR_ERR_INVALID_ARG;
  if (int st = check_workspace(workspace, workspace_bytes)) return st;
  if (workspace_bytes < int64_t(block_norm_grad_ws_bytes(T, H, block_weight != nullptr, gate != nullptr)))
    return QLINEAR_ERR_INVALID_ARG;
  const size_t rs = out_size(residual_dtype), es = out_size(dtype), ps = out_size(param_dtype);
  if (!aligned(grad_out, es) || !aligned(grad_residual_out, rs) || !aligned(residual_out, rs) || !aligned(weight, ps) ||
      !aligned(block, es) || !aligned(block_weight, ps) || !aligned(gate, ps) || !aligned(grad_residual, rs) ||
      !aligned(grad_block, es) || !aligned(grad_weight, ps) || !aligned(grad_block_weight, ps) || !aligned(grad_gate, ps))
    return QLINEAR_ERR_INVALID_ARG;
  int num_cus = 0;
  if (int st = current_device(&num_cus)) return st;
  const auto s = static_cast<hipStream_t>(stream);
  if (T == 0) {
    if (int st = finish(launch_clear(grad_weight, H * int64_t(ps), s))) return st;
    if (block_weight)
      if (int st = finish(launch_clear(grad_block_weight, H * int64_t(ps), s))) return st;
    return gate ? finish(launch_clear(grad_gate, gates * H * int64_t(ps), s)) : QLINEAR_OK;
  }
  return finish(launch_block_norm_grad(grad_out, dtype == QLINEAR_BF16, grad_residual_out, residual_out,
                                       residual_dtype == QLINEAR_BF16, weight, param_dtype == QLINEAR_BF16, block,
                                       block_weight, gate, gates, grad_residual, grad_block, grad_weight,
                                       grad_block_weight, grad_gate, T, H, block ? residual_scale : 1.f, eps,
                                       static_cast<float*>(workspace), s));
}

}  // extern "C"
