"""Python binding of libqlinear, the MI355X (gfx950) weight-quantized linear
layer ``out = x @ dequant(W)^T``.

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libqlinear.so``.  torch provides device memory and the current
stream.  There is no fallback: if the library is not built, importing this
package raises ImportError.

The C entry points (``include/qlinear.h``) are exposed unchanged as
``weight_quantized_linear_amd.lib.<name>``; the functions below take and
return torch tensors.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "lib",
    "LIB_PATH",
    "QLinearError",
    "EXPORTED",
    "fp8_gemv",
    "fp8_gemm",
    "bf16_gemm",
    "fp8_materialize",
    "fp8_grouped_gemm",
    "nvfp4_grouped_gemm",
    "int8_grouped_gemm",
    "fp8_quantize_act",
    "fp8_w8a8_gemm",
    "nvfp4_gemm",
    "nvfp4_dequant",
    "int8_quantize_act",
    "int8_gemm",
    "int4_gemm",
    "int4_grouped_gemm",
    "moe_route",
    "moe_route_backward",
    "moe_sort",
    "moe_gather",
    "moe_combine",
    "moe_combine_backward",
    "swiglu",
    "swiglu_backward",
    "PATHS",
    "gemm_workspace_bytes",
    "WEIGHT_FP8",
    "WEIGHT_NVFP4",
    "WEIGHT_BF16",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqlinear.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_DEVICE, ERR_LAUNCH, ERR_SCRATCH_LIMIT = 0, 1, 2, 3, 4, 5
F32, BF16, I32 = 0, 1, 2
PATHS = {"auto": 0, "gemv": 1, "skinny": 2, "tiled": 3, "splitk": 4}

_p, _i, _i64, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class EpilogueDesc(ctypes.Structure):
    """``qlinear_epilogue``: the fused element-wise steps of the *_epilogue calls."""
    _fields_ = [("row_scale", _p), ("col_scale", _p), ("bias", _p), ("residual", _p),
                ("residual_ld", _i64), ("residual_dtype", _i), ("activation", _i)]


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu_tanh": 3}
_EP = ctypes.POINTER(EpilogueDesc)

# name -> argument types (all return int status except where noted)
EXPORTED = {
    "qlinear_abi_version": [],
    "qlinear_status_string": [_i],
    "qlinear_fp8_gemv": [_p, _p, _p, _i, _i64, _i64, _f, _p],
    "qlinear_fp8_gemm": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _p],
    "qlinear_fp8_gemm_path": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _i, _p],
    "qlinear_bf16_gemm": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _p],
    "qlinear_bf16_gemm_path": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _i, _p],
    "qlinear_fp8_materialize": [_p, _p, _i, _i64, _i64, _p],
    "qlinear_fp8_grouped_gemm": [_p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _i64, _i64, _i64, _p],
    "qlinear_nvfp4_gemm": [_p, _p, _p, _p, _i, _i64, _i64, _i64, _f, _p],
    "qlinear_nvfp4_grouped_gemm": [_p, _p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _i64, _i64, _i64, _p],
    "qlinear_fp8_quantize_act": [_p, _p, _f, _i64, _i64, _p],
    "qlinear_fp8_w8a8_gemm": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _p],
    "qlinear_nvfp4_gemm_path": [_p, _p, _p, _p, _i, _i64, _i64, _i64, _f, _i, _p],
    "qlinear_nvfp4_dequant": [_p, _p, _p, _i, _i64, _i64, _p],
    "qlinear_int8_quantize_act": [_p, _p, _p, _i64, _i64, _p],
    "qlinear_int8_gemm": [_p, _p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _p],
    "qlinear_fp8_gemm_epilogue": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _p],
    "qlinear_fp8_gemm_epilogue_path": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _i, _p],
    "qlinear_nvfp4_gemm_epilogue": [_p, _p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _p],
    "qlinear_bf16_gemm_epilogue": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _p],
    "qlinear_fp8_grouped_gemm_scaled": [_p, _p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _i64, _i64, _i64, _p],
    "qlinear_nvfp4_grouped_gemm_scaled": [_p, _p, _p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _i64, _i64, _i64, _p],
    "qlinear_int8_grouped_gemm": [_p, _p, _p, _p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _i64, _i64, _i64, _p],
    "qlinear_gemm_workspace_size": [_i, _i, _i64, _i64, _i64, ctypes.POINTER(_i64)],
    "qlinear_fp8_gemm_ws": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _i, _p, _i64, _p],
    "qlinear_nvfp4_gemm_ws": [_p, _p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _i, _p, _i64, _p],
    "qlinear_bf16_gemm_ws": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _i, _p, _i64, _p],
    "qlinear_fp8_gemm_noalloc": [_p, _p, _p, _i, _i64, _i64, _i64, _f, _EP, _i, _p],
    "qlinear_int4_gemm": [_p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _i64, _f, _EP, _p],
    "qlinear_int4_grouped_gemm": [_p, _p, _p, _p, _p, _p, _p, _i, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _p],
    "qlinear_moe_route": [_p, _i, _p, _p, _i64, _i64, _i64, _i, _p],
    "qlinear_moe_route_backward": [_p, _i, _p, _p, _p, _i64, _i64, _i64, _i, _p],
    "qlinear_moe_sort_workspace_size": [_i64, _i64, ctypes.POINTER(_i64)],
    "qlinear_moe_sort": [_p, _p, _p, _p, _i64, _i64, _p, _i64, _p],
    "qlinear_moe_gather": [_p, _p, _p, _i, _i64, _i64, _i64, _p],
    "qlinear_moe_combine": [_p, _i, _p, _p, _p, _i, _i64, _i64, _i64, _p],
    "qlinear_moe_combine_backward": [_p, _p, _i, _p, _p, _p, _p, _i64, _i64, _i64, _p],
    "qlinear_swiglu": [_p, _p, _i, _i64, _i64, _p],
    "qlinear_swiglu_backward": [_p, _p, _p, _i, _i64, _i64, _p],
}

WEIGHT_FP8, WEIGHT_NVFP4, WEIGHT_BF16 = 0, 1, 2


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python weight_quantized_linear_amd/build.py`")
    handle = ctypes.CDLL(LIB_PATH)
    for name, argtypes in EXPORTED.items():
        fn = getattr(handle, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_char_p if name == "qlinear_status_string" else _i
    return handle


lib = _load()


class QLinearError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {lib.qlinear_status_string(status).decode()} (status {status})")


def _check(status: int, call: str):
    if status != OK:
        raise QLinearError(status, call)


def _stream(t: torch.Tensor):
    """The handle of the current stream of t's device.  Read as a plain integer: a
    torch.cuda.Stream object costs 2.0 us a call, this 0.1, and a call of a small kernel
    is bound by its host side (10 us in all before, with 4 us in the C call)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _ptr(t: torch.Tensor):
    return t.data_ptr()


def _as_u8(w: torch.Tensor, what: str) -> torch.Tensor:
    if w.dtype in (torch.uint8, torch.int8):
        return w
    if w.dtype == torch.float8_e4m3fn:
        return w.view(torch.uint8)
    raise TypeError(f"{what}: expected float8_e4m3fn/uint8 storage, got {w.dtype}")


def _as_bf16(x: torch.Tensor, what: str) -> torch.Tensor:
    if x.dtype == torch.bfloat16:
        return x
    if x.dtype in (torch.int16, torch.uint16):
        return x.view(torch.bfloat16)
    raise TypeError(f"{what}: expected bfloat16 storage, got {x.dtype}")


def _require(t: torch.Tensor, what: str):
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


_OUT_CODES = {torch.float32: F32, torch.bfloat16: BF16}


def _out(out, shape, dtype, device):
    if out is None:
        if len(shape) == 2:  # the same tensor as torch.empty's, in 1.3 us instead of 1.7
            return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
        return torch.empty(shape, dtype=dtype, device=device)
    _require(out, "out")
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError(f"out must be {tuple(shape)} {dtype}, got {tuple(out.shape)} {out.dtype}")
    return out


def _epilogue(m: int, n: int, row_scale, col_scale, bias, residual, activation: str):
    """The ``qlinear_epilogue`` of the given tensors (None when nothing is fused)."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    if row_scale is None and col_scale is None and bias is None and residual is None and activation == "none":
        return None
    d = EpilogueDesc(None, None, None, None, 0, F32, ACTIVATIONS[activation])
    for t, name, size, dt in ((row_scale, "row_scale", m, torch.float32), (col_scale, "col_scale", n, torch.float32),
                              (bias, "bias", n, torch.bfloat16)):
        if t is None:
            continue
        _require(t, name)
        if t.dtype != dt or t.numel() != size:
            raise ValueError(f"{name} must be {dt} with {size} elements")
        setattr(d, name, t.data_ptr())
    if residual is not None:
        if not residual.is_cuda or residual.dim() != 2 or residual.shape[0] != m or residual.shape[1] < n \
                or residual.stride(1) != 1 or residual.dtype not in _OUT_CODES:
            raise ValueError("residual must be a float32/bfloat16 device tensor [M, >= N] with unit column stride")
        d.residual = residual.data_ptr()
        d.residual_ld = residual.stride(0) if m > 1 else residual.shape[1]
        d.residual_dtype = _OUT_CODES[residual.dtype]
    return d


def _epi_ref(d):
    return ctypes.byref(d) if d is not None else None


def gemm_workspace_bytes(weight_format: int, m: int, n: int, k: int, path: str = "auto") -> int:
    """Bytes of split-K workspace the ``*_gemm_ws`` call of ``weight_format``
    (WEIGHT_FP8 / WEIGHT_NVFP4 / WEIGHT_BF16) takes for (m, n, k) on the
    current device (``qlinear_gemm_workspace_size``); 0 = none."""
    b = _i64(0)
    _check(lib.qlinear_gemm_workspace_size(weight_format, PATHS[path], m, n, k, ctypes.byref(b)),
           "qlinear_gemm_workspace_size")
    return int(b.value)


def _workspace(workspace, weight_format: int, m: int, n: int, k: int, path: str, device):
    """(pointer, bytes, tensor) of the split-K workspace: "auto" allocates what
    the call takes (a torch tensor, so torch's caching allocator serves it),
    None passes none (whole-K tiles), a tensor is used as given."""
    if workspace is None:
        return None, 0, None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a device tensor")
        nbytes = gemm_workspace_bytes(weight_format, m, n, k, path)
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _require(workspace, "workspace")
    return _ptr(workspace), workspace.numel() * workspace.element_size(), workspace


def fp8_gemm(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
             out_dtype: torch.dtype = torch.bfloat16, alpha: float = 1.0, path: str = "auto",
             row_scale: torch.Tensor | None = None, col_scale: torch.Tensor | None = None,
             bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
             activation: str = "none", workspace="auto") -> torch.Tensor:
    """out[M, N] = alpha * x[M, K] @ dec_e4m3(w[N, K])^T (``qlinear_fp8_gemm_ws``), with
    the fused epilogue of any of row_scale / col_scale / bias / residual / activation,
    the kernel family ``path`` and the split-K ``workspace`` ("auto": allocated to the
    size ``qlinear_gemm_workspace_size`` gives; None: none)."""
    w = _as_u8(w, "w")
    x = _as_bf16(x, "x")
    _require(w, "w")
    _require(x, "x")
    if w.dim() != 2 or x.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"shapes: w {tuple(w.shape)} must be [N, K], x {tuple(x.shape)} must be [M, K]")
    m, k = x.shape
    n = w.shape[0]
    out = _out(out, (m, n), out_dtype, x.device)
    d = _epilogue(m, n, row_scale, col_scale, bias, residual, activation)
    wsp, wsb, _keep = _workspace(workspace, WEIGHT_FP8, m, n, k, path, x.device)
    st = lib.qlinear_fp8_gemm_ws(_ptr(w), _ptr(x), _ptr(out), _OUT_CODES[out_dtype], m, n, k, float(alpha),
                                 _epi_ref(d), PATHS[path], wsp, wsb, _stream(x))
    _check(st, "qlinear_fp8_gemm_ws")
    return out


def bf16_gemm(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.bfloat16, alpha: float = 1.0, path: str = "auto",
              row_scale: torch.Tensor | None = None, col_scale: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
              activation: str = "none", workspace="auto") -> torch.Tensor:
    """Dense bf16 control: out[M, N] = alpha * x[M, K] @ w[N, K]^T (``qlinear_bf16_gemm_ws``);
    epilogue, ``path`` and ``workspace`` as ``fp8_gemm``."""
    w = _as_bf16(w, "w")
    x = _as_bf16(x, "x")
    _require(w, "w")
    _require(x, "x")
    if w.dim() != 2 or x.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"shapes: w {tuple(w.shape)} must be [N, K], x {tuple(x.shape)} must be [M, K]")
    m, k = x.shape
    n = w.shape[0]
    out = _out(out, (m, n), out_dtype, x.device)
    d = _epilogue(m, n, row_scale, col_scale, bias, residual, activation)
    wsp, wsb, _keep = _workspace(workspace, WEIGHT_BF16, m, n, k, path, x.device)
    st = lib.qlinear_bf16_gemm_ws(_ptr(w), _ptr(x), _ptr(out), _OUT_CODES[out_dtype], m, n, k, float(alpha),
                                  _epi_ref(d), PATHS[path], wsp, wsb, _stream(x))
    _check(st, "qlinear_bf16_gemm_ws")
    return out


def fp8_gemv(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
             out_dtype: torch.dtype = torch.float32, alpha: float = 1.0) -> torch.Tensor:
    """out[N] = alpha * dec_e4m3(w[N, K]) @ x[K] (``qlinear_fp8_gemv``)."""
    w = _as_u8(w, "w")
    x = _as_bf16(x, "x")
    _require(w, "w")
    _require(x, "x")
    if w.dim() != 2 or x.numel() != w.shape[1]:
        raise ValueError("w must be [N, K] and x must hold K elements")
    n, k = w.shape
    out = _out(out, (n,), out_dtype, x.device)
    st = lib.qlinear_fp8_gemv(_ptr(w), _ptr(x), _ptr(out), _OUT_CODES[out_dtype], n, k, float(alpha), _stream(x))
    _check(st, "qlinear_fp8_gemv")
    return out


def fp8_materialize(w: torch.Tensor, out_dtype: torch.dtype = torch.float32,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Dense [N, K] copy of the decoded FP8 weight (``qlinear_fp8_materialize``)."""
    w = _as_u8(w, "w")
    _require(w, "w")
    w2 = w.reshape(1, -1) if w.dim() == 1 else w
    n, k = w2.shape
    out = _out(out, tuple(w.shape), out_dtype, w.device)
    st = lib.qlinear_fp8_materialize(_ptr(w2), _ptr(out), _OUT_CODES[out_dtype], n, k, _stream(w))
    _check(st, "qlinear_fp8_materialize")
    return out


def _expert_scale(expert_scale, e: int):
    if expert_scale is None:
        return None
    _require(expert_scale, "expert_scale")
    if expert_scale.dtype != torch.float32 or expert_scale.numel() != e:
        raise ValueError(f"expert_scale must be float32 with {e} elements")
    return _ptr(expert_scale)


def fp8_grouped_gemm(w: torch.Tensor, x: torch.Tensor, a_offsets: torch.Tensor, expert_ids: torch.Tensor,
                     out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                     max_tokens_per_group: int | None = None,
                     expert_scale: torch.Tensor | None = None) -> torch.Tensor:
    """Grouped MoE W8A16 (``qlinear_fp8_grouped_gemm_scaled``): rows a_offsets[z] ..
    a_offsets[z+1]-1 of x times dec(w[expert_ids[z]])^T, times expert_scale[expert_ids[z]]
    when given (raw otherwise).  Rows outside every group keep whatever ``out`` held
    (a new ``out`` starts uninitialised)."""
    w = _as_u8(w, "w")
    x = _as_bf16(x, "x")
    for t, name in ((w, "w"), (x, "x"), (a_offsets, "a_offsets"), (expert_ids, "expert_ids")):
        _require(t, name)
    if a_offsets.dtype not in (torch.int32, torch.uint32) or expert_ids.dtype != torch.int32:
        raise TypeError("a_offsets must be uint32/int32 and expert_ids int32")
    if w.dim() != 3 or x.dim() != 2 or x.shape[1] != w.shape[2]:
        raise ValueError("w must be [E, N, K] and x [T, K]")
    g = expert_ids.numel()
    if a_offsets.numel() != g + 1:
        raise ValueError("a_offsets needs num_groups + 1 entries")
    e, n, k = w.shape
    t = x.shape[0]
    if max_tokens_per_group is None:
        max_tokens_per_group = t
    out = _out(out, (t, n), out_dtype, x.device)
    st = lib.qlinear_fp8_grouped_gemm_scaled(_ptr(w), _ptr(x), _ptr(a_offsets), _ptr(expert_ids),
                                             _expert_scale(expert_scale, e), _ptr(out), _OUT_CODES[out_dtype], g,
                                             int(max_tokens_per_group), e, t, n, k, _stream(x))
    _check(st, "qlinear_fp8_grouped_gemm_scaled")
    return out


def fp8_quantize_act(x: torch.Tensor, input_scale: float, q: torch.Tensor | None = None) -> torch.Tensor:
    """Static per-tensor FP8 activation quantisation (``qlinear_fp8_quantize_act``):
    q = E4M3(clamp(x / input_scale, -448, 448)) as uint8 codes [M, K]."""
    x = _as_bf16(x, "x")
    _require(x, "x")
    m, k = x.shape
    if q is None:
        q = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    elif q.dtype != torch.uint8 or tuple(q.shape) != (m, k) or not q.is_contiguous():
        raise ValueError("q must be a contiguous uint8 [M, K] tensor")
    st = lib.qlinear_fp8_quantize_act(_ptr(x), _ptr(q), float(input_scale), m, k, _stream(x))
    _check(st, "qlinear_fp8_quantize_act")
    return q


def fp8_w8a8_gemm(xq: torch.Tensor, w: torch.Tensor, out: torch.Tensor | None = None,
                  out_dtype: torch.dtype = torch.bfloat16, alpha: float = 1.0) -> torch.Tensor:
    """FP8 W8A8 (``qlinear_fp8_w8a8_gemm``): out = alpha * dec(xq) @ dec(w)^T,
    xq and w float8_e4m3fn codes (uint8 or float8 tensors)."""
    xq = _as_u8(xq, "xq")
    w = _as_u8(w, "w")
    for t, name in ((xq, "xq"), (w, "w")):
        _require(t, name)
    m, k = xq.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError("xq must be [M, K] and w [N, K]")
    out = _out(out, (m, n), out_dtype, xq.device)
    st = lib.qlinear_fp8_w8a8_gemm(_ptr(xq), _ptr(w), _ptr(out), _OUT_CODES[out_dtype], m, n, k, float(alpha),
                                   _stream(xq))
    _check(st, "qlinear_fp8_w8a8_gemm")
    return out


def nvfp4_grouped_gemm(w_packed: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, a_offsets: torch.Tensor,
                       expert_ids: torch.Tensor, out: torch.Tensor | None = None,
                       out_dtype: torch.dtype = torch.bfloat16, max_tokens_per_group: int | None = None,
                       expert_scale: torch.Tensor | None = None) -> torch.Tensor:
    """Grouped MoE W4A16 NVFP4 (``qlinear_nvfp4_grouped_gemm_scaled``): rows a_offsets[z] ..
    a_offsets[z+1]-1 of x times D_e^T, e = expert_ids[z], D_e the expert's NVFP4
    weight (w_packed [E, N, K/2], w_scale [E, N, K/16]), times expert_scale[e] when
    given (raw otherwise).  Rows outside every group keep whatever ``out`` held (a
    new ``out`` starts uninitialised)."""
    p = _as_u8(w_packed, "w_packed")
    sc = _as_u8(w_scale, "w_scale")
    x = _as_bf16(x, "x")
    for t, name in ((p, "w_packed"), (sc, "w_scale"), (x, "x"), (a_offsets, "a_offsets"), (expert_ids, "expert_ids")):
        _require(t, name)
    if a_offsets.dtype not in (torch.int32, torch.uint32) or expert_ids.dtype != torch.int32:
        raise TypeError("a_offsets must be uint32/int32 and expert_ids int32")
    if p.dim() != 3 or x.dim() != 2:
        raise ValueError("w_packed must be [E, N, K/2] and x [T, K]")
    e, n, _ = p.shape
    t, k = x.shape
    if tuple(p.shape) != (e, n, k // 2) or tuple(sc.shape) != (e, n, k // 16):
        raise ValueError("w_packed must be [E, N, K/2] and w_scale [E, N, K/16]")
    g = expert_ids.numel()
    if a_offsets.numel() != g + 1:
        raise ValueError("a_offsets needs num_groups + 1 entries")
    if max_tokens_per_group is None:
        max_tokens_per_group = t
    out = _out(out, (t, n), out_dtype, x.device)
    st = lib.qlinear_nvfp4_grouped_gemm_scaled(_ptr(p), _ptr(sc), _ptr(x), _ptr(a_offsets), _ptr(expert_ids),
                                               _expert_scale(expert_scale, e), _ptr(out), _OUT_CODES[out_dtype], g,
                                               int(max_tokens_per_group), e, t, n, k, _stream(x))
    _check(st, "qlinear_nvfp4_grouped_gemm_scaled")
    return out


def nvfp4_gemm(w_packed: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
               out_dtype: torch.dtype = torch.bfloat16, alpha: float = 1.0, path: str = "auto",
               row_scale: torch.Tensor | None = None, col_scale: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
               activation: str = "none", workspace="auto") -> torch.Tensor:
    """out[M, N] = alpha * x[M, K] @ D^T, D the NVFP4 weight (``qlinear_nvfp4_gemm_ws``);
    epilogue, ``path`` and ``workspace`` as ``fp8_gemm``."""
    p = _as_u8(w_packed, "w_packed")
    sc = _as_u8(w_scale, "w_scale")
    x = _as_bf16(x, "x")
    for t, name in ((p, "w_packed"), (sc, "w_scale"), (x, "x")):
        _require(t, name)
    m, k = x.shape
    n = p.shape[0]
    if tuple(p.shape) != (n, k // 2) or tuple(sc.shape) != (n, k // 16):
        raise ValueError("w_packed must be [N, K/2] and w_scale [N, K/16]")
    out = _out(out, (m, n), out_dtype, x.device)
    d = _epilogue(m, n, row_scale, col_scale, bias, residual, activation)
    wsp, wsb, _keep = _workspace(workspace, WEIGHT_NVFP4, m, n, k, path, x.device)
    st = lib.qlinear_nvfp4_gemm_ws(_ptr(p), _ptr(sc), _ptr(x), _ptr(out), _OUT_CODES[out_dtype], m, n, k,
                                   float(alpha), _epi_ref(d), PATHS[path], wsp, wsb, _stream(x))
    _check(st, "qlinear_nvfp4_gemm_ws")
    return out


def nvfp4_dequant(w_packed: torch.Tensor, w_scale: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Dense [N, K] dequantised NVFP4 weight (``qlinear_nvfp4_dequant``)."""
    p = _as_u8(w_packed, "w_packed")
    sc = _as_u8(w_scale, "w_scale")
    _require(p, "w_packed")
    _require(sc, "w_scale")
    n, half = p.shape
    k = 2 * half
    if tuple(sc.shape) != (n, k // 16):
        raise ValueError("w_scale must be [N, K/16]")
    out = _out(out, (n, k), out_dtype, p.device)
    st = lib.qlinear_nvfp4_dequant(_ptr(p), _ptr(sc), _ptr(out), _OUT_CODES[out_dtype], n, k, _stream(p))
    _check(st, "qlinear_nvfp4_dequant")
    return out


def int8_quantize_act(x: torch.Tensor, q: torch.Tensor | None = None, a_scale: torch.Tensor | None = None):
    """Per-row absmax int8 quantisation (``qlinear_int8_quantize_act``) -> (q int8 [M, K], a_scale f32 [M])."""
    x = _as_bf16(x, "x")
    _require(x, "x")
    m, k = x.shape
    q = _out(q, (m, k), torch.int8, x.device)
    a_scale = _out(a_scale, (m,), torch.float32, x.device)
    st = lib.qlinear_int8_quantize_act(_ptr(x), _ptr(q), _ptr(a_scale), m, k, _stream(x))
    _check(st, "qlinear_int8_quantize_act")
    return q, a_scale


_INT8_OUT = {torch.float32: F32, torch.bfloat16: BF16, torch.int32: I32}


def int8_gemm(a: torch.Tensor, b: torch.Tensor, a_scale: torch.Tensor | None, b_scale: torch.Tensor | None,
              bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """W8A8: out = (a @ b^T) * a_scale[:, None] * b_scale[None, :] + bias (``qlinear_int8_gemm``);
    out_dtype=torch.int32 returns the raw accumulators."""
    for t, name in ((a, "a"), (b, "b")):
        _require(t, name)
        if t.dtype != torch.int8:
            raise TypeError(f"{name} must be int8")
    m, k = a.shape
    n = b.shape[0]
    if b.shape[1] != k:
        raise ValueError("a must be [M, K] and b [N, K]")
    args = []
    for t, name, shape in ((a_scale, "a_scale", (m,)), (b_scale, "b_scale", (n,))):
        if t is None:
            args.append(None)
            continue
        _require(t, name)
        if t.dtype != torch.float32 or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be float32 {shape}")
        args.append(_ptr(t))
    bias_p = None
    if bias is not None:
        bias = _as_bf16(bias, "bias")
        _require(bias, "bias")
        if tuple(bias.shape) != (n,):
            raise ValueError("bias must be [N]")
        bias_p = _ptr(bias)
    out = _out(out, (m, n), out_dtype, a.device)
    st = lib.qlinear_int8_gemm(_ptr(a), _ptr(b), args[0], args[1], bias_p, _ptr(out), _INT8_OUT[out_dtype],
                               m, n, k, _stream(a))
    _check(st, "qlinear_int8_gemm")
    return out


def int8_grouped_gemm(a: torch.Tensor, b: torch.Tensor, a_scale: torch.Tensor | None, b_scale: torch.Tensor | None,
                      a_offsets: torch.Tensor, expert_ids: torch.Tensor, bias: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                      max_tokens_per_group: int | None = None) -> torch.Tensor:
    """Grouped MoE W8A8 (``qlinear_int8_grouped_gemm``): rows a_offsets[z] ..
    a_offsets[z+1]-1 of the int8 activation a [T, K] times b[expert_ids[z]] [N, K]^T,
    dequantised by a_scale[r] * b_scale[e, n] + bias[e, n] (out_dtype bf16 / f32) or
    raw int32 accumulators (out_dtype int32).  Rows outside every group keep whatever
    ``out`` held (a new ``out`` starts uninitialised)."""
    codes = {torch.float32: F32, torch.bfloat16: BF16, torch.int32: I32}
    if out_dtype not in codes:
        raise ValueError("out_dtype must be bfloat16, float32 or int32")
    for t, name in ((a, "a"), (b, "b"), (a_offsets, "a_offsets"), (expert_ids, "expert_ids")):
        _require(t, name)
    if a.dtype != torch.int8 or b.dtype != torch.int8:
        raise TypeError("a and b must be int8")
    if a_offsets.dtype not in (torch.int32, torch.uint32) or expert_ids.dtype != torch.int32:
        raise TypeError("a_offsets must be uint32/int32 and expert_ids int32")
    if b.dim() != 3 or a.dim() != 2 or a.shape[1] != b.shape[2]:
        raise ValueError("b must be [E, N, K] and a [T, K]")
    e, n, k = b.shape
    t = a.shape[0]
    g = expert_ids.numel()
    if a_offsets.numel() != g + 1:
        raise ValueError("a_offsets needs num_groups + 1 entries")
    if out_dtype != torch.int32:
        if a_scale is None or b_scale is None:
            raise ValueError("a_scale and b_scale are needed for a dequantised output")
        for s_, name, size in ((a_scale, "a_scale", t), (b_scale, "b_scale", e * n)):
            _require(s_, name)
            if s_.dtype != torch.float32 or s_.numel() != size:
                raise ValueError(f"{name} must be float32 with {size} elements")
        if bias is not None:
            _require(bias, "bias")
            if bias.dtype != torch.bfloat16 or bias.numel() != e * n:
                raise ValueError(f"bias must be bfloat16 with {e * n} elements")
    if max_tokens_per_group is None:
        max_tokens_per_group = t
    out = _out(out, (t, n), out_dtype, a.device)
    opt = lambda x: None if x is None else _ptr(x)  # noqa: E731
    st = lib.qlinear_int8_grouped_gemm(_ptr(a), _ptr(b), opt(a_scale), opt(b_scale), opt(bias), _ptr(a_offsets),
                                       _ptr(expert_ids), _ptr(out), codes[out_dtype], g, int(max_tokens_per_group),
                                       e, t, n, k, _stream(a))
    _check(st, "qlinear_int8_grouped_gemm")
    return out



def _int4_operands(w_packed, w_scale, w_zero, x, group_size: int, lead: str):
    """The checked int4 operands (w, scale, zero pointer, x, K, group size); ``lead`` names
    the leading dimension of an expert stack ("" for one matrix).  The group size comes
    back as at most K, which means the same and fits the call's 64-bit argument."""
    w = _as_u8(w_packed, "w_packed")
    sc = _as_bf16(w_scale, "w_scale")
    x = _as_bf16(x, "x")
    for t, name in ((w, "w_packed"), (sc, "w_scale"), (x, "x")):
        _require(t, name)
    dims = 3 if lead else 2
    if w.dim() != dims or x.dim() != 2:
        raise ValueError(f"w_packed must be [{lead}N, (K + 1) / 2] and x [M, K]")
    k = x.shape[1]
    if not (group_size >= k or (group_size >= 32 and group_size & (group_size - 1) == 0)):
        raise ValueError("group_size must be a power of two >= 32, or at least K")
    groups = -(-k // group_size) if group_size > 0 else 0
    if w.shape[-1] != (k + 1) // 2 or tuple(sc.shape) != (*w.shape[:-1], groups):
        raise ValueError(f"w_packed must be [{lead}N, (K + 1) / 2] and w_scale [{lead}N, ceil(K / group_size)]")
    zero = None
    if w_zero is not None:
        _require(w_zero, "w_zero")
        if w_zero.dtype != torch.uint8 or w_zero.shape != sc.shape:
            raise ValueError("w_zero must be uint8 of w_scale's shape")
        zero = _ptr(w_zero)
    return w, sc, zero, x, k, min(int(group_size), k)


def int4_gemm(w_packed: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, w_zero: torch.Tensor | None = None,
              group_size: int = 128, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
              alpha: float = 1.0, row_scale: torch.Tensor | None = None, col_scale: torch.Tensor | None = None,
              bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
              activation: str = "none") -> torch.Tensor:
    """out[M, N] = alpha * x[M, K] @ D^T with D = (code - zero) * scale, 4-bit codes
    packed [N, (K + 1) / 2] (even k in the low nibble), one bfloat16 scale and one uint8
    zero point (None: 8) per ``group_size`` consecutive k (``qlinear_int4_gemm``);
    epilogue as ``fp8_gemm``."""
    w, sc, zero, x, k, group = _int4_operands(w_packed, w_scale, w_zero, x, group_size, "")
    m, n = x.shape[0], w.shape[0]
    out = _out(out, (m, n), out_dtype, x.device)
    d = _epilogue(m, n, row_scale, col_scale, bias, residual, activation) if m else None
    if m == 0:
        return out
    st = lib.qlinear_int4_gemm(_ptr(w), _ptr(sc), zero, _ptr(x), _ptr(out), _OUT_CODES[out_dtype], m, n, k,
                               group, float(alpha), _epi_ref(d), _stream(x))
    _check(st, "qlinear_int4_gemm")
    return out


def int4_grouped_gemm(w_packed: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, a_offsets: torch.Tensor,
                      expert_ids: torch.Tensor, w_zero: torch.Tensor | None = None, group_size: int = 128,
                      out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                      max_tokens_per_group: int | None = None) -> torch.Tensor:
    """Grouped MoE W4A16 with integer codes (``qlinear_int4_grouped_gemm``): rows
    a_offsets[z] .. a_offsets[z+1]-1 of x times D_e^T, e = expert_ids[z], D_e as in
    ``int4_gemm`` from the expert stack w_packed [E, N, (K + 1) / 2], w_scale and w_zero
    [E, N, ceil(K / group_size)].  Rows outside every group keep whatever ``out`` held
    (a new ``out`` starts uninitialised).  ``max_tokens_per_group`` is accepted as by the
    other grouped calls and does not change the launch."""
    w, sc, zero, x, k, group = _int4_operands(w_packed, w_scale, w_zero, x, group_size, "E, ")
    _require(a_offsets, "a_offsets")
    _require(expert_ids, "expert_ids")
    if a_offsets.dtype not in (torch.int32, torch.uint32) or expert_ids.dtype != torch.int32:
        raise TypeError("a_offsets must be uint32/int32 and expert_ids int32")
    g = expert_ids.numel()
    if a_offsets.numel() != g + 1:
        raise ValueError("a_offsets needs num_groups + 1 entries")
    e, n, _ = w.shape
    t = x.shape[0]
    if max_tokens_per_group is None:
        max_tokens_per_group = t
    out = _out(out, (t, n), out_dtype, x.device)
    if t == 0:
        return out
    st = lib.qlinear_int4_grouped_gemm(_ptr(w), _ptr(sc), zero, _ptr(x), _ptr(a_offsets), _ptr(expert_ids), _ptr(out),
                                       _OUT_CODES[out_dtype], g, int(max_tokens_per_group), e, t, n, k,
                                       group, _stream(x))
    _check(st, "qlinear_int4_grouped_gemm")
    return out


def _float_tensor(t: torch.Tensor, what: str, shape=None):
    _require(t, what)
    if t.dtype not in _OUT_CODES:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {tuple(shape)}, got {tuple(t.shape)}")


def _typed(t: torch.Tensor, what: str, dtype: torch.dtype, shape):
    _require(t, what)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True, expert_ids: torch.Tensor | None = None,
              weights: torch.Tensor | None = None):
    """The top_k experts of every token by logit, largest first, and their softmax
    weights, over the chosen experts (renormalize) or over all (``qlinear_moe_route``)
    -> (expert_ids int32 [T, top_k], weights f32 [T, top_k]).  A logit of -inf masks its
    expert; slots for which no expert is left get id -1 and weight 0."""
    _float_tensor(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    t, e = logits.shape
    expert_ids = _out(expert_ids, (t, top_k), torch.int32, logits.device)
    weights = _out(weights, (t, top_k), torch.float32, logits.device)
    if t == 0:
        return expert_ids, weights
    st = lib.qlinear_moe_route(_ptr(logits), _OUT_CODES[logits.dtype], _ptr(expert_ids), _ptr(weights), t, e,
                               int(top_k), int(bool(renormalize)), _stream(logits))
    _check(st, "qlinear_moe_route")
    return expert_ids, weights


def moe_route_backward(logits: torch.Tensor, expert_ids: torch.Tensor, grad_weights: torch.Tensor,
                       renormalize: bool = True, grad_logits: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``moe_route``'s weights with respect to the logits
    (``qlinear_moe_route_backward``), in the logits' dtype."""
    _float_tensor(logits, "logits")
    if logits.dim() != 2 or expert_ids.dim() != 2:
        raise ValueError("logits must be [T, E] and expert_ids [T, top_k]")
    t, e = logits.shape
    k = expert_ids.shape[1]
    _typed(expert_ids, "expert_ids", torch.int32, (t, k))
    _typed(grad_weights, "grad_weights", torch.float32, (t, k))
    grad_logits = _out(grad_logits, (t, e), logits.dtype, logits.device)
    if t == 0:
        return grad_logits
    st = lib.qlinear_moe_route_backward(_ptr(logits), _OUT_CODES[logits.dtype], _ptr(expert_ids), _ptr(grad_weights),
                                        _ptr(grad_logits), t, e, k, int(bool(renormalize)), _stream(logits))
    _check(st, "qlinear_moe_route_backward")
    return grad_logits


@functools.lru_cache(maxsize=256)
def _sort_workspace_bytes(slots: int, num_experts: int) -> int:
    """``qlinear_moe_sort_workspace_size``, a function of the sizes alone."""
    need = _i64(0)
    _check(lib.qlinear_moe_sort_workspace_size(slots, num_experts, ctypes.byref(need)), "qlinear_moe_sort_workspace_size")
    return need.value


def moe_sort(expert_ids: torch.Tensor, num_experts: int, workspace: torch.Tensor | None = None):
    """Stable sort of the slots of expert_ids [T, top_k] by expert (``qlinear_moe_sort``)
    -> (a_offsets int32 [num_experts + 1], row_slot int32 [T * top_k], slot_row int32
    [T, top_k]).  Rows a_offsets[e] .. a_offsets[e + 1] - 1 belong to expert e; slots with
    an id outside 0 .. num_experts - 1 are dropped: they fill the rows behind, and both
    maps hold the complement (~) for them.  ``workspace``: a device tensor of at least the
    bytes of ``qlinear_moe_sort_workspace_size`` (None: allocated)."""
    _require(expert_ids, "expert_ids")
    if expert_ids.dtype != torch.int32 or expert_ids.dim() != 2:
        raise TypeError("expert_ids must be int32 [T, top_k]")
    slots, dev = expert_ids.numel(), expert_ids.device
    need = _sort_workspace_bytes(slots, int(num_experts))
    offsets = torch.empty_strided((num_experts + 1,), (1,), dtype=torch.int32, device=dev)
    row_slot = torch.empty_strided((slots,), (1,), dtype=torch.int32, device=dev)
    slot_row = _out(None, expert_ids.shape, torch.int32, dev)
    if slots == 0:
        return offsets.zero_(), row_slot, slot_row
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    nbytes = 0
    if workspace is not None:
        _require(workspace, "workspace")
        nbytes = workspace.numel() * workspace.element_size()
    st = lib.qlinear_moe_sort(_ptr(expert_ids), _ptr(offsets), _ptr(row_slot), _ptr(slot_row), slots, int(num_experts),
                              None if workspace is None else _ptr(workspace), nbytes, _stream(expert_ids))
    _check(st, "qlinear_moe_sort")
    return offsets, row_slot, slot_row


def moe_gather(x: torch.Tensor, slot_row: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Token rows x [T, H] into expert order, [T * top_k, H] (``qlinear_moe_gather``): row
    slot_row[t, j] is token t; the rows of dropped slots are zeros.  Its gradient is
    ``moe_combine`` without weights."""
    _float_tensor(x, "x")
    if x.dim() != 2 or slot_row.dim() != 2:
        raise ValueError("x must be [T, H] and slot_row [T, top_k]")
    t, h = x.shape
    k = slot_row.shape[1]
    _typed(slot_row, "slot_row", torch.int32, (t, k))
    out = _out(out, (t * k, h), x.dtype, x.device)
    if t == 0:
        return out
    st = lib.qlinear_moe_gather(_ptr(x), _ptr(slot_row), _ptr(out), _OUT_CODES[x.dtype], t, k, h, _stream(x))
    _check(st, "qlinear_moe_gather")
    return out


def moe_combine(rows: torch.Tensor, slot_row: torch.Tensor, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Rows in expert order [T * top_k, H] back to tokens [T, H], summed with the router's
    weights (None: all 1) over the slots that were not dropped (``qlinear_moe_combine``);
    out_dtype defaults to the rows' dtype."""
    _float_tensor(rows, "rows")
    if rows.dim() != 2 or slot_row.dim() != 2:
        raise ValueError("rows must be [T * top_k, H] and slot_row [T, top_k]")
    t, k = slot_row.shape
    _typed(slot_row, "slot_row", torch.int32, (t, k))
    h = rows.shape[1]
    _float_tensor(rows, "rows", (t * k, h))
    if weights is not None:
        _typed(weights, "weights", torch.float32, (t, k))
    out_dtype = rows.dtype if out_dtype is None else out_dtype
    if out_dtype not in _OUT_CODES:
        raise TypeError("out_dtype must be float32 or bfloat16")
    out = _out(out, (t, h), out_dtype, rows.device)
    if t == 0:
        return out
    st = lib.qlinear_moe_combine(_ptr(rows), _OUT_CODES[rows.dtype], _ptr(slot_row),
                                 None if weights is None else _ptr(weights), _ptr(out), _OUT_CODES[out_dtype], t, k, h,
                                 _stream(rows))
    _check(st, "qlinear_moe_combine")
    return out


def moe_combine_backward(grad_out: torch.Tensor, rows: torch.Tensor, slot_row: torch.Tensor, weights: torch.Tensor,
                         grad_rows: torch.Tensor | None = None, grad_weights: torch.Tensor | None = None):
    """Gradients of ``moe_combine`` (``qlinear_moe_combine_backward``) -> (grad_rows
    [T * top_k, H] in the rows' dtype, grad_weights f32 [T, top_k])."""
    _float_tensor(grad_out, "grad_out")
    if grad_out.dim() != 2 or slot_row.dim() != 2:
        raise ValueError("grad_out must be [T, H] and slot_row [T, top_k]")
    t, h = grad_out.shape
    k = slot_row.shape[1]
    _typed(slot_row, "slot_row", torch.int32, (t, k))
    _typed(rows, "rows", grad_out.dtype, (t * k, h))
    _typed(weights, "weights", torch.float32, (t, k))
    grad_rows = _out(grad_rows, (t * k, h), rows.dtype, rows.device)
    grad_weights = _out(grad_weights, (t, k), torch.float32, rows.device)
    if t == 0:
        return grad_rows, grad_weights
    st = lib.qlinear_moe_combine_backward(_ptr(grad_out), _ptr(rows), _OUT_CODES[rows.dtype], _ptr(slot_row),
                                          _ptr(weights), _ptr(grad_rows), _ptr(grad_weights), t, k, h, _stream(rows))
    _check(st, "qlinear_moe_combine_backward")
    return grad_rows, grad_weights


def swiglu(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """silu(x[:, :F]) * x[:, F:] of x [M, 2F] (``qlinear_swiglu``)."""
    _float_tensor(x, "x")
    if x.dim() != 2 or x.shape[1] % 2 != 0:
        raise ValueError("x must be [M, 2F]")
    m, f = x.shape[0], x.shape[1] // 2
    out = _out(out, (m, f), x.dtype, x.device)
    if m == 0:
        return out
    st = lib.qlinear_swiglu(_ptr(x), _ptr(out), _OUT_CODES[x.dtype], m, f, _stream(x))
    _check(st, "qlinear_swiglu")
    return out


def swiglu_backward(grad_y: torch.Tensor, x: torch.Tensor, grad_x: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of ``swiglu`` with respect to x [M, 2F] (``qlinear_swiglu_backward``)."""
    _float_tensor(x, "x")
    if x.dim() != 2 or x.shape[1] % 2 != 0:
        raise ValueError("x must be [M, 2F]")
    m, f = x.shape[0], x.shape[1] // 2
    _typed(grad_y, "grad_y", x.dtype, (m, f))
    grad_x = _out(grad_x, (m, 2 * f), x.dtype, x.device)
    if m == 0:
        return grad_x
    st = lib.qlinear_swiglu_backward(_ptr(grad_y), _ptr(x), _ptr(grad_x), _OUT_CODES[x.dtype], m, f, _stream(x))
    _check(st, "qlinear_swiglu_backward")
    return grad_x
