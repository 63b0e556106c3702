"""libfp8w: FP8 (e4m3fn) weights for the decode path on MI355X (gfx950).

A thin ctypes binding over the C ABI of ``include/fp8w.h``.  Every function
here only checks and marshals arguments; all arithmetic runs in the HIP
kernels of ``libfp8w.so``.  PyTorch supplies device memory and the stream.
There is no CPU fallback: importing works on any host (so the symbol table
can be checked), but every call needs a ROCm GPU and the built library, and
fails loudly otherwise.

Functions carry the names of the C entry points:

* ``fp8w_quantize_block(w) -> (codes, scales)``   bf16 [n,k] -> u8 [n,k], f32 grid
* ``fp8w_quantize_mx(w) -> (codes, e8m0)``        bf16 [n,k] -> u8 [n,k], u8 [n,ceil(k/32)]
* ``fp8w_gemv_block(x, codes, scales) -> y``      bf16 [m,k] -> bf16 [m,n]
* ``fp8w_gemv_mx(x, codes, e8m0) -> y``
* ``fp8w_grouped_plan_init(xs, codes, scales) -> plan`` and
  ``fp8w_gemv_grouped(plan) -> ys``: many independent GEMVs in one launch
* ``fp8w_dequantize_block(codes, scales) -> w`` / ``fp8w_dequantize_mx``: bf16 [n,k]
* ``fp8w_gemm_block(x, codes, scales) -> y`` / ``fp8w_gemm_mx``: any m, through
  dequantize + a dense bf16 GEMM (the large-M route)
* ``fp8w_quantize_act(x) -> (x_codes, x_scale)`` and
  ``fp8w_gemv_block_w8a8(x_codes, x_scale, codes, scales) -> y`` / ``_mx_w8a8``:
  the W8A8 route (per-tensor fp8 activation, fp8 x fp8 matrix cores)
* ``fp8w_route_experts(logits, top_k) -> ExpertRouting``: the experts of each
  token, their weights, and the tokens sorted by expert
* ``fp8w_gemm_experts(x, codes, scales, offsets, rows) -> y``: products grouped
  by expert on fp8 weights [E,n,k], plain or with a gated SiLU, and
  ``fp8w_combine_experts(y, weights, slots) -> out``: the weighted sum of each
  token's experts
* ``fp8w_logprobs(logits, targets, top) -> Logprobs``: log probabilities of
  given tokens, entropy and top alternatives

plus ``Fp8Experts``, the fp8 weights of a layer's experts, and ``Fp8Weight``,
a format-tagged weight whose GEMV asserts the format before dispatch (a scale
buffer of the wrong format cannot be detected by a kernel: "quantize_fp8_bs.rs", Atlas weight_map, module notes).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import NamedTuple, Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8w.so")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED, ERR_OVERLAP, ERR_HIP, ERR_CAPTURE = range(8)
ROUTE_AUTO, ROUTE_VALU, ROUTE_MFMA = 0, 1, 2
MAX_M = 32
TILE = 128
MX_GROUP = 32

# name -> (restype, argtypes); the exported C ABI, mirrored from include/fp8w.h
_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
SIGNATURES = {
    "fp8w_scale_bytes": (_I64, [_I, _I64, _I64]),
    "fp8w_gemv_auto_route": (_I, [_I, _I64, _I64, _I64]),
    "fp8w_quantize": (_I, [_P, _I64, _I64, _I, _P, _P, _P, _I64, _P]),
    "fp8w_dequantize": (_I, [_P, _P, _I, _I64, _I64, _P, _P]),
    "fp8w_gemv": (_I, [_P, _I64, _P, _P, _I, _I64, _I64, _P, _I, _P]),
    "fp8w_gemm": (_I, [_P, _I64, _P, _P, _I, _I64, _I64, _P, _P, _I64, _P]),
    "fp8w_gemv_w8a8": (_I, [_P, _P, _I64, _P, _P, _I, _I64, _I64, _P, _P]),
    "fp8w_quantize_block": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "fp8w_quantize_mx": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "fp8w_gemv_block": (_I, [_P, _I64, _P, _P, _I64, _I64, _P, _P]),
    "fp8w_gemv_mx": (_I, [_P, _I64, _P, _P, _I64, _I64, _P, _P]),
    "fp8w_gemv_block_route": (_I, [_P, _I64, _P, _P, _I64, _I64, _P, _I, _P]),
    "fp8w_gemv_mx_route": (_I, [_P, _I64, _P, _P, _I64, _I64, _P, _I, _P]),
    "fp8w_dequantize_block": (_I, [_P, _P, _I64, _I64, _P, _P]),
    "fp8w_dequantize_mx": (_I, [_P, _P, _I64, _I64, _P, _P]),
    "fp8w_gemm_workspace_bytes": (_I64, [_I64, _I64]),
    "fp8w_gemm_prepare": (_I, []),
    "fp8w_gemm_block": (_I, [_P, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _P]),
    "fp8w_gemm_mx": (_I, [_P, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _P]),
    "fp8w_quantize_act_workspace_bytes": (_I64, []),
    "fp8w_quantize_act": (_I, [_P, _I64, _I64, _P, _P, _P, _I64, _P]),
    "fp8w_quantize_act_noalloc": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "fp8w_gemv_block_w8a8": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _P, _P]),
    "fp8w_gemv_mx_w8a8": (_I, [_P, _P, _I64, _P, _P, _I64, _I64, _P, _P]),
    "fp8w_read_ceiling": (_I, [_P, _I64, _P, _I64, _P]),
    "fp8w_grouped_table_bytes": (_I64, [_I64]),
    "fp8w_grouped_plan_init": (_I, [_P, _I64, _I64, _I, _I, _P, _P]),
    "fp8w_gemv_grouped": (_I, [_P, _P]),
    "fp8w_quant_table_bytes": (_I64, [_I64]),
    "fp8w_quant_plan_init": (_I, [_P, _I64, _I, _P, _P]),
    "fp8w_quantize_grouped": (_I, [_P, _P]),
    "fp8w_route_experts_workspace_bytes": (_I64, [_I64, _I64]),
    "fp8w_route_experts": (_I, [_P, _I, _I64, _I64, _I64, _I64, _I, _P, _I, ctypes.c_float, _P, _P, _P, _P, _P,
                                _P, _I64, _P]),
    "fp8w_gemm_experts": (_I, [_P, _I64, _P, _P, _I64, _I64, _P, _P, _I, _I64, _I64, _I, _P, _P]),
    "fp8w_combine_experts": (_I, [_P, _I64, _P, _P, _I64, _I64, _I64, _P, _P]),
    "fp8w_logprobs_workspace_bytes": (_I64, [_I64, _I64, _I64]),
    "fp8w_logprobs": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P, _I64, _P]),
    "fp8w_block_scale_count": (_I64, [_I64, _I64]),
    "fp8w_mx_scale_count": (_I64, [_I64, _I64]),
    "fp8w_status_string": (ctypes.c_char_p, [_I]),
    "fp8w_version": (_I, []),
}

FORMAT_BLOCK, FORMAT_MX, FORMAT_BLOCK_BF16, FORMAT_ROW, FORMAT_TENSOR = 0, 1, 2, 3, 4
FORMAT_IDS = {"block": FORMAT_BLOCK, "mx": FORMAT_MX, "block_bf16": FORMAT_BLOCK_BF16,
              "row": FORMAT_ROW, "tensor": FORMAT_TENSOR}


class GemvDesc(ctypes.Structure):
    """fp8w_gemv_desc of include/fp8w.h."""
    _fields_ = [("x", _P), ("codes", _P), ("scales", _P), ("y", _P),
                ("n", _I64), ("k", _I64)]


class GroupedPlanC(ctypes.Structure):
    """fp8w_grouped_plan of include/fp8w.h."""
    _fields_ = [("table", _P), ("count", ctypes.c_int32), ("m", ctypes.c_int32),
                ("format", ctypes.c_int32), ("route", ctypes.c_int32), ("blocks", _I64),
                ("tiles", _I64), ("tiles_per_block", ctypes.c_int32), ("seg_cols", ctypes.c_int32),
                ("mx_packed8", ctypes.c_int32)]


class QuantDesc(ctypes.Structure):
    """fp8w_quant_desc of include/fp8w.h."""
    _fields_ = [("w", _P), ("codes", _P), ("scales", _P), ("n", _I64), ("k", _I64)]


class QuantPlanC(ctypes.Structure):
    """fp8w_quant_plan of include/fp8w.h."""
    _fields_ = [("table", _P), ("count", ctypes.c_int32), ("format", ctypes.c_int32), ("blocks", _I64)]


_lib = None


class Fp8wError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """Load ``libfp8w.so`` (built by ``__graft_entry__.build()``), or raise."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m fp8_block_scaled_02_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype, fn.argtypes = res, args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().fp8w_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise Fp8wError(status, what)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _current_handle() -> int:
    """The current stream's handle, without the Stream object (0.3 us, not 2.7)."""
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        return _current_handle()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _record(stream, handle: int, used) -> None:
    """Tensors recorded on a stream (a Stream, a handle, or None for the
    current one): their memory is not handed out again before what the stream
    was given until then has run."""
    cuda = _torch().cuda
    if stream is None:
        stream = cuda.current_stream()
    elif not isinstance(stream, cuda.Stream):   # 0 would make an ExternalStream one of the pool's
        stream = cuda.ExternalStream(handle) if handle else cuda.default_stream()
    for t in used:
        if t is not None:
            t.record_stream(stream)


def _launch_stream(stream, *used):
    """The handle of the stream a call goes to.  The call's outputs and
    workspaces belong to the stream they were made on, the current one as a
    rule: used on another, they are recorded there."""
    handle = _current_handle()
    if stream is None:
        return handle
    current, handle = handle, _stream_handle(stream)
    if handle != current:
        _record(stream, handle, used)
    return handle


def _table(nbytes: int, device):
    """Device memory for a plan's table, which the set-up call writes at once,
    not in a stream's order: what the current stream may still do with the
    memory it is made of comes first."""
    torch = _torch()
    table = torch.empty(nbytes, dtype=torch.uint8, device=device)
    torch.cuda.current_stream().synchronize()
    return table


def _plan_stream(plan, stream, *used):
    """The same for a plan, whose table and outputs were made some time ago,
    under any stream: recorded on each stream that the plan is used on, once,
    since a recording lasts until the memory is freed.  A plan may then be
    dropped behind its call."""
    handle = _stream_handle(stream)
    if handle not in plan.streams:
        _record(stream, handle, (plan.table, *used))
        plan.streams.add(handle)
    return handle


def _require(t, dtypes, what: str, dims: int):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what}: must be a GPU tensor (libfp8w has no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype} not in {dtypes}")
    if t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dims}-d tensor")
    return t


def _bf16_like(torch):
    return (torch.bfloat16, torch.int16, torch.uint16)


def block_scale_shape(n: int, k: int):
    return ((n + TILE - 1) // TILE, (k + TILE - 1) // TILE)


def mx_scale_shape(n: int, k: int):
    return (n, (k + MX_GROUP - 1) // MX_GROUP)


def scale_shape(fmt: str, n: int, k: int):
    """Shape of the scale buffer of an [n, k] weight in format ``fmt``."""
    if fmt in ("block", "block_bf16"):
        return block_scale_shape(n, k)
    if fmt == "mx":
        return mx_scale_shape(n, k)
    return {"row": (n,), "tensor": (1,)}[fmt]


def _scale_dtype(torch, fmt: str):
    return {"block": torch.float32, "mx": torch.uint8, "block_bf16": torch.bfloat16,
            "row": torch.float32, "tensor": torch.float32}[fmt]


def _format_id(fmt: str) -> int:
    if fmt not in FORMAT_IDS:
        raise ValueError(f"unknown scale format {fmt!r}")
    return FORMAT_IDS[fmt]


def _check_scales(torch, fmt, scales, n, k, what):
    _require(scales, (_scale_dtype(torch, fmt),), "scales", len(scale_shape(fmt, n, k)))
    if tuple(scales.shape) != scale_shape(fmt, n, k):
        raise ValueError(f"{what}: {fmt} scales must be {scale_shape(fmt, n, k)}, got {tuple(scales.shape)}")


# --------------------------------------------------------------- quantize --

def fp8w_quantize(w, fmt: str = "block", codes=None, scales=None, workspace=None, stream=None):
    """bf16 W [n,k] -> (e4m3 codes u8 [n,k], scales in format ``fmt``)."""
    torch = _torch()
    _require(w, _bf16_like(torch), "w", 2)
    n, k = w.shape
    fid = _format_id(fmt)
    if codes is None:
        codes = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(scale_shape(fmt, n, k), dtype=_scale_dtype(torch, fmt), device=w.device)
    if workspace is None and fmt == "tensor":
        workspace = torch.empty(int(lib().fp8w_quantize_act_workspace_bytes()), dtype=torch.uint8,
                                device=w.device)
    _require(codes, (torch.uint8,), "codes", 2)
    _check_scales(torch, fmt, scales, n, k, "fp8w_quantize")
    ws_ptr, ws_n = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
    _check(lib().fp8w_quantize(w.data_ptr(), n, k, fid, codes.data_ptr(), scales.data_ptr(), ws_ptr,
                               ws_n, _launch_stream(stream, codes, scales, workspace)), "fp8w_quantize")
    return codes, scales


def fp8w_dequantize(codes, scales, fmt: str = "block", w=None, stream=None):
    torch = _torch()
    _require(codes, (torch.uint8,), "codes", 2)
    n, k = codes.shape
    _check_scales(torch, fmt, scales, n, k, "fp8w_dequantize")
    if w is None:
        w = torch.empty((n, k), dtype=torch.bfloat16, device=codes.device)
    _require(w, _bf16_like(torch), "w", 2)
    _check(lib().fp8w_dequantize(codes.data_ptr(), scales.data_ptr(), _format_id(fmt), n, k,
                                 w.data_ptr(), _launch_stream(stream, w)), "fp8w_dequantize")
    return w


def fp8w_gemv(x, codes, scales, fmt: str = "block", y=None, route=0, stream=None):
    torch = _torch()
    _require(x, _bf16_like(torch), "x", 2)
    _require(codes, (torch.uint8,), "codes", 2)
    m, k = x.shape
    n = codes.shape[0]
    _check_scales(torch, fmt, scales, n, k, "fp8w_gemv")
    if y is None:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _require(y, _bf16_like(torch), "y", 2)
    _check(lib().fp8w_gemv(x.data_ptr(), m, codes.data_ptr(), scales.data_ptr(), _format_id(fmt), n,
                           k, y.data_ptr(), int(route), _launch_stream(stream, y)), "fp8w_gemv")
    return y


def fp8w_gemv_auto_route(m: int, n: int, k: int, fmt: str = "block") -> int:
    """The kernel family AUTO takes for a single GEMV of m activation rows on an
    [n, k] weight with `fmt` scales: ROUTE_VALU or ROUTE_MFMA (ROUTE_AUTO when
    out of range)."""
    return int(lib().fp8w_gemv_auto_route(_format_id(fmt), int(m), int(n), int(k)))


def fp8w_gemm(x, codes, scales, fmt: str = "block", y=None, workspace=None, stream=None):
    torch = _torch()
    _require(x, _bf16_like(torch), "x", 2)
    _require(codes, (torch.uint8,), "codes", 2)
    m, k = x.shape
    n = codes.shape[0]
    _check_scales(torch, fmt, scales, n, k, "fp8w_gemm")
    if y is None:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(int(lib().fp8w_gemm_workspace_bytes(n, k)), dtype=torch.uint8,
                                device=x.device)
    _require(y, _bf16_like(torch), "y", 2)
    _check(lib().fp8w_gemm(x.data_ptr(), m, codes.data_ptr(), scales.data_ptr(), _format_id(fmt), n, k,
                           y.data_ptr(), workspace.data_ptr(), workspace.numel(), _launch_stream(stream, y, workspace)),
           "fp8w_gemm")
    return y


def fp8w_gemv_w8a8(x_codes, x_scale, codes, scales, fmt: str = "block", y=None, stream=None):
    torch = _torch()
    _require(x_codes, (torch.uint8,), "x_codes", 2)
    _require(x_scale, (torch.float32,), "x_scale", 1)
    _require(codes, (torch.uint8,), "codes", 2)
    m, k = x_codes.shape
    n = codes.shape[0]
    _check_scales(torch, fmt, scales, n, k, "fp8w_gemv_w8a8")
    if y is None:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=codes.device)
    _require(y, _bf16_like(torch), "y", 2)
    _check(lib().fp8w_gemv_w8a8(x_codes.data_ptr(), x_scale.data_ptr(), m, codes.data_ptr(),
                                scales.data_ptr(), _format_id(fmt), n, k, y.data_ptr(),
                                _launch_stream(stream, y)), "fp8w_gemv_w8a8")
    return y



def fp8w_quantize_block(w, codes=None, scales=None, stream=None):
    """bf16 W [n,k] -> (e4m3fn codes u8 [n,k], fp32 scales [ceil(n/128), ceil(k/128)])."""
    torch = _torch()
    _require(w, _bf16_like(torch), "w", 2)
    n, k = w.shape
    if codes is None:
        codes = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(block_scale_shape(n, k), dtype=torch.float32, device=w.device)
    _require(codes, (torch.uint8,), "codes", 2)
    _require(scales, (torch.float32,), "scales", 2)
    if tuple(codes.shape) != (n, k) or tuple(scales.shape) != block_scale_shape(n, k):
        raise ValueError("fp8w_quantize_block: output shapes do not match w")
    _check(lib().fp8w_quantize_block(w.data_ptr(), n, k, codes.data_ptr(), scales.data_ptr(),
                                     _launch_stream(stream, codes, scales)), "fp8w_quantize_block")
    return codes, scales


def fp8w_quantize_mx(w, codes=None, e8m0=None, stream=None):
    """bf16 W [n,k] -> (e4m3fn codes u8 [n,k], e8m0 u8 [n, ceil(k/32)])."""
    torch = _torch()
    _require(w, _bf16_like(torch), "w", 2)
    n, k = w.shape
    if codes is None:
        codes = torch.empty((n, k), dtype=torch.uint8, device=w.device)
    if e8m0 is None:
        e8m0 = torch.empty(mx_scale_shape(n, k), dtype=torch.uint8, device=w.device)
    _require(codes, (torch.uint8,), "codes", 2)
    _require(e8m0, (torch.uint8,), "e8m0", 2)
    if tuple(codes.shape) != (n, k) or tuple(e8m0.shape) != mx_scale_shape(n, k):
        raise ValueError("fp8w_quantize_mx: output shapes do not match w")
    _check(lib().fp8w_quantize_mx(w.data_ptr(), n, k, codes.data_ptr(), e8m0.data_ptr(),
                                  _launch_stream(stream, codes, e8m0)), "fp8w_quantize_mx")
    return codes, e8m0


# ------------------------------------------------------------------- GEMV --

def _gemv(fn_name, x, codes, scale_t, scale_shape, scale_dtype, y, route, stream):
    torch = _torch()
    _require(x, _bf16_like(torch), "x", 2)
    _require(codes, (torch.uint8,), "codes", 2)
    _require(scale_t, (scale_dtype,), "scales", 2)
    m, k = x.shape
    n, k2 = codes.shape
    if k != k2:
        raise ValueError(f"{fn_name}: x has K={k}, codes have K={k2}")
    if tuple(scale_t.shape) != scale_shape(n, k):
        raise ValueError(f"{fn_name}: scale grid {tuple(scale_t.shape)} != {scale_shape(n, k)}")
    if y is None:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _require(y, _bf16_like(torch), "y", 2)
    if tuple(y.shape) != (m, n):
        raise ValueError(f"{fn_name}: y must be [{m}, {n}]")
    fn = getattr(lib(), fn_name + "_route")
    _check(fn(x.data_ptr(), m, codes.data_ptr(), scale_t.data_ptr(), n, k, y.data_ptr(),
              int(route), _launch_stream(stream, y)), fn_name)
    return y


def fp8w_gemv_block(x, codes, scales, y=None, route=ROUTE_AUTO, stream=None):
    """y[m,n] = x[m,k] . deq(W)^T with 128x128 fp32 block scales (bf16 out)."""
    torch = _torch()
    return _gemv("fp8w_gemv_block", x, codes, scales, block_scale_shape, torch.float32, y,
                 route, stream)


def fp8w_gemv_mx(x, codes, e8m0, y=None, route=ROUTE_AUTO, stream=None):
    """y[m,n] = x[m,k] . deq(W)^T with per-32 e8m0 scales (bf16 out)."""
    torch = _torch()
    return _gemv("fp8w_gemv_mx", x, codes, e8m0, mx_scale_shape, torch.uint8, y, route, stream)


# ------------------------------------------------------------- dequantize --

def _dequantize(fn_name, codes, scale_t, scale_shape, scale_dtype, w, stream):
    torch = _torch()
    _require(codes, (torch.uint8,), "codes", 2)
    _require(scale_t, (scale_dtype,), "scales", 2)
    n, k = codes.shape
    if tuple(scale_t.shape) != scale_shape(n, k):
        raise ValueError(f"{fn_name}: scale grid {tuple(scale_t.shape)} != {scale_shape(n, k)}")
    if w is None:
        w = torch.empty((n, k), dtype=torch.bfloat16, device=codes.device)
    _require(w, _bf16_like(torch), "w", 2)
    if tuple(w.shape) != (n, k):
        raise ValueError(f"{fn_name}: w must be [{n}, {k}]")
    _check(getattr(lib(), fn_name)(codes.data_ptr(), scale_t.data_ptr(), n, k, w.data_ptr(),
                                   _launch_stream(stream, w)), fn_name)
    return w


def fp8w_dequantize_block(codes, scales, w=None, stream=None):
    """bf16 W [n,k] = fl32(dec(codes) * block scale), rounded to bf16."""
    torch = _torch()
    return _dequantize("fp8w_dequantize_block", codes, scales, block_scale_shape, torch.float32, w, stream)


def fp8w_dequantize_mx(codes, e8m0, w=None, stream=None):
    """bf16 W [n,k] = dec(codes) * 2^(e8m0 - 127), rounded to bf16."""
    torch = _torch()
    return _dequantize("fp8w_dequantize_mx", codes, e8m0, mx_scale_shape, torch.uint8, w, stream)


# ------------------------------------------------------------------- GEMM --

def _gemm(fn_name, x, codes, scale_t, scale_shape, scale_dtype, y, workspace, stream):
    torch = _torch()
    _require(x, _bf16_like(torch), "x", 2)
    _require(codes, (torch.uint8,), "codes", 2)
    _require(scale_t, (scale_dtype,), "scales", 2)
    m, k = x.shape
    n, k2 = codes.shape
    if k != k2:
        raise ValueError(f"{fn_name}: x has K={k}, codes have K={k2}")
    if tuple(scale_t.shape) != scale_shape(n, k):
        raise ValueError(f"{fn_name}: scale grid {tuple(scale_t.shape)} != {scale_shape(n, k)}")
    if y is None:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _require(y, _bf16_like(torch), "y", 2)
    if tuple(y.shape) != (m, n):
        raise ValueError(f"{fn_name}: y must be [{m}, {n}]")
    nbytes = int(lib().fp8w_gemm_workspace_bytes(n, k))
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    _require(workspace, (torch.uint8,), "workspace", 1)
    _check(getattr(lib(), fn_name)(x.data_ptr(), m, codes.data_ptr(), scale_t.data_ptr(), n, k,
                                   y.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                   _launch_stream(stream, y, workspace)), fn_name)
    return y


def fp8w_gemm_block(x, codes, scales, y=None, workspace=None, stream=None):
    """y[m,n] = x[m,k] . deq(W)^T for any m: dequantize into ``workspace``
    (u8, fp8w_gemm_workspace_bytes(n, k) bytes; allocated when None), then a
    dense bf16 GEMM."""
    torch = _torch()
    return _gemm("fp8w_gemm_block", x, codes, scales, block_scale_shape, torch.float32, y,
                 workspace, stream)


def fp8w_gemm_mx(x, codes, e8m0, y=None, workspace=None, stream=None):
    torch = _torch()
    return _gemm("fp8w_gemm_mx", x, codes, e8m0, mx_scale_shape, torch.uint8, y, workspace, stream)


def fp8w_gemm_prepare() -> None:
    """Create the current device's rocBLAS handle for the GEMM calls (outside
    stream capture), so that GEMM calls can then be captured in a graph."""
    _check(lib().fp8w_gemm_prepare(), "fp8w_gemm_prepare")


# ------------------------------------------------------------------- W8A8 --

def fp8w_read_ceiling(buf, out=None, stream=None):
    """Read every byte of the contiguous GPU tensor ``buf`` once (measurement
    aid: the practical HBM read ceiling); returns the per-workgroup XOR words
    (2048 int32 by default), whose XOR is the XOR of the buffer's dwords."""
    torch = _torch()
    if not isinstance(buf, torch.Tensor) or buf.device.type != "cuda" or not buf.is_contiguous():
        raise ValueError("fp8w_read_ceiling: buf must be a contiguous GPU tensor")
    if out is None:
        out = torch.empty(2048, dtype=torch.int32, device=buf.device)
    _require(out, (torch.int32,), "out", 1)
    _check(lib().fp8w_read_ceiling(buf.data_ptr(), buf.numel() * buf.element_size(), out.data_ptr(),
                                   out.numel(), _launch_stream(stream, out)), "fp8w_read_ceiling")
    return out


def fp8w_quantize_act(x, codes=None, scale=None, workspace=None, stream=None):
    """Per-tensor activation quantization: bf16 x [m,k] -> (e4m3 codes u8
    [m,k], fp32 scale [1] on the device)."""
    torch = _torch()
    _require(x, _bf16_like(torch), "x", 2)
    m, k = x.shape
    if codes is None:
        codes = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(int(lib().fp8w_quantize_act_workspace_bytes()), dtype=torch.uint8,
                                device=x.device)
    _require(codes, (torch.uint8,), "codes", 2)
    _require(scale, (torch.float32,), "scale", 1)
    _require(workspace, (torch.uint8,), "workspace", 1)
    if tuple(codes.shape) != (m, k) or scale.numel() != 1:
        raise ValueError("fp8w_quantize_act: codes must be [m, k] and scale one element")
    _check(lib().fp8w_quantize_act(x.data_ptr(), m, k, codes.data_ptr(), scale.data_ptr(),
                                   workspace.data_ptr(), workspace.numel(),
                                   _launch_stream(stream, codes, scale, workspace)), "fp8w_quantize_act")
    return codes, scale


def fp8w_quantize_act_noalloc(x, codes, scale, stream=None):
    """fp8w_quantize_act with its partial maxima in the library's own device
    array: no workspace and no allocation.  The outputs are the caller's
    (codes u8 [m,k], scale fp32 [1])."""
    torch = _torch()
    _require(x, _bf16_like(torch), "x", 2)
    _require(codes, (torch.uint8,), "codes", 2)
    _require(scale, (torch.float32,), "scale", 1)
    m, k = x.shape
    if tuple(codes.shape) != (m, k) or scale.numel() != 1:
        raise ValueError("fp8w_quantize_act_noalloc: codes must be [m, k] and scale one element")
    _check(lib().fp8w_quantize_act_noalloc(x.data_ptr(), m, k, codes.data_ptr(), scale.data_ptr(),
                                           _stream_handle(stream)), "fp8w_quantize_act_noalloc")
    return codes, scale


def _gemv_w8a8(fn_name, x_codes, x_scale, codes, scale_t, scale_shape, scale_dtype, y, stream):
    torch = _torch()
    _require(x_codes, (torch.uint8,), "x_codes", 2)
    _require(x_scale, (torch.float32,), "x_scale", 1)
    _require(codes, (torch.uint8,), "codes", 2)
    _require(scale_t, (scale_dtype,), "scales", 2)
    m, k = x_codes.shape
    n, k2 = codes.shape
    if k != k2:
        raise ValueError(f"{fn_name}: x has K={k}, codes have K={k2}")
    if tuple(scale_t.shape) != scale_shape(n, k):
        raise ValueError(f"{fn_name}: scale grid {tuple(scale_t.shape)} != {scale_shape(n, k)}")
    if y is None:
        y = torch.empty((m, n), dtype=torch.bfloat16, device=codes.device)
    _require(y, _bf16_like(torch), "y", 2)
    _check(getattr(lib(), fn_name)(x_codes.data_ptr(), x_scale.data_ptr(), m, codes.data_ptr(),
                                   scale_t.data_ptr(), n, k, y.data_ptr(), _launch_stream(stream, y)),
           fn_name)
    return y


def fp8w_gemv_block_w8a8(x_codes, x_scale, codes, scales, y=None, stream=None):
    """y = x_scale * dec(x_codes) . deq(W)^T with fp8 x fp8 matrix cores."""
    torch = _torch()
    return _gemv_w8a8("fp8w_gemv_block_w8a8", x_codes, x_scale, codes, scales, block_scale_shape,
                      torch.float32, y, stream)


def fp8w_gemv_mx_w8a8(x_codes, x_scale, codes, e8m0, y=None, stream=None):
    torch = _torch()
    return _gemv_w8a8("fp8w_gemv_mx_w8a8", x_codes, x_scale, codes, e8m0, mx_scale_shape,
                      torch.uint8, y, stream)


# ---------------------------------------------------------------- grouped --

class GroupedPlan:
    """A group of independent GEMVs launched as one kernel.

    Holds the device table and references to every buffer it names, so the
    buffers stay alive as long as the plan.  ``y`` tensors are allocated here
    when not given.
    """

    def __init__(self, xs, codes, scales, ys=None, fmt: str = "block", route=ROUTE_AUTO):
        torch = _torch()
        if not (len(xs) == len(codes) == len(scales)) or not xs:
            raise ValueError("xs, codes and scales must be non-empty lists of equal length")
        fmt_id = _format_id(fmt)
        sdt, sshape = _scale_dtype(torch, fmt), (lambda n, k: scale_shape(fmt, n, k))
        m = int(xs[0].shape[0])
        if ys is None:
            ys = [torch.empty((m, int(c.shape[0])), dtype=torch.bfloat16, device=c.device) for c in codes]
        descs = (GemvDesc * len(xs))()
        for i, (x, c, s, y) in enumerate(zip(xs, codes, scales, ys)):
            _require(x, _bf16_like(torch), "x", 2)
            _require(c, (torch.uint8,), "codes", 2)
            _require(s, (sdt,), "scales", len(sshape(1, 16)))
            _require(y, _bf16_like(torch), "y", 2)
            n, k = c.shape
            if x.shape[0] != m or x.shape[1] != k or tuple(s.shape) != sshape(n, k) \
                    or tuple(y.shape) != (m, n):
                raise ValueError(f"grouped GEMV {i}: inconsistent shapes")
            descs[i] = GemvDesc(x.data_ptr(), c.data_ptr(), s.data_ptr(), y.data_ptr(), n, k)
        nbytes = int(lib().fp8w_grouped_table_bytes(len(xs)))
        self.table = _table(nbytes, codes[0].device)
        self.plan = GroupedPlanC()
        _check(lib().fp8w_grouped_plan_init(descs, len(xs), m, fmt_id, int(route),
                                            self.table.data_ptr(), ctypes.byref(self.plan)),
               "fp8w_grouped_plan_init")
        self.xs, self.codes, self.scales, self.ys = list(xs), list(codes), list(scales), list(ys)
        self.m, self.fmt = m, fmt
        self.streams = set()   # handles that the table and ys are recorded on

    @property
    def blocks(self) -> int:
        return int(self.plan.blocks)

    @property
    def route(self) -> int:
        return int(self.plan.route)


def fp8w_grouped_plan_init(xs, codes, scales, ys=None, fmt="block", route=ROUTE_AUTO) -> GroupedPlan:
    """Validate a group of GEMVs and write its device table (set-up call)."""
    return GroupedPlan(xs, codes, scales, ys, fmt, route)


def fp8w_gemv_grouped(plan: GroupedPlan, stream=None):
    """Enqueue every GEMV of ``plan`` in one launch; returns the ``y`` list."""
    _check(lib().fp8w_gemv_grouped(ctypes.byref(plan.plan), _plan_stream(plan, stream, *plan.ys)),
           "fp8w_gemv_grouped")
    return plan.ys


# ------------------------------------------------------- grouped quantize --

class QuantPlan:
    """Many weights quantized by one kernel launch (load time).

    Holds the device table and references to every buffer it names; codes
    and scales are allocated here when not given."""

    def __init__(self, ws, fmt: str = "block", codes=None, scales=None):
        torch = _torch()
        if not ws:
            raise ValueError("ws must be a non-empty list of bf16 [n, k] weights")
        fid = _format_id(fmt)
        if codes is None:
            codes = [torch.empty(tuple(w.shape), dtype=torch.uint8, device=w.device) for w in ws]
        if scales is None:
            scales = [torch.empty(scale_shape(fmt, *w.shape), dtype=_scale_dtype(torch, fmt), device=w.device)
                      for w in ws]
        if not (len(ws) == len(codes) == len(scales)):
            raise ValueError("ws, codes and scales must have equal lengths")
        descs = (QuantDesc * len(ws))()
        for i, (w, c, sc) in enumerate(zip(ws, codes, scales)):
            _require(w, _bf16_like(torch), "w", 2)
            _require(c, (torch.uint8,), "codes", 2)
            n, k = w.shape
            if tuple(c.shape) != (n, k):
                raise ValueError(f"grouped quantize {i}: codes shape {tuple(c.shape)} != {(n, k)}")
            _check_scales(torch, fmt, sc, n, k, "fp8w_quant_plan_init")
            descs[i] = QuantDesc(w.data_ptr(), c.data_ptr(), sc.data_ptr(), n, k)
        nbytes = int(lib().fp8w_quant_table_bytes(len(ws)))
        self.table = _table(nbytes, ws[0].device)
        self.plan = QuantPlanC()
        _check(lib().fp8w_quant_plan_init(descs, len(ws), fid, self.table.data_ptr(), ctypes.byref(self.plan)),
               "fp8w_quant_plan_init")
        self.ws, self.codes, self.scales, self.fmt = list(ws), list(codes), list(scales), fmt
        self.streams = set()   # handles that the table, codes and scales are recorded on

    @property
    def blocks(self) -> int:
        return int(self.plan.blocks)


def fp8w_quant_plan_init(ws, fmt="block", codes=None, scales=None) -> QuantPlan:
    """Validate a group of weights to quantize and write its device table
    (set-up call)."""
    return QuantPlan(ws, fmt, codes, scales)


def fp8w_quantize_grouped(plan: QuantPlan, stream=None):
    """Enqueue the quantization of every weight of ``plan`` in one launch;
    returns (codes list, scales list)."""
    _check(lib().fp8w_quantize_grouped(ctypes.byref(plan.plan), _plan_stream(plan, stream, *plan.codes, *plan.scales)),
           "fp8w_quantize_grouped")
    return plan.codes, plan.scales


# ---------------------------------------------------------------- experts --

SCORE_IDS = {"softmax": 0, "sigmoid": 1}
ACT_IDS = {"none": 0, "swiglu": 1}


class ExpertRouting(NamedTuple):
    """A router's choice: ``ids`` / ``weights`` / ``slots`` [tokens, top_k],
    ``rows`` [tokens * top_k] (the token of each slot) and ``offsets``
    [experts + 1] (expert e's slots)."""
    ids: object
    weights: object
    slots: object
    rows: object
    offsets: object


class Logprobs(NamedTuple):
    """``logprob`` [tokens] (None without targets), ``entropy`` [tokens], and
    ``top_ids`` / ``top_logprobs`` [tokens, top]."""
    logprob: object
    entropy: object
    top_ids: object
    top_logprobs: object


def _logits(t, what: str):
    """The dtype id and row stride of a [tokens, columns] logits tensor whose
    rows are contiguous."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what}: must be a GPU tensor (libfp8w has no CPU path)")
    if t.dtype is not torch.bfloat16 and t.dtype is not torch.float32:
        raise TypeError(f"{what}: dtype {t.dtype} is neither bfloat16 nor float32")
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-d tensor")
    rows, cols = t.shape
    stride = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or stride < cols:
        raise ValueError(f"{what}: rows must be contiguous and must not overlap")
    return (1 if t.dtype is torch.float32 else 0), stride


def _buffer(t, shape, dtype, device, what: str):
    """An output buffer: a new one, or the caller's after a check."""
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    _require(t, (dtype,), what, len(shape))   # says what is wrong
    raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")


def _workspace_bytes(t) -> int:
    """The size of a caller's workspace, any GPU tensor without gaps."""
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("workspace: expected a contiguous GPU tensor")
    return t.numel() * t.element_size()


def fp8w_route_experts(logits, top_k: int, score: str = "softmax", bias=None, renorm: bool = True,
                       scale: float = 1.0, ids=None, weights=None, slots=None, rows=None, offsets=None,
                       workspace=None, stream=None) -> ExpertRouting:
    """Router logits [tokens, experts] (bf16 or f32) -> each token's ``top_k``
    experts, their weights, and the map that sorts the tokens by expert."""
    torch = _torch()
    dtype, stride = _logits(logits, "logits")
    t, e = logits.shape
    k = int(top_k)
    if score not in SCORE_IDS:
        raise ValueError(f"unknown score {score!r}")
    if bias is not None:
        _require(bias, (torch.float32,), "bias", 1)
        if bias.shape[0] != e:
            raise ValueError(f"bias: expected shape {(e,)}, got {tuple(bias.shape)}")
    if k < 1:
        raise Fp8wError(ERR_SHAPE, "fp8w_route_experts")
    dev, i32 = logits.device, torch.int32
    ids = _buffer(ids, (t, k), i32, dev, "ids")
    weights = _buffer(weights, (t, k), torch.float32, dev, "weights")
    slots = _buffer(slots, (t, k), i32, dev, "slots")
    rows = _buffer(rows, (t * k,), i32, dev, "rows")
    offsets = _buffer(offsets, (e + 1,), i32, dev, "offsets")
    need = 0
    if workspace is not None:
        need = _workspace_bytes(workspace)
    elif t > 32:
        need = lib().fp8w_route_experts_workspace_bytes(t, e)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib().fp8w_route_experts(
        logits.data_ptr(), dtype, stride, t, e, k, SCORE_IDS[score], None if bias is None else bias.data_ptr(),
        1 if renorm else 0, scale, ids.data_ptr(), weights.data_ptr(), slots.data_ptr(), rows.data_ptr(),
        offsets.data_ptr(), None if workspace is None else workspace.data_ptr(), need,
        _launch_stream(stream, ids, weights, slots, rows, offsets, workspace)), "fp8w_route_experts")
    return ExpertRouting(ids, weights, slots, rows, offsets)


def fp8w_gemm_experts(x, codes, scales, offsets, rows=None, fmt: str = "block", act: str = "none", y=None,
                      stream=None):
    """Products grouped by expert: slot i of expert e (``offsets[e] <= i <
    offsets[e + 1]``) gets ``x[rows[i]] . deq(W_e)^T``, or with ``act="swiglu"``
    ``silu(g) * u`` of the products with W_e's two halves of rows.  codes u8
    [E,n,k]; scales the E scale buffers of ``fmt`` stacked.  Without ``rows``
    slot i takes x's row i."""
    torch = _torch()
    _require(x, _bf16_like(torch), "x", 2)
    _require(codes, (torch.uint8,), "codes", 3)
    _require(offsets, (torch.int32,), "offsets", 1)
    if act not in ACT_IDS:
        raise ValueError(f"unknown act {act!r}")
    fid = _format_id(fmt)
    e, n, k = codes.shape
    if x.shape[1] != k:
        raise ValueError(f"fp8w_gemm_experts: x has {x.shape[1]} columns, the weights {k}")
    want = (e, *scale_shape(fmt, n, k))
    _require(scales, (_scale_dtype(torch, fmt),), "scales", len(want))
    if scales.shape != want:
        raise ValueError(f"fp8w_gemm_experts: {fmt} scales must be {want}, got {tuple(scales.shape)}")
    if offsets.shape[0] != e + 1:
        raise ValueError(f"offsets: expected shape {(e + 1,)}, got {tuple(offsets.shape)}")
    if rows is not None:
        _require(rows, (torch.int32,), "rows", 1)
    slots = x.shape[0] if rows is None else rows.shape[0]
    n_out = n // 2 if act == "swiglu" else n
    if y is None:
        y = torch.empty((slots, n_out), dtype=torch.bfloat16, device=x.device)
    else:
        _require(y, _bf16_like(torch), "y", 2)
        if y.shape != (slots, n_out):
            raise ValueError(f"y: expected shape {(slots, n_out)}, got {tuple(y.shape)}")
    _check(lib().fp8w_gemm_experts(x.data_ptr(), x.shape[0], None if rows is None else rows.data_ptr(),
                                   offsets.data_ptr(), e, slots, codes.data_ptr(), scales.data_ptr(), fid, n, k,
                                   ACT_IDS[act], y.data_ptr(), _launch_stream(stream, y)), "fp8w_gemm_experts")
    return y


def fp8w_combine_experts(y, weights, slots, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * y[slots[t, j]] (slots of -1 add nothing)."""
    torch = _torch()
    _require(y, _bf16_like(torch), "y", 2)
    _require(weights, (torch.float32,), "weights", 2)
    _require(slots, (torch.int32,), "slots", 2)
    if weights.shape != slots.shape:
        raise ValueError(f"weights {tuple(weights.shape)} and slots {tuple(slots.shape)} differ in shape")
    t, k = slots.shape
    n = y.shape[1]
    if out is None:
        out = torch.empty((t, n), dtype=torch.bfloat16, device=y.device)
    else:
        _require(out, _bf16_like(torch), "out", 2)
        if out.shape != (t, n):
            raise ValueError(f"out: expected shape {(t, n)}, got {tuple(out.shape)}")
    _check(lib().fp8w_combine_experts(y.data_ptr(), y.shape[0], weights.data_ptr(), slots.data_ptr(), t, k, n,
                                      out.data_ptr(), _launch_stream(stream, out)), "fp8w_combine_experts")
    return out


@dataclass
class Fp8Experts:
    """The fp8 weights of a layer's experts: ``codes`` u8 [E,n,k] and the E
    scale buffers of ``fmt`` (the C ABI's names) stacked."""
    codes: object
    scales: object
    fmt: str

    @classmethod
    def quantize(cls, w, fmt: str = "block", stream=None) -> "Fp8Experts":
        """bf16 [E,n,k] weights, each expert quantized by ``fp8w_quantize``."""
        torch = _torch()
        _require(w, _bf16_like(torch), "w", 3)
        e, n, k = w.shape
        codes = torch.empty((e, n, k), dtype=torch.uint8, device=w.device)
        scales = torch.empty((e, *scale_shape(fmt, n, k)), dtype=_scale_dtype(torch, fmt), device=w.device)
        for i in range(e):
            fp8w_quantize(w[i], fmt, codes[i], scales[i], stream=stream)
        return cls(codes, scales, fmt)

    def matmul(self, x, offsets, rows=None, act: str = "none", y=None, stream=None):
        return fp8w_gemm_experts(x, self.codes, self.scales, offsets, rows, self.fmt, act, y, stream)


# --------------------------------------------------------------- logprobs --

def fp8w_logprobs(logits, targets=None, top: int = 0, logprob=None, entropy=None, top_ids=None, top_logprobs=None,
                  workspace=None, stream=None) -> Logprobs:
    """Log probabilities of ``targets`` (i32 [tokens]) under softmax(logits)
    (bf16 or f32 [tokens, vocab]), the entropy of each row and its ``top``
    most likely tokens."""
    torch = _torch()
    dtype, stride = _logits(logits, "logits")
    t, v = logits.shape
    top = int(top)
    dev, f32 = logits.device, torch.float32
    if targets is not None:
        _require(targets, (torch.int32,), "targets", 1)
        if targets.shape[0] != t:
            raise ValueError(f"targets: expected shape {(t,)}, got {tuple(targets.shape)}")
        logprob = _buffer(logprob, (t,), f32, dev, "logprob")
    elif logprob is not None:
        raise ValueError("logprob: given without targets")
    if top < 0:
        raise Fp8wError(ERR_SHAPE, "fp8w_logprobs")
    entropy = _buffer(entropy, (t,), f32, dev, "entropy")
    top_ids = _buffer(top_ids, (t, top), torch.int32, dev, "top_ids")
    top_logprobs = _buffer(top_logprobs, (t, top), f32, dev, "top_logprobs")
    if workspace is not None:
        need = _workspace_bytes(workspace)
    else:
        need = lib().fp8w_logprobs_workspace_bytes(t, v, top)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib().fp8w_logprobs(
        logits.data_ptr(), dtype, stride, t, v, None if targets is None else targets.data_ptr(), top,
        None if logprob is None else logprob.data_ptr(), entropy.data_ptr(), top_ids.data_ptr() if top else None,
        top_logprobs.data_ptr() if top else None, None if workspace is None else workspace.data_ptr(), need,
        _launch_stream(stream, logprob, entropy, top_ids, top_logprobs, workspace)), "fp8w_logprobs")
    return Logprobs(logprob, entropy, top_ids, top_logprobs)


# ----------------------------------------------------------- tagged weight --

BLOCK128, MX32, BLOCK128_BF16, ROW, TENSOR = "block128", "mx32", "block128_bf16", "row", "tensor"
_FMT_OF = {BLOCK128: "block", MX32: "mx", BLOCK128_BF16: "block_bf16", ROW: "row", TENSOR: "tensor"}


@dataclass
class Fp8Weight:
    """Quantized weight with its scale format fixed at construction.

    ``fmt`` is one of block128 (fp32 per 128x128 tile), mx32 (e8m0 per 32
    along K), block128_bf16, row (fp32 per row) and tensor (one fp32)."""
    codes: object
    scales: object
    n: int
    k: int
    fmt: str

    @classmethod
    def quantize(cls, w, fmt: str = BLOCK128, stream=None) -> "Fp8Weight":
        if fmt not in _FMT_OF:
            raise ValueError(f"unknown scale format {fmt!r}")
        c, s = fp8w_quantize(w, _FMT_OF[fmt], stream=stream)
        return cls(c, s, int(w.shape[0]), int(w.shape[1]), fmt)

    @property
    def format(self) -> str:
        """The C ABI's name of the scale format."""
        return _FMT_OF[self.fmt]

    def check_format(self) -> None:
        """The single place that decides which scale layout a weight carries."""
        torch = _torch()
        if self.fmt not in _FMT_OF:
            raise ValueError(f"Fp8Weight: unknown format {self.fmt!r}")
        f = _FMT_OF[self.fmt]
        if self.scales.dtype != _scale_dtype(torch, f) or tuple(self.scales.shape) != scale_shape(f, self.n, self.k):
            raise ValueError(f"Fp8Weight: scales do not match format {self.fmt!r}")

    def gemv(self, x, y=None, route=ROUTE_AUTO, stream=None):
        self.check_format()
        return fp8w_gemv(x, self.codes, self.scales, self.format, y, route, stream)

    def dequantize(self, w=None, stream=None):
        self.check_format()
        return fp8w_dequantize(self.codes, self.scales, self.format, w, stream)

    def matmul(self, x, y=None, workspace=None, stream=None):
        """y = x . deq(W)^T for any m: the fused GEMV for m <= 32 (the
        blockwise page's decode routing, Summary), dequantize + dense GEMM
        above."""
        self.check_format()
        if int(x.shape[0]) <= MAX_M:
            return self.gemv(x, y, ROUTE_AUTO, stream)
        return fp8w_gemm(x, self.codes, self.scales, self.format, y, workspace, stream)

    def gemv_w8a8(self, x_codes, x_scale, y=None, stream=None):
        self.check_format()
        return fp8w_gemv_w8a8(x_codes, x_scale, self.codes, self.scales, self.format, y, stream)
