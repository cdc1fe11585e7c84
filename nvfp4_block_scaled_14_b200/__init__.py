"""NVFP4 quantized linear layer for NVIDIA B200 (sm_100a).

The compute runs in libnvfp4.so (hand-written CUDA for sm_100a behind the C ABI of
include/nvfp4.h). This module marshals torch tensors into those calls: PyTorch supplies
device memory and the current stream, nothing else.

    q_w = quantize_fp8(w_e4m3, w_scale)       # double quantization of an FP8 checkpoint
    q_x = quantize(x_bf16)                    # dynamic per-tensor amax
    y = linear(q_x, q_w)                      # block-scaled W4A4 GEMM, bf16 out
    pct, mx = calib_percentile_amax(batches)  # static p99.9 input scale
    q_s = quantize(x_bf16, static_amax=pct)
    e_w = quantize_e4m3(w_bf16)               # FP8 E4M3 tensorwise (embed / lm_head layers)
    y8 = linear_e4m3(quantize_e4m3(x_bf16), e_w)
    y_lr = linear_lowrank(q_x, q_w, x_bf16, down, up)  # FP4 + BF16 rank-r branch
    m_x, m_xt = quantize_mxfp4(x_bf16, orient="both")  # MXFP4 along the rows and the columns
    y_mx = linear_mxfp4(m_x, m_w)             # microscaled product, no global scale
    ids, p = moe_route(x_bf16, w_router, 4)   # mixture-of-experts layer, up to 64 tokens
    y_moe = moe_experts(x_bf16, ids, p, gate_up, down)  # NVFP4 or MXFP4 expert weights

The C entry points are also available under their own names (``nvfp4_quantize`` ...).
"""
import functools
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import (NVFP4_BF16, NVFP4_F32, NVFP4_LINEAR_DEFAULT, NVFP4_LINEAR_RESIDENT_WEIGHTS,
                   NVFP4_OP_CALIB_BF16, NVFP4_OP_CALIB_F32, NVFP4_OP_LINEAR, NVFP4_OP_QUANTIZE,
                   NVFP4Error, check, load)

__all__ = ["NVFP4Tensor", "quantize", "quantize_fp8", "quantize_batch", "dequantize", "linear",
           "linear_dynamic", "linear_nvfp4_out", "linear_lowrank", "E4M3Tensor", "quantize_e4m3", "linear_e4m3",
           "MXFP4Tensor", "quantize_mxfp4", "dequantize_mxfp4", "linear_mxfp4",
           "linear_dynamic_mxfp4", "ExpertWeights", "stack_experts", "moe_route", "moe_experts",
           "calib_percentile_amax", "sync_status", "free_workspaces", "load", "NVFP4Error"]


def __getattr__(name):
    if name.startswith("nvfp4_"):
        return getattr(_lib, name)
    raise AttributeError(name)


@dataclass
class NVFP4Tensor:
    """A quantized [rows x cols] matrix: codes [rows, cols/2] u8, scales in the tensor-core
    layout (flat u8) and / or linear [rows, cols/16] u8, global scale (1-element fp32)."""
    codes: torch.Tensor
    scales_swz: torch.Tensor
    scales_lin: torch.Tensor
    global_scale: torch.Tensor
    rows: int
    cols: int


def _stream(device):
    return ctypes_ptr(torch.cuda.current_stream(device).cuda_stream)


def ctypes_ptr(v):
    return v if v else None


def _ptr(t):
    return None if t is None else t.data_ptr()


_ws_cache = {}


def _workspace(device, nbytes):
    """The calling stream's workspace on `device` (grown as needed). A workspace holds a call's
    state until its kernels finish, so calls on different streams, which may run at the same
    time, never share one; a buffer is only ever used (and freed) on the stream that
    allocated it. Each stream that has called the library keeps its workspace (at least
    1 MiB) for the life of the process; free_workspaces() drops them all."""
    if nbytes == 0:
        return None
    idx = device.index if device.index is not None else torch.cuda.current_device()
    key = (idx, torch.cuda.current_stream(idx).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def free_workspaces():
    """Drop every cached workspace (after the device work that used them has finished, e.g.
    after torch.cuda.synchronize()); later calls allocate afresh."""
    _ws_cache.clear()


def _alloc_outputs(rows, cols, device, swizzled, linear):
    L = load()
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
    swz = (torch.empty(L.nvfp4_scales_bytes(rows, cols, 1), dtype=torch.uint8, device=device)
           if swizzled else None)
    lin = torch.empty((rows, cols // 16), dtype=torch.uint8, device=device) if linear else None
    gs = torch.empty(1, dtype=torch.float32, device=device)
    return codes, swz, lin, gs


def quantize(x: torch.Tensor, static_amax: torch.Tensor = None, swizzled=True, linear=False,
             out: NVFP4Tensor = None) -> NVFP4Tensor:
    """NVFP4-quantize a 2-D fp32 / bf16 CUDA tensor (row-major, cols % 32 == 0)."""
    if x.dtype not in (torch.float32, torch.bfloat16) or x.dim() != 2 or not x.is_cuda:
        raise TypeError("quantize expects a 2-D CUDA fp32 or bf16 tensor")
    x = x.contiguous()
    rows, cols = x.shape
    if out is None:
        codes, swz, lin, gs = _alloc_outputs(rows, cols, x.device, swizzled, linear)
        out = NVFP4Tensor(codes, swz, lin, gs, rows, cols)
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(NVFP4_OP_QUANTIZE, rows, 0, cols)
    ws = _workspace(x.device, ws_bytes)
    dt = NVFP4_F32 if x.dtype == torch.float32 else NVFP4_BF16
    st = L.nvfp4_quantize(_ptr(x), dt, rows, cols, _ptr(static_amax), _ptr(out.codes),
                          _ptr(out.scales_swz), _ptr(out.scales_lin), _ptr(out.global_scale),
                          _ptr(ws), ws_bytes, _stream(x.device))
    check(st, "nvfp4_quantize")
    return out


def quantize_fp8(x_e4m3: torch.Tensor, fp8_scale: torch.Tensor = None,
                 static_amax: torch.Tensor = None, swizzled=True, linear=False,
                 out: NVFP4Tensor = None) -> NVFP4Tensor:
    """Double quantization: FP8 E4M3 (uint8 bits or float8_e4m3fn) x fp8_scale -> NVFP4."""
    if x_e4m3.dtype == torch.float8_e4m3fn:
        x_e4m3 = x_e4m3.view(torch.uint8)
    if x_e4m3.dtype != torch.uint8 or x_e4m3.dim() != 2 or not x_e4m3.is_cuda:
        raise TypeError("quantize_fp8 expects a 2-D CUDA uint8 / float8_e4m3fn tensor")
    x_e4m3 = x_e4m3.contiguous()
    rows, cols = x_e4m3.shape
    if out is None:
        codes, swz, lin, gs = _alloc_outputs(rows, cols, x_e4m3.device, swizzled, linear)
        out = NVFP4Tensor(codes, swz, lin, gs, rows, cols)
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(NVFP4_OP_QUANTIZE, rows, 0, cols)
    ws = _workspace(x_e4m3.device, ws_bytes)
    st = L.nvfp4_quantize_fp8_src(_ptr(x_e4m3), _ptr(fp8_scale), rows, cols, _ptr(static_amax),
                                  _ptr(out.codes), _ptr(out.scales_swz), _ptr(out.scales_lin),
                                  _ptr(out.global_scale), _ptr(ws), ws_bytes,
                                  _stream(x_e4m3.device))
    check(st, "nvfp4_quantize_fp8_src")
    return out


def quantize_batch(jobs) -> list:
    """Quantize several tensors in one pass (one amax launch and one encode launch for all);
    every tensor gets exactly what quantize / quantize_fp8 give it. jobs: a list of dicts with
    keys x (fp32 / bf16 tensor, or uint8 / float8_e4m3fn E4M3 bits), and optionally
    fp8_scale, static_amax, swizzled, linear, out. Returns the NVFP4Tensors."""
    import ctypes
    if not 1 <= len(jobs) <= _lib.NVFP4_MAX_QUANT_JOBS:
        raise ValueError("quantize_batch takes 1 to 8 tensors")
    descs = (_lib.QuantJob * len(jobs))()
    outs, keep = [], []
    dev = None
    for i, jb in enumerate(jobs):
        x = jb["x"]
        if x.dtype == torch.float8_e4m3fn:
            x = x.view(torch.uint8)
        if x.dim() != 2 or not x.is_cuda:
            raise TypeError("quantize_batch expects 2-D CUDA tensors")
        if x.dtype == torch.float32:
            src = _lib.NVFP4_SRC_F32
        elif x.dtype == torch.bfloat16:
            src = _lib.NVFP4_SRC_BF16
        elif x.dtype == torch.uint8:
            src = _lib.NVFP4_SRC_E4M3
        else:
            raise TypeError("quantize_batch: fp32, bf16 or E4M3 tensors")
        x = x.contiguous()
        keep.append(x)
        dev = x.device
        rows, cols = x.shape
        out = jb.get("out")
        if out is None:
            codes, swz, lin, gs = _alloc_outputs(rows, cols, x.device, jb.get("swizzled", True),
                                                 jb.get("linear", False))
            out = NVFP4Tensor(codes, swz, lin, gs, rows, cols)
        outs.append(out)
        d = descs[i]
        d.x, d.src = _ptr(x), src
        d.fp8_scale = _ptr(jb.get("fp8_scale"))
        d.rows, d.cols = rows, cols
        d.static_amax = _ptr(jb.get("static_amax"))
        d.codes, d.scales_swz = _ptr(out.codes), _ptr(out.scales_swz)
        d.scales_lin, d.global_scale = _ptr(out.scales_lin), _ptr(out.global_scale)
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(NVFP4_OP_QUANTIZE, 0, 0, 0)
    ws = _workspace(dev, ws_bytes)
    st = L.nvfp4_quantize_batch(descs, len(jobs), _ptr(ws), ws_bytes, _stream(dev))
    check(st, "nvfp4_quantize_batch")
    return outs


def dequantize(q: NVFP4Tensor, out_dtype=torch.float32, out: torch.Tensor = None) -> torch.Tensor:
    """fp32 / bf16 values of q [rows, cols]; out: an optional preallocated contiguous output."""
    if q.scales_lin is None:
        raise ValueError("dequantize needs the linear scales (quantize(..., linear=True))")
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.codes.device)
    elif out.dtype != out_dtype or tuple(out.shape) != (q.rows, q.cols) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [rows, cols] tensor of out_dtype")
    dt = NVFP4_F32 if out_dtype == torch.float32 else NVFP4_BF16
    st = load().nvfp4_dequantize(_ptr(q.codes), _ptr(q.scales_lin), _ptr(q.global_scale),
                                 q.rows, q.cols, dt, _ptr(out), _stream(q.codes.device))
    check(st, "nvfp4_dequantize")
    return out


def linear(a: NVFP4Tensor, w: NVFP4Tensor, out_dtype=torch.bfloat16,
           out: torch.Tensor = None, resident_weights: bool = False) -> torch.Tensor:
    """Y = dequant(a) . dequant(w)^T, [a.rows x w.rows], fp32 accumulation.

    resident_weights: w is not written by work still running on the stream (weights quantized
    ahead of time); lets small-M calls start reading w before the previous kernel finishes."""
    if a.cols != w.cols:
        raise ValueError("K mismatch")
    M, N, K = a.rows, w.rows, a.cols
    dev = a.codes.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(NVFP4_OP_LINEAR, M, N, K)
    ws = _workspace(dev, ws_bytes)
    dt = NVFP4_F32 if out.dtype == torch.float32 else NVFP4_BF16
    flags = NVFP4_LINEAR_RESIDENT_WEIGHTS if resident_weights else NVFP4_LINEAR_DEFAULT
    st = L.nvfp4_linear_ex(_ptr(a.codes), _ptr(a.scales_swz), _ptr(a.global_scale),
                           _ptr(w.codes), _ptr(w.scales_swz), _ptr(w.global_scale), M, N, K, dt,
                           _ptr(out), _ptr(ws), ws_bytes, flags, _stream(dev))
    check(st, "nvfp4_linear_ex")
    return out


def linear_dynamic(x: torch.Tensor, w: NVFP4Tensor, out_dtype=torch.bfloat16,
                   out: torch.Tensor = None, resident_weights: bool = False,
                   x_gs_out: torch.Tensor = None) -> torch.Tensor:
    """Y = dequant(quantize(x)) . dequant(w)^T with the dynamic per-tensor amax, from fp32 / bf16
    activations x [M x K]; one fused kernel for M <= 16. x_gs_out (1-element fp32 CUDA tensor)
    receives the activations' global scale."""
    if x.dtype not in (torch.float32, torch.bfloat16) or x.dim() != 2 or not x.is_cuda:
        raise TypeError("linear_dynamic expects a 2-D CUDA fp32 or bf16 tensor")
    x = x.contiguous()
    M, K = x.shape
    if K != w.cols:
        raise ValueError("K mismatch")
    N = w.rows
    dev = x.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(_lib.NVFP4_OP_LINEAR_DYNAMIC, M, N, K)
    ws = _workspace(dev, ws_bytes)
    flags = NVFP4_LINEAR_RESIDENT_WEIGHTS if resident_weights else NVFP4_LINEAR_DEFAULT
    st = L.nvfp4_linear_dynamic(_ptr(x), NVFP4_F32 if x.dtype == torch.float32 else NVFP4_BF16,
                                _ptr(w.codes), _ptr(w.scales_swz), _ptr(w.global_scale), M, N, K,
                                NVFP4_F32 if out.dtype == torch.float32 else NVFP4_BF16,
                                _ptr(out), _ptr(x_gs_out), _ptr(ws), ws_bytes, flags,
                                _stream(dev))
    check(st, "nvfp4_linear_dynamic")
    return out


def linear_nvfp4_out(a: NVFP4Tensor, w: NVFP4Tensor, static_amax: torch.Tensor,
                     act: str = "identity", out: NVFP4Tensor = None) -> NVFP4Tensor:
    """NVFP4 (static amax) of act(dequant(a) . dequant(w)^T), quantized in the GEMM's epilogue;
    act is "identity" or "gelu_tanh". The result feeds linear() as its activation operand."""
    if a.cols != w.cols:
        raise ValueError("K mismatch")
    acts = {"identity": _lib.NVFP4_ACT_IDENTITY, "gelu_tanh": _lib.NVFP4_ACT_GELU_TANH}
    if act not in acts:
        raise ValueError(f"act must be one of {sorted(acts)}")
    M, N, K = a.rows, w.rows, a.cols
    dev = a.codes.device
    if out is None:
        codes, swz, _, gs = _alloc_outputs(M, N, dev, True, False)
        out = NVFP4Tensor(codes, swz, None, gs, M, N)
    st = load().nvfp4_linear_nvfp4_out(_ptr(a.codes), _ptr(a.scales_swz), _ptr(a.global_scale),
                                       _ptr(w.codes), _ptr(w.scales_swz), _ptr(w.global_scale),
                                       M, N, K, acts[act], _ptr(static_amax), _ptr(out.codes),
                                       _ptr(out.scales_swz), _ptr(out.global_scale),
                                       _stream(dev))
    check(st, "nvfp4_linear_nvfp4_out")
    return out


def linear_lowrank(a: NVFP4Tensor, w: NVFP4Tensor, x: torch.Tensor, down: torch.Tensor,
                   up: torch.Tensor, out: torch.Tensor = None) -> torch.Tensor:
    """Y = dequant(a) . dequant(w)^T + (x . down^T) . up^T, bf16 [a.rows x w.rows].

    x: the layer's bf16 input [M, K] (a is its NVFP4 quantization); down: bf16 [rank, K];
    up: bf16 [N, rank]. The branch's intermediate is kept in bf16 (divided by the FP4 product's
    global scales, so that both parts share one fp32 tensor-core accumulator)."""
    if a.cols != w.cols:
        raise ValueError("K mismatch")
    M, N, K = a.rows, w.rows, a.cols
    if x.dtype != torch.bfloat16 or down.dtype != torch.bfloat16 or up.dtype != torch.bfloat16:
        raise TypeError("x, down and up must be bfloat16")
    rank = down.shape[0]
    if tuple(x.shape) != (M, K) or tuple(down.shape) != (rank, K) or tuple(up.shape) != (N, rank):
        raise ValueError("shape mismatch: x [M, K], down [rank, K], up [N, rank]")
    x, down, up = x.contiguous(), down.contiguous(), up.contiguous()
    dev = a.codes.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(_lib.NVFP4_OP_LINEAR_LOWRANK, M, rank, 0)
    ws = _workspace(dev, ws_bytes)
    st = L.nvfp4_linear_lowrank(_ptr(a.codes), _ptr(a.scales_swz), _ptr(a.global_scale),
                                _ptr(w.codes), _ptr(w.scales_swz), _ptr(w.global_scale),
                                _ptr(x), _ptr(down), _ptr(up), M, N, K, rank, _ptr(out), _ptr(ws),
                                ws_bytes, _stream(dev))
    check(st, "nvfp4_linear_lowrank")
    return out


@dataclass
class E4M3Tensor:
    """FP8 E4M3 tensorwise: codes [rows, cols] uint8 and one fp32 scale (device, [1])."""
    codes: torch.Tensor
    scale: torch.Tensor

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def cols(self):
        return self.codes.shape[1]


def quantize_e4m3(x: torch.Tensor, static_amax: torch.Tensor = None,
                  out: E4M3Tensor = None) -> E4M3Tensor:
    """FP8 E4M3 tensorwise quantize of a 2-D fp32 / bf16 CUDA tensor: s = amax / 448,
    code = sign | E4M3(|x| / s) (nearest, ties to even, saturating)."""
    if x.dtype not in (torch.float32, torch.bfloat16) or x.dim() != 2 or not x.is_cuda:
        raise TypeError("quantize_e4m3 expects a 2-D CUDA fp32 or bf16 tensor")
    x = x.contiguous()
    rows, cols = x.shape
    if out is None:
        out = E4M3Tensor(torch.empty((rows, cols), dtype=torch.uint8, device=x.device),
                         torch.empty(1, dtype=torch.float32, device=x.device))
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(_lib.NVFP4_OP_QUANTIZE_E4M3, 0, 0, 0)
    ws = _workspace(x.device, ws_bytes)
    dt = NVFP4_F32 if x.dtype == torch.float32 else NVFP4_BF16
    st = L.nvfp4_quantize_e4m3(_ptr(x), dt, rows, cols, _ptr(static_amax), _ptr(out.codes),
                               _ptr(out.scale), _ptr(ws), ws_bytes, _stream(x.device))
    check(st, "nvfp4_quantize_e4m3")
    return out


def linear_e4m3(a: E4M3Tensor, w: E4M3Tensor, out_dtype=torch.bfloat16,
                out: torch.Tensor = None) -> torch.Tensor:
    """Y = (sA * sW) * A . W^T from E4M3 codes, [a.rows x w.rows], fp32 accumulation."""
    if a.cols != w.cols:
        raise ValueError("K mismatch")
    M, N, K = a.rows, w.rows, a.cols
    dev = a.codes.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    dt = NVFP4_F32 if out.dtype == torch.float32 else NVFP4_BF16
    st = load().nvfp4_linear_e4m3(_ptr(a.codes), _ptr(a.scale), _ptr(w.codes), _ptr(w.scale),
                                  M, N, K, dt, _ptr(out), _stream(dev))
    check(st, "nvfp4_linear_e4m3")
    return out


@dataclass
class MXFP4Tensor:
    """An MXFP4 [rows x cols] matrix: codes [rows, cols/2] u8, E8M0 scales (one per 32 values) in
    the tensor-core layout (flat u8) and / or linear [rows, cols/32] u8."""
    codes: torch.Tensor
    scales_swz: torch.Tensor
    scales_lin: torch.Tensor
    rows: int
    cols: int


_MX_RULES = {"floor": _lib.NVFP4_MX_SCALE_FLOOR, "ceil": _lib.NVFP4_MX_SCALE_CEIL}
_OUT_TYPES = {torch.float32: NVFP4_F32, torch.bfloat16: NVFP4_BF16}


def _scratch(device, nbytes):
    """A call's own workspace on the current stream (None if it needs none). It is not kept: a
    captured graph holds its own in its memory pool, so two graphs never share one, and the
    allocator hands an eager call's back to this stream only."""
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


@functools.lru_cache(maxsize=4096)
def _workspace_size(index, op, m, n, k):
    """nvfp4_workspace_bytes on device `index` (a function of the sizes and the device)."""
    with torch.cuda.device(index):
        return load().nvfp4_workspace_bytes(op, m, n, k)


@functools.lru_cache(maxsize=4096)
def _moe_workspace_size(index, T, H, F, k):
    with torch.cuda.device(index):
        return load().nvfp4_moe_workspace_bytes(T, H, F, k)


try:  # the integers behind torch.cuda.current_device() / current_stream(), without the objects
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _device_index
except ImportError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

    def _device_index():
        return torch.cuda.current_device()


def _launch(what, dev, *args):
    """The C call `what` on the device's current stream (appended to args), with that device current:
    the library launches on the current device, which is normally that one already."""
    f = getattr(load(), what)
    if _device_index() == dev.index:
        st = f(*args, _raw_stream(dev.index) or None)
    else:
        with torch.cuda.device(dev):
            st = f(*args, _raw_stream(dev.index) or None)
    if st:
        check(st, what)


def _bad_array(what, name, t, device, dtype, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise ValueError(f"{what}: {name} must be a tensor on {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: {name} must be {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: {name} must have shape {tuple(shape)}")
    raise ValueError(f"{what}: {name} must be contiguous")


def _check_array(what, name, t, device, dtype, shape):
    """t lies contiguous on the CUDA device, with that type and shape (None: any)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == device and
            (dtype is None or t.dtype == dtype) and (shape is None or t.shape == shape) and
            t.is_contiguous()):
        _bad_array(what, name, t, device, dtype, shape)


def _mx_swizzled_bytes(rows, cols):
    return -(-rows // 128) * 512 * -(-cols // 128)


def _check_mx(what, q, device, swizzled=False):
    """An MXFP4Tensor's arrays on `device`, of its size, with the scales the call reads (operand
    layout, or linear)."""
    if not isinstance(q, MXFP4Tensor):
        raise TypeError(f"{what} expects MXFP4Tensor operands")
    rows, cols = q.rows, q.cols
    if cols % 32 or rows < 0 or cols < 0:
        raise ValueError(f"{what}: cols must be a multiple of 32")
    _check_array(what, "codes", q.codes, device, torch.uint8, (rows, cols // 2))
    if swizzled:
        if q.scales_swz is None:
            raise ValueError(f"{what} needs the swizzled scales")
        _check_array(what, "scales_swz", q.scales_swz, device, torch.uint8,
                     (_mx_swizzled_bytes(rows, cols),))
    else:
        if q.scales_lin is None:
            raise ValueError(f"{what} needs the linear scales")
        _check_array(what, "scales_lin", q.scales_lin, device, torch.uint8, (rows, cols // 32))


def _codes_device(what, q):
    if not isinstance(q.codes, torch.Tensor):
        raise TypeError(f"{what} expects codes as a tensor")
    return q.codes.device


def _empty(rows, cols, dtype, device):
    """torch.empty((rows, cols)), by the constructor that takes two thirds of its time."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _mx_out(what, out, rows, cols, dtype, device):
    if dtype not in _OUT_TYPES:
        raise TypeError(f"{what}: out_dtype must be float32 or bfloat16")
    if out is None:
        return _empty(rows, cols, dtype, device)
    _check_array(what, "out", out, device, dtype, (rows, cols))
    return out


def _mx_alloc(rows, cols, device, swizzled, linear):
    """An MXFP4Tensor [rows, cols] with uninitialized arrays, and their addresses."""
    u8 = torch.uint8
    codes = _empty(rows, cols // 2, u8, device)
    swz = torch.empty(_mx_swizzled_bytes(rows, cols), dtype=u8, device=device) if swizzled else None
    lin = _empty(rows, cols // 32, u8, device) if linear else None
    return MXFP4Tensor(codes, swz, lin, rows, cols), (
        codes.data_ptr(), swz.data_ptr() if swizzled else None, lin.data_ptr() if linear else None)


def quantize_mxfp4(x: torch.Tensor, scale_rule: str = "floor", orient: str = "rows",
                   swizzled=True, linear=False):
    """MXFP4-quantize a 2-D fp32 / bf16 CUDA tensor (cols % 32 == 0): E2M1 codes with one
    power-of-two scale per 32 values. scale_rule: "floor" (2^(floor(log2 max) - 2), large values
    may saturate) or "ceil" (the smallest scale at which nothing saturates). orient: "rows" (blocks
    along the rows, an MXFP4Tensor [rows, cols]), "cols" (the same of x^T, [cols, rows padded to a
    multiple of 32 with zeros]) or "both" (the pair of them, x read once)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _OUT_TYPES or x.dim() != 2 or \
            not x.is_cuda:
        raise TypeError("quantize_mxfp4 expects a 2-D CUDA fp32 or bf16 tensor")
    if scale_rule not in _MX_RULES:
        raise ValueError(f"scale_rule must be one of {sorted(_MX_RULES)}")
    if orient not in ("rows", "cols", "both"):
        raise ValueError("orient must be 'rows', 'cols' or 'both'")
    if not swizzled and not linear:
        raise ValueError("quantize_mxfp4 needs swizzled or linear scales")
    x = x.contiguous()
    rows, cols = x.shape
    if cols % 32:
        raise ValueError("quantize_mxfp4: cols must be a multiple of 32")
    dev = x.device
    qr = qc = None
    to_r = to_c = (None, None, None)
    if orient != "cols":
        qr, to_r = _mx_alloc(rows, cols, dev, swizzled, linear)
    if orient != "rows":
        qc, to_c = _mx_alloc(cols, -(-rows // 32) * 32, dev, swizzled, linear)
    _launch("nvfp4_quantize_mxfp4", dev, x.data_ptr(), _OUT_TYPES[x.dtype], rows, cols,
            _MX_RULES[scale_rule], *to_r, *to_c)
    return (qr, qc) if orient == "both" else qr or qc


def dequantize_mxfp4(q: MXFP4Tensor, out_dtype=torch.float32,
                     out: torch.Tensor = None) -> torch.Tensor:
    """fp32 / bf16 values of q [rows, cols] (needs its linear scales)."""
    if not isinstance(q, MXFP4Tensor):
        raise TypeError("dequantize_mxfp4 expects an MXFP4Tensor")
    dev = _codes_device("dequantize_mxfp4", q)
    _check_mx("dequantize_mxfp4", q, dev)
    out = _mx_out("dequantize_mxfp4", out, q.rows, q.cols, out_dtype, dev)
    _launch("nvfp4_dequantize_mxfp4", dev, q.codes.data_ptr(), q.scales_lin.data_ptr(), q.rows,
            q.cols, _OUT_TYPES[out_dtype], out.data_ptr())
    return out


def linear_mxfp4(a: MXFP4Tensor, w: MXFP4Tensor, out_dtype=torch.bfloat16,
                 out: torch.Tensor = None, resident_weights: bool = False) -> torch.Tensor:
    """Y = dequant(a) . dequant(w)^T, [a.rows x w.rows], from MXFP4 operands with fp32
    accumulation. With x quantized "rows" and "cols", w and dy likewise, the gradients of
    y = x . w^T are linear_mxfp4(dy_rows, w_cols) and linear_mxfp4(dy_cols, x_cols).
    resident_weights: as in linear()."""
    if not isinstance(a, MXFP4Tensor):
        raise TypeError("linear_mxfp4 expects MXFP4Tensor operands")
    dev = _codes_device("linear_mxfp4", a)
    _check_mx("linear_mxfp4", a, dev, swizzled=True)
    _check_mx("linear_mxfp4", w, dev, swizzled=True)
    if a.cols != w.cols:
        raise ValueError("K mismatch")
    M, N, K = a.rows, w.rows, a.cols
    out = _mx_out("linear_mxfp4", out, M, N, out_dtype, dev)
    flags = NVFP4_LINEAR_RESIDENT_WEIGHTS if resident_weights else NVFP4_LINEAR_DEFAULT
    ws_bytes = _workspace_size(dev.index, NVFP4_OP_LINEAR, M, N, K)
    ws = _scratch(dev, ws_bytes)
    _launch("nvfp4_linear_mxfp4", dev, a.codes.data_ptr(), a.scales_swz.data_ptr(),
            w.codes.data_ptr(), w.scales_swz.data_ptr(), M, N, K, _OUT_TYPES[out_dtype],
            out.data_ptr(), _ptr(ws), ws_bytes, flags)
    return out


def linear_dynamic_mxfp4(x: torch.Tensor, w: MXFP4Tensor, out_dtype=torch.bfloat16,
                         out: torch.Tensor = None,
                         resident_weights: bool = False) -> torch.Tensor:
    """Y = dequant(quantize_mxfp4(x)) . dequant(w)^T from fp32 / bf16 activations x [M x K]; one
    fused kernel for M <= 16."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _OUT_TYPES or x.dim() != 2 or \
            not x.is_cuda:
        raise TypeError("linear_dynamic_mxfp4 expects a 2-D CUDA fp32 or bf16 tensor")
    dev = x.device
    _check_mx("linear_dynamic_mxfp4", w, dev, swizzled=True)
    x = x.contiguous()
    M, K = x.shape
    if K != w.cols:
        raise ValueError("K mismatch")
    N = w.rows
    out = _mx_out("linear_dynamic_mxfp4", out, M, N, out_dtype, dev)
    flags = NVFP4_LINEAR_RESIDENT_WEIGHTS if resident_weights else NVFP4_LINEAR_DEFAULT
    ws_bytes = _workspace_size(dev.index, _lib.NVFP4_OP_LINEAR_DYNAMIC_MXFP4, M, N, K)
    ws = _scratch(dev, ws_bytes)
    _launch("nvfp4_linear_dynamic_mxfp4", dev, x.data_ptr(), _OUT_TYPES[x.dtype],
            w.codes.data_ptr(), w.scales_swz.data_ptr(), M, N, K, _OUT_TYPES[out_dtype],
            out.data_ptr(), _ptr(ws), ws_bytes, flags)
    return out


@dataclass
class ExpertWeights:
    """The 4-bit weights [rows x cols] of E experts, stacked: codes [E, rows, cols/2] u8, linear
    block scales [E, rows, cols/16] (NVFP4) or [E, rows, cols/32] (MXFP4) u8, and for NVFP4 the
    global scales [E] fp32 (None: MXFP4). stack_experts() builds one from quantized matrices."""
    codes: torch.Tensor
    scales: torch.Tensor
    global_scale: torch.Tensor = None


def stack_experts(experts) -> ExpertWeights:
    """ExpertWeights of a list of NVFP4Tensor or MXFP4Tensor matrices (one per expert, all of one
    kind and size, quantized with linear=True)."""
    experts = list(experts)
    if not experts or any(type(q) is not type(experts[0]) or (q.rows, q.cols) !=
                          (experts[0].rows, experts[0].cols) for q in experts) or \
            not isinstance(experts[0], (NVFP4Tensor, MXFP4Tensor)):
        raise TypeError("stack_experts expects NVFP4Tensor or MXFP4Tensor matrices of one size")
    if any(q.scales_lin is None for q in experts):
        raise ValueError("stack_experts needs the linear scales (quantize(..., linear=True))")
    gs = torch.cat([q.global_scale for q in experts]) if isinstance(experts[0], NVFP4Tensor) \
        else None
    return ExpertWeights(torch.stack([q.codes for q in experts]),
                         torch.stack([q.scales_lin for q in experts]), gs)


def moe_route(x: torch.Tensor, w: torch.Tensor, top_k: int, bias: torch.Tensor = None,
              renormalize: bool = True):
    """Router: (ids int32 [T, top_k], weights fp32 [T, top_k]) of the top_k largest x . w^T + bias
    of each token (equal ones: the lower expert), x [T, H] and w [E, H] bf16, bias [E] fp32. The
    weights are the softmax over the chosen experts (renormalize) or over all. An expert whose
    logit is -inf or NaN is never chosen; slots left over hold id -1 and weight 0."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 2 or \
            not x.is_cuda:
        raise TypeError("moe_route expects 2-D CUDA bfloat16 activations")
    if not isinstance(w, torch.Tensor) or w.dtype != torch.bfloat16 or w.dim() != 2:
        raise TypeError("moe_route expects a 2-D bfloat16 router weight")
    dev = x.device
    x, w = x.contiguous(), w.contiguous()
    T, H = x.shape
    E = w.shape[0]
    _check_array("moe_route", "w", w, dev, None, (E, H))
    if bias is not None:
        _check_array("moe_route", "bias", bias, dev, torch.float32, (E,))
    if not 1 <= top_k <= min(E, 32):
        raise ValueError("moe_route: top_k must be 1..min(experts, 32)")
    ids = _empty(T, top_k, torch.int32, dev)
    weights = _empty(T, top_k, torch.float32, dev)
    _launch("nvfp4_moe_route", dev, x.data_ptr(), w.data_ptr(), _ptr(bias), T, H, E, top_k,
            int(renormalize), ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                gate_up: ExpertWeights, down: ExpertWeights,
                out: torch.Tensor = None) -> torch.Tensor:
    """Experts of a mixture-of-experts layer for up to 64 tokens, bf16 [T, H]:
    y[t] = sum_s weights[t, s] * down_e (silu(gate_e x[t]) * (up_e x[t])), e = ids[t, s].

    x [T, H] bf16; ids int32 and weights fp32 [T, k] (an id outside the experts names none);
    gate_up: E x [2F, H] (gate rows first); down: E x [H, F]; both NVFP4 or both MXFP4. x and the
    hidden values are not rounded to 4 bits: off by at most 2^-22 of the largest of a block of 32
    (MXFP4 weights) or 16 (NVFP4; at least 2^-39 of the row's largest). The same call gives the
    same bits."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.dim() != 2 or \
            not x.is_cuda:
        raise TypeError("moe_experts expects 2-D CUDA bfloat16 activations")
    if not isinstance(gate_up, ExpertWeights) or not isinstance(down, ExpertWeights):
        raise TypeError("moe_experts expects ExpertWeights")
    if (gate_up.global_scale is None) != (down.global_scale is None):
        raise ValueError("moe_experts: gate_up and down must have the same format")
    if not isinstance(ids, torch.Tensor) or not isinstance(gate_up.codes, torch.Tensor):
        raise TypeError("moe_experts expects ids and codes as tensors")
    dev = x.device
    x = x.contiguous()
    T, H = x.shape
    if gate_up.codes.dim() != 3 or ids.dim() != 2:
        raise ValueError("moe_experts: codes must be [experts, rows, cols / 2], ids [T, k]")
    E, F = gate_up.codes.shape[0], gate_up.codes.shape[1] // 2
    k = ids.shape[1]
    if T > 64:
        raise ValueError("moe_experts takes up to 64 tokens")
    if H % 32 or F % 32 or H == 0 or F == 0:
        raise ValueError("moe_experts: H and F must be multiples of 32")
    mx = gate_up.global_scale is None
    b = 32 if mx else 16
    u8 = torch.uint8
    for name, t, dtype, shape in (
            ("ids", ids, torch.int32, (T, k)), ("weights", weights, torch.float32, (T, k)),
            ("gate_up codes", gate_up.codes, u8, (E, 2 * F, H // 2)),
            ("gate_up scales", gate_up.scales, u8, (E, 2 * F, H // b)),
            ("down codes", down.codes, u8, (E, H, F // 2)),
            ("down scales", down.scales, u8, (E, H, F // b))):
        _check_array("moe_experts", name, t, dev, dtype, shape)
    if not mx:
        for name, w in (("gate_up global_scale", gate_up), ("down global_scale", down)):
            _check_array("moe_experts", name, w.global_scale, dev, torch.float32, (E,))
    if out is None:
        out = _empty(T, H, torch.bfloat16, dev)
    else:
        _check_array("moe_experts", "out", out, dev, torch.bfloat16, (T, H))
    ws_bytes = _moe_workspace_size(dev.index, T, H, F, k)
    ws = _scratch(dev, ws_bytes)
    _launch("nvfp4_moe_experts", dev, x.data_ptr(), T, H, F, E, k, ids.data_ptr(),
            weights.data_ptr(), _lib.NVFP4_EXPERTS_MXFP4 if mx else _lib.NVFP4_EXPERTS_NVFP4,
            gate_up.codes.data_ptr(), gate_up.scales.data_ptr(), _ptr(gate_up.global_scale),
            down.codes.data_ptr(), down.scales.data_ptr(), _ptr(down.global_scale),
            out.data_ptr(), _ptr(ws), ws_bytes)
    return out


def calib_percentile_amax(batches, num=999, den=1000):
    """Exact nearest-rank num/den percentile of |x| over all batches, and max |x|.
    Returns two 1-element fp32 CUDA tensors (usable as static_amax)."""
    import ctypes
    batches = [b.contiguous() for b in batches]
    dtype = batches[0].dtype
    n = batches[0].numel()
    if any(b.dtype != dtype or b.numel() != n for b in batches):
        raise ValueError("all batches must share dtype and size")
    dev = batches[0].device
    dt = NVFP4_BF16 if dtype == torch.bfloat16 else NVFP4_F32
    L = load()
    ws_bytes = L.nvfp4_workspace_bytes(NVFP4_OP_CALIB_BF16 if dt == NVFP4_BF16
                                       else NVFP4_OP_CALIB_F32, 0, 0, 0)
    ws = _workspace(dev, ws_bytes)
    out = torch.empty(2, dtype=torch.float32, device=dev)
    ptrs = (ctypes.c_void_p * len(batches))(*[b.data_ptr() for b in batches])
    st = L.nvfp4_calib_percentile_amax(ptrs, len(batches), n, dt, num, den, out.data_ptr(),
                                       out.data_ptr() + 4, _ptr(ws), ws_bytes, _stream(dev))
    check(st, "nvfp4_calib_percentile_amax")
    return out[0:1], out[1:2]


def sync_status(device=None):
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    return load().nvfp4_sync_status(_stream(dev))
