"""Python front end of the C ABI: argument marshalling only.

Each function takes torch tensors that already live on the GPU, passes their
device pointers and the current CUDA stream to the C entry point of the same
name, and raises ``FFNError`` on a non-OK status.  PyTorch supplies device
memory (outputs and workspace come from torch's allocator) and streams;
every step of the computation runs in the library's own kernels.
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import _lib
from ._lib import (FFN_AUTO, FFN_BF16, FFN_F16, FFN_F32, FFN_GATEUP_FUSED,  # noqa: F401
                   FFN_GATEUP_UNFUSED, FFN_ACT_SINGLE, FFN_ACT_SPLIT, FFN_PATH_GEMM,
                   FFN_PATH_GEMV, FFN_PREPARED_WEIGHTS, FFN_RESIDUAL, FFN_DECODE_ONE_KERNEL,
                   FFN_ROUTE_RENORM, FFN_ROUTE_SIGMOID,
                   Fp8Weight, Q4Weight, Q8Weight)

_DT = {torch.float32: FFN_F32, torch.float16: FFN_F16, torch.bfloat16: FFN_BF16}

_LIB = _lib.load()  # fail at import when the CUDA library is missing


class FFNError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib.load()
        msg = lib.ffn_status_string(status).decode()
        super().__init__(f"{where}: {_lib.STATUS.get(status, status)} ({msg})")
        self.status = status


def _check(status: int, where: str):
    if status != 0:
        raise FFNError(status, where)


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _expect(name: str, t, shape, dtype, device):
    """A tensor the C side cannot look into: its sizes, type and place."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, is {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    raise ValueError(f"{name} must be a contiguous CUDA tensor on the device of the input")


def _launch(fn, where: str, device: int, *args):
    """fn(*args, stream) on the current stream of `device`, with it current."""
    if device != _current_device():
        with torch.cuda.device(device):
            return _launch(fn, where, device, *args)
    status = fn(*args, _raw_stream(device))
    if status != 0:
        raise FFNError(status, where)


# what torch.cuda.current_device() and current_stream() come down to once a
# CUDA tensor exists (these calls are a third of a small operator's time)
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _rows_of(x: torch.Tensor):
    """(rows, d, device index) of a [..., d] input tensor."""
    dev = x.get_device()
    if dev < 0 or not x.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    d = x.shape[-1]
    return (x.numel() // d if d else 0), d, dev


def ffn_add_rmsnorm(x: torch.Tensor, g: torch.Tensor, eps: float, res: torch.Tensor | None = None,
                    r_out: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None):
    """(r, n): r = x + res (x itself without `res`) and n = RMSNorm(r) * g.

    `r_out` may be x or res (in place); without it a new tensor takes r."""
    if stream is not None:   # outputs and workspaces made here belong to that stream
        with torch.cuda.stream(stream):
            return ffn_add_rmsnorm(x, g, eps, res, r_out, out)
    rows, d, dev = _rows_of(x)
    dt, shape = x.dtype, x.shape
    code = _dtype(x)
    _expect("g", g, (d,), dt, dev)
    if res is not None:
        _expect("res", res, shape, dt, dev)
        if r_out is None:
            r_out = torch.empty_like(x)
    if r_out is not None:
        _expect("r_out", r_out, shape, dt, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _expect("out", out, shape, dt, dev)
    _launch(_LIB.ffn_add_rmsnorm, "ffn_add_rmsnorm", dev, x.data_ptr(),
            None if res is None else res.data_ptr(), g.data_ptr(), None if r_out is None else r_out.data_ptr(),
            out.data_ptr(), rows, d, eps, code)
    return (x if r_out is None else r_out), out


def ffn_add_rmsnorm_e4m3(x: torch.Tensor, g: torch.Tensor, eps: float, res: torch.Tensor | None = None,
                         group: int = 0, r_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         scales: torch.Tensor | None = None, stream=None):
    """(r, q, scales): as ffn_add_rmsnorm with the norm's output as
    torch.float8_e4m3fn codes and fp32 scales, one per row (group 0, shape
    [rows, 1]) or per `group` columns (32, 64 or 128; [rows, ceil(d / group)]):
    RMSNorm(r) * g is about q * scale."""
    if stream is not None:   # outputs and workspaces made here belong to that stream
        with torch.cuda.stream(stream):
            return ffn_add_rmsnorm_e4m3(x, g, eps, res, group, r_out, out, scales)
    rows, d, dev = _rows_of(x)
    dt, shape = x.dtype, x.shape
    code = _dtype(x)
    _expect("g", g, (d,), dt, dev)
    if res is not None:
        _expect("res", res, shape, dt, dev)
        if r_out is None:
            r_out = torch.empty_like(x)
    if r_out is not None:
        _expect("r_out", r_out, shape, dt, dev)
    sshape = shape[:-1] + (-(-d // group) if group > 0 else 1,)
    if out is None:
        out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
    else:
        _expect("out", out, shape, torch.float8_e4m3fn, dev)
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.float32, device=x.device)
    else:
        _expect("scales", scales, sshape, torch.float32, dev)
    _launch(_LIB.ffn_add_rmsnorm_e4m3, "ffn_add_rmsnorm_e4m3", dev, x.data_ptr(),
            None if res is None else res.data_ptr(), g.data_ptr(), None if r_out is None else r_out.data_ptr(),
            out.data_ptr(), scales.data_ptr(), rows, d, group, eps, code)
    return (x if r_out is None else r_out), out, scales


def ffn_moe_route(logits: torch.Tensor, k: int, bias: torch.Tensor | None = None, groups: int = 1,
                  topk_groups: int = 1, scale: float = 1.0, flags: int = 0, idx: torch.Tensor | None = None,
                  weights: torch.Tensor | None = None, stream=None):
    """(idx int32 [rows, k], weights fp32 [rows, k]) of a [rows, experts] tensor
    of router logits; flags: FFN_ROUTE_SIGMOID, FFN_ROUTE_RENORM.  A slot
    that no eligible expert is left for has index -1 and weight 0."""
    if stream is not None:   # outputs and workspaces made here belong to that stream
        with torch.cuda.stream(stream):
            return ffn_moe_route(logits, k, bias, groups, topk_groups, scale, flags, idx, weights)
    rows, experts, dev = _rows_of(logits)
    code = _dtype(logits)
    if bias is not None:
        _expect("bias", bias, (experts,), torch.float32, dev)
    shape = logits.shape[:-1] + (k,)
    if idx is None:
        idx = torch.empty(shape, dtype=torch.int32, device=logits.device)
    else:
        _expect("idx", idx, shape, torch.int32, dev)
    if weights is None:
        weights = torch.empty(shape, dtype=torch.float32, device=logits.device)
    else:
        _expect("weights", weights, shape, torch.float32, dev)
    _launch(_LIB.ffn_moe_route, "ffn_moe_route", dev, logits.data_ptr(),
            None if bias is None else bias.data_ptr(), idx.data_ptr(), weights.data_ptr(), rows, experts, k, groups,
            topk_groups, scale, code, flags)
    return idx, weights


def ffn_moe_workspace_bytes(rows: int, d: int, ffn: int, experts: int, k: int, dtype: torch.dtype,
                            flags: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_LIB.ffn_moe_workspace_bytes(rows, d, ffn, experts, k, _DT[dtype], flags, ctypes.byref(out)),
           "ffn_moe_workspace_bytes")
    return out.value


def _moe_inputs(x, idx, weights, res, out):
    """Checks what both routed blocks take; (rows, d, k, device index)."""
    rows, d, dev = _rows_of(x)
    k = idx.shape[-1]
    shape = x.shape[:-1] + (k,)
    _expect("idx", idx, shape, torch.int32, dev)
    _expect("weights", weights, shape, torch.float32, dev)
    if res is not None:
        _expect("res", res, x.shape, x.dtype, dev)
    if out is not None:
        _expect("out", out, x.shape, x.dtype, dev)
    return rows, d, k, dev


def ffn_moe_forward(x: torch.Tensor, idx: torch.Tensor, weights: torch.Tensor, w_gate: torch.Tensor,
                    w_up: torch.Tensor, w_down: torch.Tensor, res: torch.Tensor | None = None, flags: int = 0,
                    out: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The routed block: y = [res +] sum over a token's slots of weight * the
    chosen expert's SwiGLU block of x.  idx, weights: ffn_moe_route's [rows, k];
    w_gate, w_up [experts, ffn, d], w_down [experts, d, ffn] of x's type, or
    ffn_prepare_weights output with FFN_PREPARED_WEIGHTS."""
    if stream is not None:   # outputs and workspaces made here belong to that stream
        with torch.cuda.stream(stream):
            return ffn_moe_forward(x, idx, weights, w_gate, w_up, w_down, res, flags, out, ws)
    rows, d, k, dev = _moe_inputs(x, idx, weights, res, out)
    code = _dtype(x)
    experts, ffn = w_gate.shape[0], w_gate.shape[1]
    wt = torch.float16 if flags & FFN_PREPARED_WEIGHTS else x.dtype
    _expect("w_gate", w_gate, (experts, ffn, d), wt, dev)
    _expect("w_up", w_up, (experts, ffn, d), wt, dev)
    _expect("w_down", w_down, (experts, d, ffn), wt, dev)
    y = torch.empty_like(x) if out is None else out
    if ws is None:   # (a passed workspace is checked against the need by the C side)
        ws = workspace(ffn_moe_workspace_bytes(rows, d, ffn, experts, k, x.dtype, flags), x.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous CUDA tensor on the device of the input")
    _launch(_LIB.ffn_moe_forward, "ffn_moe_forward", dev, x.data_ptr(), idx.data_ptr(), weights.data_ptr(),
            w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), None if res is None else res.data_ptr(),
            y.data_ptr(), rows, d, ffn, experts, k, code, flags, ws.data_ptr(), ws.numel() * ws.element_size())
    return y


def ffn_moe_q4_workspace_bytes(rows: int, d: int, ffn: int, experts: int, k: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_LIB.ffn_moe_q4_workspace_bytes(rows, d, ffn, experts, k, ctypes.byref(out)), "ffn_moe_q4_workspace_bytes")
    return out.value


_F16_BITS = (torch.float16, torch.int16, torch.uint16)   # (bf16 has other bits)


def _moe_q4_weight(name, w, experts, out, inn, dev):
    qs, sc = w
    groups = -(-inn // 128)
    _expect(name + " qs", qs, (experts, out, 64 * groups), torch.uint8, dev)
    if sc.dtype not in _F16_BITS:
        raise TypeError(f"{name} scales must be fp16 or their 16-bit patterns, are {sc.dtype}")
    _expect(name + " scales", sc, (experts, out, 4 * groups), sc.dtype, dev)
    return Q4Weight(qs.data_ptr(), sc.data_ptr())


def ffn_moe_forward_q4(x: torch.Tensor, idx: torch.Tensor, weights: torch.Tensor, w_gate, w_up, w_down, ffn: int,
                       res: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """ffn_moe_forward (bf16) with Q4 weights: ``w_*`` are (qs uint8 [experts,
    rows, 64 ceil(in/128)], scales [experts, rows, 4 ceil(in/128)] fp16 or
    their bits) pairs in the device layout of include/ffn.h."""
    if stream is not None:   # outputs and workspaces made here belong to that stream
        with torch.cuda.stream(stream):
            return ffn_moe_forward_q4(x, idx, weights, w_gate, w_up, w_down, ffn, res, out, ws)
    rows, d, k, dev = _moe_inputs(x, idx, weights, res, out)
    if x.dtype is not torch.bfloat16:
        raise TypeError("x must be torch.bfloat16")
    experts = w_gate[0].shape[0]
    wg = _moe_q4_weight("w_gate", w_gate, experts, ffn, d, dev)
    wu = _moe_q4_weight("w_up", w_up, experts, ffn, d, dev)
    wd = _moe_q4_weight("w_down", w_down, experts, d, ffn, dev)
    y = torch.empty_like(x) if out is None else out
    if ws is None:
        ws = workspace(ffn_moe_q4_workspace_bytes(rows, d, ffn, experts, k), x.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous CUDA tensor on the device of the input")
    _launch(_LIB.ffn_moe_forward_q4, "ffn_moe_forward_q4", dev, x.data_ptr(), idx.data_ptr(), weights.data_ptr(),
            wg, wu, wd, None if res is None else res.data_ptr(), y.data_ptr(), rows, d, ffn, experts, k,
            ws.data_ptr(), ws.numel() * ws.element_size())
    return y


def ffn_rmsnorm(x: torch.Tensor, g: torch.Tensor, eps: float, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    _need_cuda(x, g, out)
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    n = torch.empty_like(x) if out is None else out
    _check(_lib.load().ffn_rmsnorm(_ptr(x), _ptr(g), _ptr(n), rows, d, float(eps), _dtype(x),
                                   _stream(stream)), "ffn_rmsnorm")
    return n


def ffn_swiglu(gate: torch.Tensor, up: torch.Tensor, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    _need_cuda(gate, up, out)
    h = torch.empty_like(gate) if out is None else out
    _check(_lib.load().ffn_swiglu(_ptr(gate), _ptr(up), _ptr(h), gate.numel(), _dtype(gate),
                                  _stream(stream)), "ffn_swiglu")
    return h


def ffn_block_workspace_bytes(rows: int, d: int, ffn: int, dtype: torch.dtype, flags: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.load().ffn_block_workspace_bytes(rows, d, ffn, _DT[dtype], flags, ctypes.byref(out)),
           "ffn_block_workspace_bytes")
    return out.value


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def ffn_block_forward(x, g, w_gate, w_up, w_down, eps: float, flags: int = 0, out=None,
                      ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _need_cuda(x, g, w_gate, w_up, w_down, out, ws)
    d = x.shape[-1]
    rows = x.numel() // d
    ffn = w_gate.shape[0]
    y = torch.empty_like(x) if out is None else out
    if ws is None:   # (a passed workspace is checked against the need by the C side)
        ws = workspace(ffn_block_workspace_bytes(rows, d, ffn, x.dtype, flags), x.device)
    _check(_lib.load().ffn_block_forward(_ptr(x), _ptr(g), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                         _ptr(y), rows, d, ffn, float(eps), _dtype(x), flags,
                                         _ptr(ws), ws.numel(), _stream(stream)), "ffn_block_forward")
    return y


def ffn_block_forward_chained(x, g, w_gate, w_up, w_down, eps: float, flags: int = 0, x_sumsq=None,
                              y_sumsq: bool = True, out=None, ss_out=None, ws: torch.Tensor | None = None,
                              stream=None):
    """ffn_block_forward that takes each row's sum of squares of x (x_sumsq,
    fp32 [rows], or None) and returns (y, y_sumsq): the rows' sums of squares
    of the stored y (None unless y_sumsq)."""
    _need_cuda(x, g, w_gate, w_up, w_down, out, ws, x_sumsq, ss_out)
    d = x.shape[-1]
    rows = x.numel() // d
    ffn = w_gate.shape[0]
    y = torch.empty_like(x) if out is None else out
    ss = None
    if y_sumsq:
        ss = torch.empty(rows, dtype=torch.float32, device=x.device) if ss_out is None else ss_out
    if ws is None:
        ws = workspace(ffn_block_workspace_bytes(rows, d, ffn, x.dtype, flags), x.device)
    _check(_lib.load().ffn_block_forward_chained(_ptr(x), _ptr(x_sumsq), _ptr(g), _ptr(w_gate), _ptr(w_up),
                                                 _ptr(w_down), _ptr(y), _ptr(ss), rows, d, ffn, float(eps),
                                                 _dtype(x), flags, _ptr(ws), ws.numel(), _stream(stream)),
           "ffn_block_forward_chained")
    return y, ss


def ffn_block_host_workspace_bytes(rows: int, d: int, ffn: int, dtype, flags: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.load().ffn_block_host_workspace_bytes(rows, d, ffn, _DT[dtype], flags, ctypes.byref(out)),
           "ffn_block_host_workspace_bytes")
    return out.value


def ffn_block_forward_host(x_host, g, w_gate, w_up, w_down, eps: float, flags: int = 0, out=None,
                           ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The block with x and y in host memory (page-locked tensors overlap their
    copies with the compute); weights, g and the workspace on the device.
    Returns y on the host once `stream` (default: the current one) has passed
    the call; synchronise it before reading."""
    _need_cuda(g, w_gate, w_up, w_down, ws)
    if x_host.is_cuda or (out is not None and out.is_cuda):
        raise ValueError("x_host and out must be host tensors")
    if not x_host.is_contiguous() or (out is not None and not out.is_contiguous()):
        raise ValueError("x_host and out must be contiguous")
    d = x_host.shape[-1]
    rows = x_host.numel() // d
    ffn = w_gate.shape[0]
    y = torch.empty(x_host.shape, dtype=x_host.dtype, pin_memory=True) if out is None else out
    if ws is None:
        ws = workspace(ffn_block_host_workspace_bytes(rows, d, ffn, x_host.dtype, flags), g.device)
    _check(_lib.load().ffn_block_forward_host(_ptr(x_host), _ptr(g), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                              _ptr(y), rows, d, ffn, float(eps), _dtype(x_host), flags,
                                              _ptr(ws), ws.numel(), _stream(stream)), "ffn_block_forward_host")
    return y


def ffn_prepare_weights(w: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One-time re-encoding of a bf16/fp16 weight for FFN_PREPARED_WEIGHTS
    (fp16 values of w * 2^8)."""
    _need_cuda(w, out)
    dst = torch.empty(w.shape, dtype=torch.float16, device=w.device) if out is None else out
    _check(_lib.load().ffn_prepare_weights(_ptr(w), _ptr(dst), w.numel(), _dtype(w), _stream(stream)),
           "ffn_prepare_weights")
    return dst


def ffn_prepare_weights_fp8(w, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prepared fp16 weights (values of e4m3 * row scale * 2^8) from a
    (codes [out, in], scales [out]) pair, for FFN_PREPARED_WEIGHTS."""
    codes, _ = w
    o, i = codes.shape
    dst = torch.empty((o, i), dtype=torch.float16, device=codes.device) if out is None else out
    _need_cuda(dst)
    _check(_lib.load().ffn_prepare_weights_fp8(_fp8(w), _ptr(dst), o, i, _stream(stream)), "ffn_prepare_weights_fp8")
    return dst


def ffn_prepare_weights_q4(w, inn: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prepared fp16 weights (values of (u - 8) * s * 2^8) from a Q4 (qs,
    scales) pair in the device layout; `inn` is the input dimension."""
    qs, _ = w
    o = qs.shape[0]
    dst = torch.empty((o, inn), dtype=torch.float16, device=qs.device) if out is None else out
    _need_cuda(dst)
    _check(_lib.load().ffn_prepare_weights_q4(_q4(w), _ptr(dst), o, inn, _stream(stream)), "ffn_prepare_weights_q4")
    return dst


def ffn_block_q4_workspace_bytes(rows: int, d: int, ffn: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.load().ffn_block_q4_workspace_bytes(rows, d, ffn, ctypes.byref(out)),
           "ffn_block_q4_workspace_bytes")
    return out.value


def _q4(w):
    qs, sc = w
    _need_cuda(qs, sc)
    return Q4Weight(qs.data_ptr(), sc.data_ptr())


def ffn_block_forward_q4(x, g, w_gate, w_up, w_down, ffn: int, eps: float, flags: int = 0,
                         out=None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``w_*`` are (qs uint8, scales int16/uint16-bits) CUDA tensor pairs in the
    device layout of include/ffn.h."""
    _need_cuda(x, g, out, ws)
    d = x.shape[-1]
    rows = x.numel() // d
    y = torch.empty_like(x) if out is None else out
    if ws is None:
        ws = workspace(ffn_block_q4_workspace_bytes(rows, d, ffn), x.device)
    _check(_lib.load().ffn_block_forward_q4(_ptr(x), _ptr(g), _q4(w_gate), _q4(w_up), _q4(w_down),
                                            _ptr(y), rows, d, ffn, float(eps), flags, _ptr(ws),
                                            ws.numel(), _stream(stream)), "ffn_block_forward_q4")
    return y


def ffn_block_fp8_workspace_bytes(rows: int, d: int, ffn: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.load().ffn_block_fp8_workspace_bytes(rows, d, ffn, ctypes.byref(out)),
           "ffn_block_fp8_workspace_bytes")
    return out.value


def _fp8(w):
    codes, sc = w
    _need_cuda(codes, sc)
    if codes.element_size() != 1 or sc.dtype != torch.float32:
        raise TypeError("e4m3 weights are (1-byte codes, float32 row scales)")
    return Fp8Weight(codes.data_ptr(), sc.data_ptr())


def ffn_block_forward_fp8(x, g, w_gate, w_up, w_down, eps: float, flags: int = 0,
                          out=None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``w_*`` are (codes, scales) CUDA tensor pairs: e4m3 codes [out, in]
    (uint8 or torch.float8_e4m3fn) and float32 row scales [out]."""
    _need_cuda(x, g, out, ws)
    d = x.shape[-1]
    rows = x.numel() // d
    ffn = w_gate[0].shape[0]
    y = torch.empty_like(x) if out is None else out
    if ws is None:
        ws = workspace(ffn_block_fp8_workspace_bytes(rows, d, ffn), x.device)
    _check(_lib.load().ffn_block_forward_fp8(_ptr(x), _ptr(g), _fp8(w_gate), _fp8(w_up), _fp8(w_down),
                                             _ptr(y), rows, d, ffn, float(eps), flags, _ptr(ws),
                                             ws.numel(), _stream(stream)), "ffn_block_forward_fp8")
    return y


def ffn_block_q8_workspace_bytes(rows: int, d: int, ffn: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.load().ffn_block_q8_workspace_bytes(rows, d, ffn, ctypes.byref(out)),
           "ffn_block_q8_workspace_bytes")
    return out.value


def _q8(w):
    codes, sc = w
    _need_cuda(codes, sc)
    if codes.element_size() != 1 or sc.element_size() != 2:
        raise TypeError("Q8_0 weights are (1-byte codes, 2-byte fp16 scale bits)")
    return Q8Weight(codes.data_ptr(), sc.data_ptr())


def ffn_block_forward_q8(x, g, w_gate, w_up, w_down, eps: float, flags: int = 0,
                         out=None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``w_*`` are (codes int8 [out, in], scales [out, in/32] fp16 or their
    int16 bits) CUDA tensor pairs."""
    _need_cuda(x, g, out, ws)
    d = x.shape[-1]
    rows = x.numel() // d
    ffn = w_gate[0].shape[0]
    y = torch.empty_like(x) if out is None else out
    if ws is None:
        ws = workspace(ffn_block_q8_workspace_bytes(rows, d, ffn), x.device)
    _check(_lib.load().ffn_block_forward_q8(_ptr(x), _ptr(g), _q8(w_gate), _q8(w_up), _q8(w_down),
                                            _ptr(y), rows, d, ffn, float(eps), flags, _ptr(ws),
                                            ws.numel(), _stream(stream)), "ffn_block_forward_q8")
    return y


def ffn_prepare_weights_q8(w, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prepared fp16 weights (values of q * s * 2^8) from a Q8_0 (codes,
    scales) pair, for FFN_PREPARED_WEIGHTS."""
    codes, _ = w
    o, i = codes.shape
    dst = torch.empty((o, i), dtype=torch.float16, device=codes.device) if out is None else out
    _need_cuda(dst)
    _check(_lib.load().ffn_prepare_weights_q8(_q8(w), _ptr(dst), o, i, _stream(stream)), "ffn_prepare_weights_q8")
    return dst


def ffn_q4_pack_host(q: np.ndarray, scales_bits: np.ndarray):
    """Host packer: int8 q [out, in] in [-8, 7] and fp16 scale bits [out, in/32]
    into the device layout (rows of ceil(in/128) 64-byte groups, 4 scales a
    group)."""
    q = np.ascontiguousarray(q, dtype=np.int8)
    s = np.ascontiguousarray(scales_bits).view(np.uint16)
    out, inn = q.shape
    ngrp = -(-inn // 128)
    qs = np.empty((out, 64 * ngrp), dtype=np.uint8)
    so = np.empty((out, 4 * ngrp), dtype=np.uint16)
    _check(_lib.load().ffn_q4_pack_host(q.ctypes.data, s.ctypes.data, out, inn, qs.ctypes.data,
                                        so.ctypes.data), "ffn_q4_pack_host")
    return qs, so


def ffn_device_status():
    _check(_lib.load().ffn_device_status(), "ffn_device_status")


def ffn_selftest_bounded_wait(limit_ns: int = 2_000_000, stream=None):
    """Launch the bounded-wait self test: a wait that nothing completes gives
    up after limit_ns and the next ffn_device_status() raises FFN_ERR_TIMEOUT."""
    _check(_lib.load().ffn_selftest_bounded_wait(int(limit_ns), _stream(stream)), "ffn_selftest_bounded_wait")


def ffn_launch_count() -> int:
    return int(_lib.load().ffn_launch_count())


class KernelTimer:
    """Per-kernel device time from CUDA events recorded around each launch."""

    def __init__(self):
        self.lib = _lib.load()

    def __enter__(self):
        _check(self.lib.ffn_timing_reset(), "ffn_timing_reset")
        _check(self.lib.ffn_timing_enable(1), "ffn_timing_enable")
        return self

    def __exit__(self, *exc):
        self.lib.ffn_timing_enable(0)
        return False

    def read(self) -> dict:
        _check(self.lib.ffn_timing_collect(), "ffn_timing_collect")
        res = {}
        for k in range(self.lib.ffn_kernel_kinds()):
            n = ctypes.c_uint64(0)
            ms = ctypes.c_double(0.0)
            _check(self.lib.ffn_timing_read(k, ctypes.byref(n), ctypes.byref(ms)), "ffn_timing_read")
            if n.value:
                res[self.lib.ffn_kernel_name(k).decode()] = (int(n.value), float(ms.value))
        return res
