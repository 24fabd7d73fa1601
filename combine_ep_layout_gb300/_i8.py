"""ctypes binding of the int8 path (include/ep_gb300_i8.h): rows to int8, the int8
dispatch, and products of int8 rows with int8 weights, dense or grouped by
expert.  Argument checks and marshalling only, as in _native.
"""
import ctypes

import torch

from ._moe import _ACTS, _FLOATS, _NOT_CURRENT, _current_device, _is, _stream
from ._native import _check, _require, load_library

EP_ACT_NONE = -1
EP_I8_MAX_COLS = 65536

_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    L = load_library()
    c = ctypes
    vp, i32, i64 = c.c_void_p, c.c_int32, c.c_int64
    L.ep_i8_quantize.argtypes = [vp, vp, i32, i64, i64, i32, vp, vp, vp]
    L.ep_i8_dispatch.argtypes = [vp, vp, i32, vp, vp, vp]
    L.ep_i8_linear.argtypes = [vp, vp, i32, vp, vp, i32, i32, i32, vp, i32, vp]
    L.ep_i8_grouped.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp]
    L.ep_i8_status.argtypes = [c.POINTER(i32), vp]
    for f in (L.ep_i8_quantize, L.ep_i8_dispatch, L.ep_i8_linear, L.ep_i8_grouped, L.ep_i8_status):
        f.restype = c.c_int
    _lib = L
    return L


def _act(activation):
    if activation is None:
        return EP_ACT_NONE
    _require(activation in _ACTS, "activation must be None, 'silu' or 'gelu_tanh'")
    return _ACTS[activation]


def ep_i8_quantize(x, q, scales, only_of=None, stream=None):
    """Rows to int8: scales[t] = max|x[t]| / 127, q[t] = x[t] / scales[t] rounded to
    nearest even.  x: bf16 or fp32 [n, cols] (contiguous rows at any row stride); q: int8
    [n, cols]; scales: fp32 [n].  only_of: an EpHandle whose receive rows x has; rows
    that receive nothing are neither read nor written."""
    device, shape = x.get_device(), x.shape
    _require(device >= 0 and len(shape) == 2 and x.dtype in _FLOATS,
             "x must be a bf16 or fp32 CUDA tensor [n, cols]")
    _require(x.stride(1) == 1 or shape[1] == 1 or shape[0] == 0, "x must have contiguous rows")
    _require(device == _current_device(), _NOT_CURRENT)
    n, cols = shape
    _require(_is(q, torch.int8, shape, device), "q must be a contiguous int8 CUDA tensor of x's shape and device")
    _require(_is(scales, torch.float32, (n,), device),
             "scales must be a contiguous fp32 CUDA tensor [n] on the device of x")
    stride = x.stride(0) if n > 1 else max(x.stride(0), cols)
    _check(_load().ep_i8_quantize(only_of.ptr if only_of is not None else None, x.data_ptr(), _FLOATS[x.dtype],
                                  stride, n, cols, q.data_ptr(), scales.data_ptr(), _stream(stream, device)))


def ep_i8_dispatch(h, x, recv_q, recv_scales, stream=None):
    """x [N, H] (bf16 or fp32) quantised as by ep_i8_quantize, each row written to every receive
    row of its token: recv_q int8 [Rcap, H], recv_scales fp32 [Rcap]."""
    cfg, device = h.cfg, h.device
    _require(x.dtype in _FLOATS and _is(x, x.dtype, (_tokens(h), cfg.hidden_dim), device),
             "x must be a contiguous bf16 or fp32 CUDA tensor [num_tokens, hidden] on the handle's device")
    _require(_is(recv_q, torch.int8, (h.recv_capacity, cfg.hidden_dim), device),
             "recv_q must be a contiguous int8 CUDA tensor [recv_capacity, hidden] on the handle's device")
    _require(_is(recv_scales, torch.float32, (h.recv_capacity,), device),
             "recv_scales must be a contiguous fp32 CUDA tensor [recv_capacity] on the handle's device")
    _check(_load().ep_i8_dispatch(h.ptr, x.data_ptr(), _FLOATS[x.dtype], recv_q.data_ptr(),
                                  recv_scales.data_ptr(), _stream(stream, device)))


def _tokens(h):
    """Tokens of the layout that h uses."""
    while h._layout_of is not None:
        h = h._layout_of
    return h.num_tokens


def _out(out, n, rows, act, device):
    _require(act == EP_ACT_NONE or rows % 2 == 0, "a gated product has an even number of weight rows")
    width = rows if act == EP_ACT_NONE else rows // 2
    _require(out.dtype in _FLOATS and _is(out, out.dtype, (n, width), device),
             "out must be a contiguous bf16 or fp32 CUDA tensor [n, rows] (gated: [n, rows / 2]) on the device of x")


def ep_i8_linear(x, x_scales, w, w_scales, out, activation=None, stream=None):
    """out[t, r] = x_scales[t] w_scales[r] sum_c x[t, c] w[r, c]: x int8 [n, cols], w int8
    [rows, cols], scales fp32 [n] and [rows], out bf16 or fp32.  With an activation
    ("silu", "gelu_tanh") w's first half is the gate and its second the up projection:
    out[n, rows / 2] = act(gate) * up."""
    _require(x.dim() == 2 and w.dim() == 2, "x and w must be 2-D")
    n, cols = x.shape
    rows, device, act = w.shape[0], x.get_device(), _act(activation)
    _require(device >= 0 and _is(x, torch.int8, (n, cols), device), "x must be a contiguous int8 CUDA tensor [n, cols]")
    _require(device == _current_device(), _NOT_CURRENT)
    _require(_is(w, torch.int8, (rows, cols), device),
             "w must be a contiguous int8 CUDA tensor [rows, cols] on the device of x")
    _require(_is(x_scales, torch.float32, (n,), device),
             "x_scales must be a contiguous fp32 CUDA tensor [n] on the device of x")
    _require(_is(w_scales, torch.float32, (rows,), device),
             "w_scales must be a contiguous fp32 CUDA tensor [rows] on the device of x")
    _out(out, n, rows, act, device)
    _check(_load().ep_i8_linear(x.data_ptr(), x_scales.data_ptr(), n, w.data_ptr(), w_scales.data_ptr(), rows, cols,
                                act, out.data_ptr(), _FLOATS[out.dtype], _stream(stream, device)))


def ep_i8_grouped(h, x, x_scales, w, w_scales, out, activation=None, stream=None):
    """ep_i8_linear of each expert's receive rows with its own weights: x int8 [Rcap, cols],
    x_scales fp32 [Rcap], w int8 [E, rows, cols], w_scales fp32 [E, rows], out [Rcap, rows]
    (gated: [Rcap, rows / 2]).  Padding rows are left as they are."""
    _require(x.dim() == 2 and w.dim() == 3, "x must be 2-D and w 3-D")
    n, cols = x.shape
    experts, rows, device, act = h.cfg.world_size * h.cfg.num_expert_per_rank, w.shape[1], h.device, _act(activation)
    _require(_is(x, torch.int8, (h.recv_capacity, cols), device),
             "x must be a contiguous int8 CUDA tensor [recv_capacity, cols] on the handle's device")
    _require(_is(x_scales, torch.float32, (n,), device),
             "x_scales must be a contiguous fp32 CUDA tensor [recv_capacity] on the handle's device")
    _require(_is(w, torch.int8, (experts, rows, cols), device),
             "w must be a contiguous int8 CUDA tensor [experts, rows, cols] on the handle's device")
    _require(_is(w_scales, torch.float32, (experts, rows), device),
             "w_scales must be a contiguous fp32 CUDA tensor [experts, rows] on the handle's device")
    _out(out, n, rows, act, device)
    _check(_load().ep_i8_grouped(h.ptr, x.data_ptr(), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), rows,
                                 cols, act, out.data_ptr(), _FLOATS[out.dtype], _stream(stream, device)))


def ep_i8_status(stream=None):
    """Read and clear the products' error word of the current device (waits for the stream)."""
    v = ctypes.c_int32()
    _check(_load().ep_i8_status(ctypes.byref(v), _stream(stream, _current_device())))
    return v.value
