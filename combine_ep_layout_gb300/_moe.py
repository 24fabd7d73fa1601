"""ctypes binding of the decode-side MoE operators (include/ep_gb300_moe.h): the
router and its gradient, products with 4-bit weights, and a whole MoE layer for
a few tokens.  Argument checks and marshalling only, as in _native.
"""
import ctypes

import torch

from ._native import (EP_BF16, EP_EINVAL, EP_FP32, EpError, _check, _ptr, _require,
                      load_library)

EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
EP_INT4X2 = 4
EP_ACT_SILU, EP_ACT_GELU_TANH = 0, 1
EP_FEW_TOKENS = 64

_SCORES = {"softmax": EP_SCORE_SOFTMAX, "sigmoid": EP_SCORE_SIGMOID}
_WEIGHTS = {"bf16": EP_BF16, "int4": EP_INT4X2, "int4x2": EP_INT4X2}
_ACTS = {"silu": EP_ACT_SILU, "gelu_tanh": EP_ACT_GELU_TANH}
_FLOATS = {torch.bfloat16: EP_BF16, torch.float32: EP_FP32}


class ep_route_cfg_t(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class ep_moe_cfg_t(ctypes.Structure):
    _fields_ = [("hidden_dim", ctypes.c_int32), ("intermediate_dim", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("num_expert_per_token", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("activation", ctypes.c_int32)]


class ep_moe_weights_t(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_scales", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_scales", ctypes.c_void_p)]


# the current stream's handle without a Stream object (2 us a call less)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# the current device's index without the lazy set-up, which a CUDA tensor has been through
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

# a call without a handle launches on the current device
_NOT_CURRENT = "the tensors are not on the current device"


def _stream(stream, index):
    if stream is None:
        return _raw_stream(index)
    _require(stream.device_index == index, "the stream is not of the tensors' device")
    return stream.cuda_stream


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    L = load_library()
    c = ctypes
    vp, i32, i64 = c.c_void_p, c.c_int32, c.c_int64
    rc, mw = c.POINTER(ep_route_cfg_t), c.POINTER(ep_moe_weights_t)
    L.ep_route.argtypes = [rc, vp, i32, i64, vp, i32, vp, vp, vp]
    L.ep_route_backward.argtypes = [rc, vp, i32, i64, vp, vp, i32, vp, i64, vp]
    L.ep_w4_linear.argtypes = [vp, i32, vp, vp, i32, i32, i32, vp, i32, vp]
    L.ep_moe_create.argtypes = [c.POINTER(ep_moe_cfg_t), c.POINTER(vp)]
    L.ep_moe_forward.argtypes = [vp, vp, i32, vp, vp, mw, vp, vp, i32, vp]
    L.ep_moe_layer.argtypes = [vp, rc, vp, i32, vp, i32, i64, vp, mw, vp, vp, vp, vp, i32, vp]
    L.ep_moe_status.argtypes = [vp, c.POINTER(i32)]
    L.ep_moe_free.argtypes = [vp]
    L.ep_moe_free.restype = None
    for f in (L.ep_route, L.ep_route_backward, L.ep_w4_linear, L.ep_moe_create, L.ep_moe_forward,
              L.ep_moe_layer, L.ep_moe_status):
        f.restype = c.c_int
    _lib = L
    return L


def _is(t, dtype, shape, device):
    return t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()


# ------------------------------------------------------------------ router

def make_route_cfg(num_experts, topk, score="softmax", renormalize=True, scale=1.0):
    s = _SCORES[score] if isinstance(score, str) else int(score)
    return ep_route_cfg_t(num_experts, topk, s, int(bool(renormalize)), scale)


def _logits(cfg, logits, what):
    """Rows, row stride and device of scores or their gradient."""
    device, shape, experts = logits.get_device(), logits.shape, cfg.num_experts
    if device < 0 or len(shape) != 2 or shape[1] != experts or logits.dtype not in _FLOATS:
        raise ValueError("%s must be a bf16 or fp32 CUDA tensor [n, num_experts]" % what)
    n, stride = shape[0], logits.stride(0)
    if logits.stride(1) != 1 and experts != 1 and n != 0:
        raise ValueError("%s must have contiguous rows" % what)
    # a single row may carry any stride; rows may not overlap
    return n, stride if n > 1 else max(stride, experts), device


def ep_route(cfg, logits, topk_idx, topk_weights, select_bias=None, stream=None):
    """Scores [n, E] (bf16 or fp32, contiguous rows at any row stride) to the
    topk_idx (int64) and topk_weights (fp32) [n, K] that layout and combine take."""
    n, stride, device = _logits(cfg, logits, "logits")
    shape = (n, cfg.topk)
    _require(device == _current_device(), _NOT_CURRENT)
    _require(_is(topk_idx, torch.int64, shape, device),
             "topk_idx must be a contiguous int64 CUDA tensor [n, topk] on the device of logits")
    _require(_is(topk_weights, torch.float32, shape, device),
             "topk_weights must be a contiguous fp32 CUDA tensor [n, topk] on the device of logits")
    _require(select_bias is None or _is(select_bias, torch.float32, (cfg.num_experts,), device),
             "select_bias must be a contiguous fp32 CUDA tensor [num_experts] on the device of logits")
    _check(_load().ep_route(cfg, logits.data_ptr(), _FLOATS[logits.dtype], stride, _ptr(select_bias),
                            n, topk_idx.data_ptr(), topk_weights.data_ptr(), _stream(stream, device)))


def ep_route_backward(cfg, logits, topk_idx, grad_weights, grad_logits, stream=None):
    """Gradient of ep_route's topk_weights: grad_weights fp32 [n, K] in,
    grad_logits [n, E] of the logits' type out (every element written)."""
    n, stride, device = _logits(cfg, logits, "logits")
    gn, gstride, gdevice = _logits(cfg, grad_logits, "grad_logits")
    shape = (n, cfg.topk)
    _require(device == _current_device(), _NOT_CURRENT)
    _require(grad_logits.dtype is logits.dtype and gn == n and gdevice == device,
             "grad_logits must have the type, shape and device of logits")
    _require(_is(topk_idx, torch.int64, shape, device),
             "topk_idx must be a contiguous int64 CUDA tensor [n, topk] on the device of logits")
    _require(_is(grad_weights, torch.float32, shape, device),
             "grad_weights must be a contiguous fp32 CUDA tensor [n, topk] on the device of logits")
    _check(_load().ep_route_backward(cfg, logits.data_ptr(), _FLOATS[logits.dtype], stride,
                                     topk_idx.data_ptr(), grad_weights.data_ptr(), n,
                                     grad_logits.data_ptr(), gstride, _stream(stream, device)))


# ----------------------------------------------------------- 4-bit weights

def ep_w4_linear(x, qweight, scales, out, stream=None):
    """out[n, rows] = x[n, cols] . W^T for up to 64 tokens.  qweight: uint8
    [rows, cols/2] (low nibble: the even column, value nibble - 8); scales: fp32
    [rows, cols/group] with group 32, 64 or 128; x bf16, out bf16 or fp32."""
    _require(x.dim() == 2 and qweight.dim() == 2 and scales.dim() == 2, "x, qweight and scales must be 2-D")
    n, cols = x.shape
    rows, groups = scales.shape
    device = x.get_device()
    _require(x.dtype is torch.bfloat16 and device >= 0 and x.is_contiguous(),
             "x must be a contiguous bf16 CUDA tensor [n, cols]")
    _require(device == _current_device(), _NOT_CURRENT)
    _require(cols % 2 == 0 and _is(qweight, torch.uint8, (rows, cols // 2), device),
             "qweight must be a contiguous uint8 CUDA tensor [rows, cols / 2] on the device of x")
    _require(groups > 0 and cols % groups == 0 and _is(scales, torch.float32, (rows, groups), device),
             "scales must be a contiguous fp32 CUDA tensor [rows, cols / group_size] on the device of x")
    _require(out.dtype in _FLOATS and _is(out, out.dtype, (n, rows), device),
             "out must be a contiguous bf16 or fp32 CUDA tensor [n, rows] on the device of x")
    _check(_load().ep_w4_linear(x.data_ptr(), n, qweight.data_ptr(), scales.data_ptr(), rows, cols,
                                cols // groups, out.data_ptr(), _FLOATS[out.dtype],
                                _stream(stream, device)))


# --------------------------------------------- MoE layer for a few tokens

def make_moe_cfg(hidden_dim, intermediate_dim, num_experts, num_expert_per_token,
                 max_tokens=EP_FEW_TOKENS, weight_dtype="bf16", group_size=0, activation="silu"):
    wd = _WEIGHTS[weight_dtype] if isinstance(weight_dtype, str) else int(weight_dtype)
    act = _ACTS[activation] if isinstance(activation, str) else int(activation)
    return ep_moe_cfg_t(hidden_dim, intermediate_dim, num_experts, num_expert_per_token, max_tokens,
                        wd, group_size, act)


class EpMoeWeights:
    """The experts' weights: w13 [E, 2I, H] (gate rows, then up rows) and w2
    [E, H, I], both bf16, or both uint8 of the 4-bit form with fp32 scales
    [E, 2I, H/group] and [E, H, I/group].  Keeps the tensors alive."""

    def __init__(self, w13, w2, w13_scales=None, w2_scales=None):
        self.tensors = (w13, w2, w13_scales, w2_scales)
        self.device = w13.get_device()
        for t in self.tensors:
            _require(t is None or (t.is_cuda and t.is_contiguous() and t.dim() == 3),
                     "weights and scales must be contiguous 3-D CUDA tensors")
            _require(t is None or t.get_device() == self.device, "weights and scales must be on one device")
        _require((w13_scales is None) == (w2_scales is None),
                 "w13_scales and w2_scales come together")
        q = w13_scales is not None
        _require(w13.dtype == w2.dtype == (torch.uint8 if q else torch.bfloat16),
                 "w13 and w2 must be bf16, or uint8 with scales")
        _require(not q or w13_scales.dtype == w2_scales.dtype == torch.float32, "scales must be fp32")
        E, H = w2.shape[0], w2.shape[1]
        I = w13.shape[1] // 2
        per = 2 if q else 1
        g = H // max(1, w13_scales.shape[2]) if q else 0
        want = [(w13, (E, 2 * I, H // per)), (w2, (E, H, I // per))]
        if q:
            want += [(w13_scales, (E, 2 * I, H // max(g, 1))), (w2_scales, (E, H, I // max(g, 1)))]
        for t, shape in want:
            _require(tuple(t.shape) == shape, "weights have shape %s, expected %s" % (tuple(t.shape), shape))
        self.int4 = q
        self.dims = (E, H, I, g)
        self.c = ep_moe_weights_t(w13.data_ptr(), _ptr(w13_scales), w2.data_ptr(), _ptr(w2_scales))

    def check(self, cfg):
        """Raise unless the weights are those of cfg."""
        _require(self.int4 == (cfg.weight_dtype == EP_INT4X2), "weights are not of the handle's weight_dtype")
        _require(self.dims == (cfg.num_experts, cfg.hidden_dim, cfg.intermediate_dim, cfg.group_size),
                 "weights are (experts, hidden, intermediate, group) %s, expected those of the handle" % (self.dims,))


class EpMoe:
    """Owner of an ep_moe_t: the experts of a few tokens (forward), or the whole
    layer with its router (layer).  Equal inputs give equal bits."""

    def __init__(self, cfg):
        self.cfg = cfg
        self._m = None
        self.device = torch.cuda.current_device()
        m = ctypes.c_void_p()
        _check(_load().ep_moe_create(ctypes.byref(cfg), ctypes.byref(m)))
        self._m = m

    @property
    def ptr(self):
        if self._m is None:
            raise EpError(EP_EINVAL, "handle already freed")
        return self._m

    def _args(self, x, weights, topk_idx, topk_weights, out, bias):
        n, cfg, device = x.shape[0], self.cfg, self.device
        _require(_is(x, torch.bfloat16, (n, cfg.hidden_dim), device),
                 "x must be a contiguous bf16 CUDA tensor [n, hidden] on the handle's device")
        shape = (n, cfg.num_expert_per_token)
        _require(_is(topk_idx, torch.int64, shape, device),
                 "topk_idx must be a contiguous int64 CUDA tensor [n, topk] on the handle's device")
        _require(_is(topk_weights, torch.float32, shape, device),
                 "topk_weights must be a contiguous fp32 CUDA tensor [n, topk] on the handle's device")
        _require(out.dtype in _FLOATS and _is(out, out.dtype, x.shape, device),
                 "out must be a contiguous bf16 or fp32 CUDA tensor [n, hidden] on the handle's device")
        _require(bias is None or _is(bias, torch.bfloat16, x.shape, device),
                 "bias must be a contiguous bf16 CUDA tensor [n, hidden] on the handle's device")
        _require(weights.device == device, "the weights are not on the handle's device")
        weights.check(cfg)
        return n

    def forward(self, x, topk_idx, topk_weights, weights, out, bias=None, stream=None):
        """out[t] = sum_k topk_weights[t,k] * W2[e] (act(W1[e] x[t]) * W3[e] x[t]) (+ bias[t])."""
        n = self._args(x, weights, topk_idx, topk_weights, out, bias)
        _check(_load().ep_moe_forward(self.ptr, x.data_ptr(), n, topk_idx.data_ptr(),
                                      topk_weights.data_ptr(), weights.c, _ptr(bias), out.data_ptr(),
                                      _FLOATS[out.dtype], _stream(stream, self.device)))

    def layer(self, route_cfg, x, logits, weights, topk_idx, topk_weights, out, bias=None,
              select_bias=None, stream=None):
        """ep_route of logits into topk_idx and topk_weights, then forward with them."""
        n = self._args(x, weights, topk_idx, topk_weights, out, bias)
        rows, stride, device = _logits(route_cfg, logits, "logits")
        _require(rows == n and device == self.device,
                 "logits must have a row for each row of x, on its device")
        _require(select_bias is None or _is(select_bias, torch.float32, (route_cfg.num_experts,), self.device),
                 "select_bias must be a contiguous fp32 CUDA tensor [num_experts] on the handle's device")
        _check(_load().ep_moe_layer(self.ptr, route_cfg, x.data_ptr(), n, logits.data_ptr(),
                                    _FLOATS[logits.dtype], stride, _ptr(select_bias), weights.c,
                                    _ptr(bias), topk_idx.data_ptr(), topk_weights.data_ptr(),
                                    out.data_ptr(), _FLOATS[out.dtype], _stream(stream, self.device)))

    def status(self):
        v = ctypes.c_int32()
        _check(_load().ep_moe_status(self.ptr, ctypes.byref(v)))
        return v.value

    def free(self):
        if self._m is not None:
            _load().ep_moe_free(self._m)
            self._m = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
