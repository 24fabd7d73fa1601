"""ctypes binding of the router's training losses (include/ep_gb300_balance.h): the
load-balance and z losses, the experts' token counts, and the gradient of the
scores.  Argument checks and marshalling only, as in _native.
"""
import ctypes

import torch

from ._moe import _FLOATS, _is, _logits, _stream, ep_route_cfg_t
from ._native import EP_EINVAL, EpError, _check, _ptr, _require, load_library

_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    L = load_library()
    c = ctypes
    vp, i32, i64 = c.c_void_p, c.c_int32, c.c_int64
    L.ep_balance_create.argtypes = [c.POINTER(ep_route_cfg_t), i32, i32, c.POINTER(vp)]
    L.ep_balance_forward.argtypes = [vp, vp, i32, i64, vp, i32, vp, i32, vp, vp, vp, vp, vp]
    L.ep_balance_backward.argtypes = [vp, vp, i32, i64, vp, i32, vp, i32, vp, vp, vp, vp, i64, i32, vp]
    L.ep_balance_free.argtypes = [vp]
    L.ep_balance_free.restype = None
    for f in (L.ep_balance_create, L.ep_balance_forward, L.ep_balance_backward):
        f.restype = c.c_int
    _lib = L
    return L


class EpBalance:
    """Owner of an ep_balance_t: the router's training losses.  route_cfg gives the
    number of experts, topk and the score function; the handle's workspace serves
    one forward at a time (a captured one counts each time that it is replayed)."""

    def __init__(self, route_cfg, max_tokens, max_sequences=1):
        self.cfg = route_cfg
        self._b = None
        self.device = torch.cuda.current_device()
        b = ctypes.c_void_p()
        _check(_load().ep_balance_create(ctypes.byref(route_cfg), max_tokens, max_sequences, ctypes.byref(b)))
        self._b = b

    @property
    def ptr(self):
        if self._b is None:
            raise EpError(EP_EINVAL, "handle already freed")
        return self._b

    def _args(self, logits, topk_idx, counts, tokens, seq_offsets):
        """Checks of both directions; rows, row stride, sequences."""
        cfg = self.cfg
        n, stride, device = _logits(cfg, logits, "logits")
        _require(device == self.device, "the tensors are not on the handle's device")
        _require(_is(topk_idx, torch.int64, (n, cfg.topk), device),
                 "topk_idx must be a contiguous int64 CUDA tensor [n, topk] on the device of logits")
        m = 1
        if seq_offsets is not None:
            _require(seq_offsets.dim() == 1 and seq_offsets.shape[0] > 1 and
                     _is(seq_offsets, torch.int32, seq_offsets.shape, device),
                     "seq_offsets must be a contiguous int32 CUDA tensor [sequences + 1] on the device of logits")
            m = seq_offsets.shape[0] - 1
        _require(_is(counts, torch.int32, (m, cfg.num_experts), device),
                 "counts must be a contiguous int32 CUDA tensor [sequences, num_experts] on the device of logits")
        _require(_is(tokens, torch.int32, (m + 1,), device),
                 "tokens must be a contiguous int32 CUDA tensor [sequences + 1] on the device of logits")
        return n, stride, m

    def forward(self, logits, topk_idx, counts, prob_sums, tokens, loss, seq_offsets=None, stream=None):
        """loss fp32 [2]: the load-balance loss and the z loss of logits [n, E] and
        ep_route's topk_idx [n, K]; counts int32 and prob_sums fp32 [G, E], tokens int32
        [G + 1] (live tokens of each sequence, then of all).  seq_offsets int32 [G + 1]:
        where each sequence begins and the last one ends; None: one sequence."""
        n, stride, m = self._args(logits, topk_idx, counts, tokens, seq_offsets)
        _require(_is(prob_sums, torch.float32, counts.shape, self.device),
                 "prob_sums must be a contiguous fp32 CUDA tensor [sequences, num_experts] on the device of logits")
        _require(_is(loss, torch.float32, (2,), self.device),
                 "loss must be a contiguous fp32 CUDA tensor [2] on the device of logits")
        _check(_load().ep_balance_forward(self.ptr, logits.data_ptr(), _FLOATS[logits.dtype], stride,
                                          topk_idx.data_ptr(), n, _ptr(seq_offsets), m, counts.data_ptr(),
                                          prob_sums.data_ptr(), tokens.data_ptr(), loss.data_ptr(),
                                          _stream(stream, self.device)))

    def backward(self, logits, topk_idx, counts, tokens, grad_loss, grad_logits, seq_offsets=None,
                 accumulate=False, stream=None):
        """Gradient of the two losses: grad_loss fp32 [2] in, grad_logits [n, E] of the
        logits' type out, or added to with accumulate.  counts and tokens are forward's."""
        n, stride, m = self._args(logits, topk_idx, counts, tokens, seq_offsets)
        gn, gstride, gdevice = _logits(self.cfg, grad_logits, "grad_logits")
        _require(grad_logits.dtype is logits.dtype and gn == n and gdevice == self.device,
                 "grad_logits must have the type, shape and device of logits")
        _require(_is(grad_loss, torch.float32, (2,), self.device),
                 "grad_loss must be a contiguous fp32 CUDA tensor [2] on the device of logits")
        _check(_load().ep_balance_backward(self.ptr, logits.data_ptr(), _FLOATS[logits.dtype], stride,
                                           topk_idx.data_ptr(), n, _ptr(seq_offsets), m, counts.data_ptr(),
                                           tokens.data_ptr(), grad_loss.data_ptr(), grad_logits.data_ptr(),
                                           gstride, int(bool(accumulate)), _stream(stream, self.device)))

    def free(self):
        if self._b is not None:
            _load().ep_balance_free(self._b)
            self._b = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
