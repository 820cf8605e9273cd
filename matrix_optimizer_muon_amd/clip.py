"""The global norm over many gradients, and clipping (see include/dmuon_ns.h).

    grad_norm(grads)                                # 0-dim fp32 tensor on the GPU
    clip_grad_norm(grads, max_norm, outs=None)      # in place, or into outs; returns the norm
    clip = ClipGradNorm(grads, max_norm)            # prepared: clip() each step

No call waits for the GPU: the norm stays on the device.  (The constructor of
``ClipGradNorm`` waits for its tables once.)
"""
from __future__ import annotations

import ctypes
import math

from . import _binding as _b
from .training import _float_code, _on, _ptr, _ws_args

__all__ = ["ClipGradNorm", "clip_grad_norm", "grad_norm"]


def _descs(grads, outs):
    """(descriptors, their number, device); outs None: no outputs."""
    n = len(grads)
    if outs is not None and len(outs) != n:
        raise ValueError("grads and outs differ in length")
    arr = (_b.GradTensor * max(n, 1))()
    for i, g in enumerate(grads):
        _b._check_dev(g, f"grads[{i}]")
        if g.device != grads[0].device:
            raise ValueError(f"grads[{i}] is on {g.device}, grads[0] on {grads[0].device}")
        a = arr[i]
        a.numel, a.dtype, a.grad = g.numel(), _float_code(g.dtype, f"grads[{i}]"), g.data_ptr()
        if outs is not None:
            o = outs[i]
            if o is not g:
                _b._check_dev(o, f"outs[{i}]")
                if o.shape != g.shape or o.device != g.device:
                    raise ValueError(f"outs[{i}] must have the shape and device of grads[{i}]")
            a.out_dtype, a.out = _float_code(o.dtype, f"outs[{i}]"), o.data_ptr()
    return arr, n, grads[0].device if n else None


def _workspace(arr, n, workspace, on, device):
    need = ctypes.c_size_t(0)
    _b.check(_b.lib().dmuon_grad_workspace_size(arr, n, ctypes.byref(need)))
    return on.workspace(workspace, need.value, device)


def _new_norm(n, device):
    import torch
    return (torch.empty if n else torch.zeros)((), dtype=torch.float32, device=device or "cuda")


def _check_norm(norm, device):
    import torch
    _b._check_dev(norm, "norm", torch.float32)
    if norm.numel() != 1 or (device is not None and norm.device != device):
        raise ValueError("norm must be one value on the gradients' device")


def _limits(max_norm, eps):
    max_norm, eps = float(max_norm), float(eps)
    if not (max_norm >= 0 and math.isfinite(max_norm)):
        raise ValueError("max_norm must be finite and >= 0")
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError("eps must be finite and >= 0")
    return max_norm, eps


class ClipGradNorm:
    """Gradient clipping prepared over a fixed set of tensors.

    grads: bf16 or fp32 GPU tensors of any shape, contiguous; outs: where the clipped
    gradients go (bf16 or fp32 of the same shapes, for instance views of a packed reduce
    buffer), None: in place.  The constructor writes the tables of these tensors into the
    workspace and waits for that; it cannot be captured, the calls can.  Every call enqueues
    the norm and the clipping on ``stream`` and returns ``norm``, a 0-dim fp32 tensor that the
    next call overwrites.  The tensors must keep their storage; it is not handed out again
    before the queued calls are done, but what a captured graph uses the caller keeps alive.
    ``max_norm`` may be changed between calls.  Where the norm is not finite the gradients
    pass unscaled, so that the caller can skip the step.  Calls on different streams and replays of a
    captured graph share this object's workspace and must not overlap.
    """

    def __init__(self, grads, max_norm, *, outs=None, eps=1e-6, workspace=None, stream=None):
        import torch
        grads = list(grads)
        self._tensors = (grads, grads if outs is None else list(outs))
        self.max_norm, self.eps = _limits(max_norm, eps)
        self._arr, self._n, self._device = _descs(*self._tensors)
        self.workspace = None
        self._seen = set()
        with _on(stream, *grads) as on:
            self.norm = _new_norm(self._n, self._device)
            if self._n:
                self.workspace = _workspace(self._arr, self._n, workspace, on, self._device)
                _b.check(_b.lib().dmuon_grad_prepare(self._arr, self._n, *_ws_args(self.workspace), on.handle))
                torch.cuda.current_stream().synchronize()      # the tables are in place before a call on any stream

    def __call__(self, stream=None):
        import torch
        if self._n == 0:
            return self.norm
        with _on(stream, self.norm, self.workspace) as on:
            if on.handle.value not in self._seen and not torch.cuda.is_current_stream_capturing():
                # all that the queued kernels use outlives this object, on every stream it is called on
                st = _b.resolve_stream(None)
                for t in (self.workspace, self.norm, *self._tensors[0], *self._tensors[1]):
                    _b.keep_until_done(t, [st])
                self._seen.add(on.handle.value)
            _b.check(_b.lib().dmuon_grad_clip_run(self._arr, self._n, self.max_norm, self.eps, 1, _ptr(self.norm),
                                                  *_ws_args(self.workspace), on.handle))
        return self.norm


def grad_norm(grads, *, workspace=None, stream=None):
    """The 2-norm of all gradients together: a 0-dim fp32 tensor (sums in 64 bits)."""
    grads = list(grads)
    arr, n, device = _descs(grads, None)
    with _on(stream, *grads) as on:
        norm = _new_norm(n, device)
        if n:
            ws = _workspace(arr, n, workspace, on, device)
            _b.check(_b.lib().dmuon_grad_prepare(arr, n, *_ws_args(ws), on.handle))
            _b.check(_b.lib().dmuon_grad_norm_run(arr, n, _ptr(norm), *_ws_args(ws), on.handle))
    return norm


def clip_grad_norm(grads, max_norm, *, outs=None, norm=None, eps=1e-6, workspace=None, stream=None):
    """Scales the gradients by min(1, max_norm/(norm + eps)), in place or into ``outs``.

    Returns the norm, a 0-dim fp32 tensor.  ``norm``: one fp32 value on the GPU to clip by
    instead of the gradients' own (gradients on several owners: the root of the sum of
    their squared norms).  Where the norm is not finite the gradients pass unscaled.
    """
    grads = list(grads)
    max_norm, eps = _limits(max_norm, eps)
    outs = grads if outs is None else list(outs)
    arr, n, device = _descs(grads, outs)
    if norm is not None:
        _check_norm(norm, device)
    with _on(stream, *grads, *outs, norm) as on:
        measure = 1 if norm is None else 0
        if measure:
            norm = _new_norm(n, device)
        if n:
            ws = _workspace(arr, n, workspace, on, device)
            _b.check(_b.lib().dmuon_grad_prepare(arr, n, *_ws_args(ws), on.handle))
            _b.check(_b.lib().dmuon_grad_clip_run(arr, n, max_norm, eps, measure, _ptr(norm), *_ws_args(ws), on.handle))
    return norm
