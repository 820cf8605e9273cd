"""Training operators whose gradients the step consumes (see include/dmuon_ns.h).

    linear_cross_entropy(h, w, targets)                  # losses and lse per token
    linear_cross_entropy_backward(h, w, targets, lse, grad_losses)
    embedding(ids, table, scale=...)                     # lookup
    embedding_backward(ids, grad_out, rows, scale=...)   # the table's gradient
    checkpoint_quantize(x) / checkpoint_dequantize(q, exps)
    checkpoint_wgrad(grad_out, q, exps, offsets=None)    # weight gradient(s)

The functions marshal arguments only and enqueue on ``stream`` (the current
stream when None); results are allocated on it.  They take part in no autograd
graph: a caller wires them into its backward pass, for instance as the two halves
of a ``torch.autograd.Function``.  ``linear_cross_entropy`` and ``embedding`` refuse
inputs that require gradients where autograd records (outside ``torch.no_grad()``
and a Function's ``forward``), since their results would drop them.  Gradients come
in the layout ``muon_step`` and ``adamw_step`` read (dense, bf16 or fp32).
"""
from __future__ import annotations

import ctypes
import math

from . import _binding as _b

__all__ = ["linear_cross_entropy", "linear_cross_entropy_backward", "embedding",
           "embedding_backward", "checkpoint_quantize", "checkpoint_dequantize",
           "checkpoint_wgrad", "TARGET_ELSEWHERE"]

TARGET_ELSEWHERE = -2 ** 31     # a target that lies in another shard of the vocabulary
CKPT_BLOCK = 32          # columns that share one exponent byte


def _ptr(t):
    return ctypes.c_void_p(None if t is None else t.data_ptr())


def _no_graph(call, **tensors):
    """Refuse inputs whose gradients autograd expects to flow through this call."""
    import torch
    if not torch.is_grad_enabled():
        return
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and t.requires_grad:
            raise ValueError(f"{name} requires gradients, which {call} does not record: call it under torch.no_grad() or in "
                             f"a torch.autograd.Function and pass the gradients on with {call}_backward, or detach {name}")


def _gpu(t, what):
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a GPU tensor")


def _float_code(dtype, what):
    import torch
    if dtype == torch.bfloat16:
        return _b.BF16
    if dtype == torch.float32:
        return _b.F32
    raise ValueError(f"{what} must be bfloat16 or float32, got {dtype}")


def _index_code(t, what):
    import torch
    if t.dtype == torch.int64:
        return _b.I64
    if t.dtype == torch.int32:
        return _b.I32
    raise ValueError(f"{what} must be int64 or int32, got {t.dtype}")


def _matrix(t, what):
    """(rows, columns, row stride) of ``t`` seen as rows of its last dim: a 2-D
    tensor with any row stride, or a dense one of more dims."""
    _gpu(t, what)
    if t.dim() < 2:
        raise ValueError(f"{what} must have at least 2 dims")
    cols = t.shape[-1]
    rows = math.prod(t.shape[:-1])
    if t.is_contiguous():
        return rows, cols, cols
    if t.dim() != 2 or (cols > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be contiguous, or 2-D with a contiguous last dim")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{what} has overlapping rows (a broadcast or expanded tensor): make it contiguous")
    return rows, cols, t.stride(0) if rows > 1 else cols


def _dense(t, what, dtype=None, shape=None):
    _b._check_dev(t, what, dtype)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


class _Here:
    """The current stream of the current device (``stream`` None)."""

    def __init__(self, index):
        import torch
        self.handle = ctypes.c_void_p(torch.cuda.current_stream(index).cuda_stream)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False

    def workspace(self, ws, need, device):
        import torch
        if ws is None:
            return torch.empty(need or 1, dtype=torch.uint8, device=device)
        _check_workspace(ws, device)
        _b.keep_until_done(ws, [torch.cuda.current_stream(device)])
        return ws


class _On(_Here):
    """Another stream, current inside, so that what is allocated there belongs to
    it.  Tensors that were used on the caller's stream are recorded to it: their
    blocks outlive the queued work."""

    def __init__(self, st, tensors):
        import torch
        self.st = st
        self.handle = ctypes.c_void_p(st.cuda_stream)
        for t in tensors:
            _b.keep_until_done(t, [st])
        self.scope = torch.cuda.stream(st)

    def __enter__(self):
        self.scope.__enter__()
        return self

    def __exit__(self, *exc):
        return self.scope.__exit__(*exc)

    def workspace(self, ws, need, device):
        ws = super().workspace(ws, need, device)
        _b.keep_until_done(ws, [self.st])
        return ws


def _check_workspace(ws, device):
    _b._check_dev(ws, "workspace")
    if ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, the call on {device}")


def _on(stream, *tensors):
    """The scope a call allocates and enqueues in; its tensors must lie on the stream's device."""
    import torch
    index = torch.cuda.current_device() if stream is None else stream.device.index
    for t in tensors:
        if t is not None and t.device.index != index:
            raise ValueError(f"a tensor is on {t.device}, the stream on cuda:{index}")
    return _Here(index) if stream is None else _On(stream, tensors)


def _ws_args(ws):
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


def _ce_problem(h, w, targets, ignore_index):
    tokens, width, ldh = _matrix(h, "h")
    _matrix(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be 2-D (vocabulary, width)")
    vocab, w_width, ldw = _matrix(w, "w")
    if w_width != width:
        raise ValueError(f"h has width {width}, w has {w_width}")
    if h.dtype != w.dtype:
        raise ValueError("h and w must share a dtype")
    _dense(targets, "targets", None, h.shape[:-1])
    return _b.CeProblem(tokens, width, vocab, _float_code(h.dtype, "h"), _index_code(targets, "targets"),
                        h.data_ptr(), ldh, w.data_ptr(), ldw, targets.data_ptr(), int(ignore_index))


def _ce_workspace(prob, backward, workspace, on, device):
    need = ctypes.c_size_t(0)
    _b.check(_b.lib().dmuon_linear_ce_workspace_size(ctypes.byref(prob), backward, ctypes.byref(need)))
    return on.workspace(workspace, need.value, device)


def linear_cross_entropy(h, w, targets, *, ignore_index=-100, workspace=None, stream=None):
    """Softmax cross entropy of hidden states against a vocabulary, logits not kept.

    h: [..., width] hidden states; w: [vocab, width] (rows may be strided), both
    bf16 or both fp32; targets: int64 or int32 of h's leading shape.  Returns
    (losses, lse), fp32 of that shape: lse is the log-sum-exp of the token's
    logits, losses = lse − the target's logit.  Tokens whose target is
    ``ignore_index`` have loss and lse 0; a target of ``TARGET_ELSEWHERE`` gives the
    lse as the loss, another one outside the vocabulary NaN.

    A vocabulary in shards: call each with its rows of w and the targets shifted by
    its first row, ``TARGET_ELSEWHERE`` where that is not one of its rows.  Then lse
    is the logsumexp of the shards' and the loss lse − Σ (lse_shard − loss_shard).
    """
    import torch
    _no_graph("linear_cross_entropy", h=h, w=w)
    prob = _ce_problem(h, w, targets, ignore_index)
    with _on(stream, h, w, targets) as on:
        losses = torch.empty(targets.shape, dtype=torch.float32, device=h.device)
        lse = torch.empty_like(losses)
        ws = _ce_workspace(prob, 0, workspace, on, h.device)
        _b.check(_b.lib().dmuon_linear_ce(ctypes.byref(prob), _ptr(losses), _ptr(lse), *_ws_args(ws),
                                          on.handle))
    return losses, lse


def linear_cross_entropy_backward(h, w, targets, lse, grad_losses, *, ignore_index=-100, grad_h=None, grad_w=None,
                                  need_h=True, need_w=True, workspace=None, stream=None):
    """Gradients of ``linear_cross_entropy`` with respect to h and w.

    lse: as ``linear_cross_entropy`` returned it (of a vocabulary in shards: the
    joined one, with each shard's targets as there; grad_h is then the sum of the
    shards' results); grad_losses: fp32 of the same
    shape, the gradient of each token's loss (for a mean, 1/n everywhere); a token
    whose entry is 0 is left out like an ignored one.  Returns (grad_h, grad_w) in
    h's dtype, dense, of h's and w's shape; ``grad_h`` / ``grad_w`` name tensors to
    write (for instance views of a packed reduce buffer), ``need_h`` / ``need_w`` =
    False skips one (returned as None).
    """
    import torch
    prob = _ce_problem(h, w, targets, ignore_index)
    _dense(lse, "lse", torch.float32, targets.shape)
    _dense(grad_losses, "grad_losses", torch.float32, targets.shape)
    for t, what, like, need in ((grad_h, "grad_h", h, need_h), (grad_w, "grad_w", w, need_w)):
        if t is not None and not need:
            raise ValueError(f"{what} is given but not needed")
        if t is not None:
            _dense(t, what, like.dtype, like.shape)
    with _on(stream, h, w, targets, lse, grad_losses, grad_h, grad_w) as on:
        if need_h and grad_h is None:
            grad_h = torch.empty(h.shape, dtype=h.dtype, device=h.device)
        if need_w and grad_w is None:
            grad_w = torch.empty(w.shape, dtype=w.dtype, device=w.device)
        ws = _ce_workspace(prob, 1, workspace, on, h.device)
        _b.check(_b.lib().dmuon_linear_ce_backward(ctypes.byref(prob), _ptr(lse), _ptr(grad_losses), _ptr(grad_h),
                                                   _ptr(grad_w), *_ws_args(ws), on.handle))
    return grad_h, grad_w


def embedding(ids, table, *, scale=1.0, out=None, stream=None):
    """scale · table[ids] (bf16 or fp32, rounded once); zeros for ids outside the table.

    ids: int64 or int32 of any shape; table: [rows, width] (rows may be strided).
    """
    import torch
    _no_graph("embedding", table=table)
    _dense(ids, "ids")
    if isinstance(table, torch.Tensor) and table.dim() != 2:
        raise ValueError("table must be 2-D (rows, width)")
    rows, width, ldt = _matrix(table, "table")
    code, icode = _float_code(table.dtype, "table"), _index_code(ids, "ids")
    if out is not None:
        _dense(out, "out", table.dtype, (*ids.shape, width))
    with _on(stream, ids, table, out) as on:
        if out is None:
            out = torch.empty((*ids.shape, width), dtype=table.dtype, device=table.device)
        _b.check(_b.lib().dmuon_embedding(_ptr(ids), icode, ids.numel(), _ptr(table), ldt, rows, width, code,
                                          float(scale), _ptr(out), on.handle))
    return out


def embedding_backward(ids, grad_out, rows, *, scale=1.0, padding_id=None, out_dtype=None, out=None,
                       accumulate=False, workspace=None, stream=None):
    """The table's gradient: row v is scale times the sum of grad_out over the tokens with id v.

    ids: as in ``embedding``; grad_out: [*ids.shape, width], bf16 or fp32; rows: of
    the table.  Returns [rows, width] in ``out_dtype`` (grad_out's by default), or
    writes ``out``.  Tokens with ``padding_id`` or an id outside the table
    contribute nothing.  ``accumulate`` adds to ``out`` (required then) instead of
    overwriting it: for a table tied to the head, out is the head's gradient.
    Deterministic: the tokens are sorted by id and summed in a fixed order in fp32.
    """
    import torch
    _dense(ids, "ids")
    tokens, width, ldg = _matrix(grad_out, "grad_out")
    if tuple(grad_out.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"grad_out must have shape {(*ids.shape, 'width')}, got {tuple(grad_out.shape)}")
    rows = int(rows)
    if rows < 0:
        raise ValueError("rows must be >= 0")
    gcode, icode = _float_code(grad_out.dtype, "grad_out"), _index_code(ids, "ids")
    if padding_id is not None and int(padding_id) < 0:
        raise ValueError("padding_id must be >= 0 (None: no padding)")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out_dtype = grad_out.dtype if out_dtype is None else out_dtype
    else:
        _dense(out, "out", out_dtype, (rows, width))
        out_dtype = out.dtype
    ocode = _float_code(out_dtype, "out_dtype")
    need = ctypes.c_size_t(0)
    _b.check(_b.lib().dmuon_embedding_backward_workspace_size(tokens, rows, width, ctypes.byref(need)))
    with _on(stream, ids, grad_out, out) as on:
        if out is None:
            out = torch.empty((rows, width), dtype=out_dtype, device=grad_out.device)
        ws = on.workspace(workspace, need.value, grad_out.device)
        _b.check(_b.lib().dmuon_embedding_backward(
            _ptr(ids), icode, tokens, _ptr(grad_out), ldg, gcode, rows, width, float(scale),
            -1 if padding_id is None else int(padding_id), _ptr(out), ocode, 1 if accumulate else 0, *_ws_args(ws),
            on.handle))
    return out


def checkpoint_quantize(x, *, out=None, stream=None):
    """An activation kept in 8 bits: (q, exps), int8 of x's shape and uint8 [..., ceil(columns / 32)].

    x: [..., columns], bf16 or fp32.  x ≈ q·2^(exps − 133) with one exponent per 32
    columns of a row, every value to within 1/127.5 of the block's largest (half a
    step; a step for the last values below 2^128).  A block with an infinity or NaN
    reads back as NaN.
    ``out``: a (q, exps) pair to write.
    """
    import torch
    rows, cols, ldx = _matrix(x, "x")
    code = _float_code(x.dtype, "x")
    eshape = (*x.shape[:-1], -(-cols // CKPT_BLOCK))
    if out is not None:
        q, exps = out
        _dense(q, "q", torch.int8, x.shape)
        _dense(exps, "exps", torch.uint8, eshape)
    with _on(stream, x, *(out or ())) as on:
        if out is None:
            q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
            exps = torch.empty(eshape, dtype=torch.uint8, device=x.device)
        _b.check(_b.lib().dmuon_ckpt8_quantize(_ptr(x), code, rows, cols, ldx, _ptr(q), _ptr(exps),
                                               on.handle))
    return q, exps


def _check_checkpoint(q, exps):
    import torch
    _dense(q, "q", torch.int8)
    if q.dim() < 2:
        raise ValueError("q must have at least 2 dims")
    _dense(exps, "exps", torch.uint8, (*q.shape[:-1], -(-q.shape[-1] // CKPT_BLOCK)))


def checkpoint_dequantize(q, exps, *, dtype=None, out=None, stream=None):
    """The values a checkpoint holds, in ``dtype`` (bf16 by default; exact in either type)."""
    import torch
    _check_checkpoint(q, exps)
    if out is not None:
        _dense(out, "out", dtype, q.shape)
        dtype = out.dtype
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _float_code(dtype, "dtype")
    with _on(stream, q, exps, out) as on:
        if out is None:
            out = torch.empty(q.shape, dtype=dtype, device=q.device)
        _b.check(_b.lib().dmuon_ckpt8_dequantize(_ptr(q), _ptr(exps), math.prod(q.shape[:-1]), q.shape[-1], _ptr(out),
                                                 code, on.handle))
    return out


def checkpoint_wgrad(grad_out, q, exps, *, offsets=None, out_dtype=None, out=None, workspace=None, stream=None):
    """The weight gradient of y = x·Wᵀ from a kept x: grad_outᵀ · x, [n, k].

    grad_out: [..., n], bf16 or fp32 (rows may be strided); (q, exps): the
    checkpoint of x, [..., k].  With ``offsets`` (int32 [groups + 1] on the GPU) the
    result is [groups, n, k], group g over the rows offsets[g] … offsets[g + 1] − 1:
    the experts' gradients of a routed batch, as ``muon_step`` takes them.  The
    result is in ``out_dtype`` (grad_out's by default) or written to ``out``.
    """
    import torch
    _check_checkpoint(q, exps)
    tokens, n, ldg = _matrix(grad_out, "grad_out")
    if tuple(grad_out.shape[:-1]) != tuple(q.shape[:-1]):
        raise ValueError("grad_out and q differ in their leading shape")
    k = q.shape[-1]
    gcode = _float_code(grad_out.dtype, "grad_out")
    groups = 0
    shape = (n, k)
    if offsets is not None:
        _dense(offsets, "offsets", torch.int32)
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be 1-D with groups + 1 entries")
        groups = offsets.numel() - 1
        shape = (groups, n, k)
    if out is not None:
        _dense(out, "out", out_dtype, shape)
        out_dtype = out.dtype
    out_dtype = grad_out.dtype if out_dtype is None else out_dtype
    ocode = _float_code(out_dtype, "out_dtype")
    with _on(stream, grad_out, q, exps, offsets, out) as on:
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device=q.device)
        prob = _b.Ckpt8WgradProblem(tokens, n, k, gcode, ocode, grad_out.data_ptr(), ldg, q.data_ptr(),
                                    exps.data_ptr(), None if offsets is None else offsets.data_ptr(), groups, 0,
                                    out.data_ptr())
        need = ctypes.c_size_t(0)
        _b.check(_b.lib().dmuon_ckpt8_wgrad_workspace_size(ctypes.byref(prob), ctypes.byref(need)))
        ws = on.workspace(workspace, need.value, q.device)
        _b.check(_b.lib().dmuon_ckpt8_wgrad(ctypes.byref(prob), *_ws_args(ws), on.handle))
    return out
