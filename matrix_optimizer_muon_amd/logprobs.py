"""Log probabilities of given tokens with entropies, and their gradients (see include/dmuon_ns.h).

    token_logprobs(logits, targets, top=20)              # from logits: also the alternatives
    token_logprobs_backward(logits, targets, lse, entropy, grad_logprobs, grad_entropy)
    linear_token_logprobs(h, w, targets)                 # from hidden states, logits not kept
    linear_token_logprobs_backward(h, w, targets, lse, entropy, grad_logprobs, grad_entropy)

Calls, streams and autograd as in ``training``: the functions record nothing, and the
forward ones refuse inputs that require gradients where autograd records.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import _binding as _b
from .training import _ce_problem, _dense, _float_code, _index_code, _matrix, _no_graph, _on, _ptr, _ws_args

__all__ = ["TokenLogprobs", "token_logprobs", "token_logprobs_backward", "linear_token_logprobs",
           "linear_token_logprobs_backward"]


class TokenLogprobs(NamedTuple):
    """Per token: ``logprobs`` of its target, ``entropy`` and ``lse`` of its scaled logits
    (fp32), and with alternatives ``top_ids`` (int64) and ``top_logprobs`` (fp32) [..., top].
    What was not asked for is None.  Each is a tensor of its own."""
    logprobs: Optional[object]
    entropy: object
    lse: object
    top_ids: Optional[object] = None
    top_logprobs: Optional[object] = None


def _results(shape, like):
    """Three fp32 results.  Each is an allocation of its own: views of one could not be changed
    in place once a Function returned them, and would share a version with what it saved."""
    import torch
    first = like.new_empty(shape, dtype=torch.float32)
    return first, torch.empty_like(first), torch.empty_like(first)


# Calls of few rows take about as long as their arguments' checks: what is plainly right is
# told at a glance, and the rest goes through the checks that say what is wrong.
def _check_rows(t, what, dtype, shape):
    import torch
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.shape == shape and t.is_contiguous() and dtype in (None, t.dtype)):
        _dense(t, what, dtype, shape)


def _rows_problem(logits, targets, scale, top, ignore_index):
    import torch
    if isinstance(logits, torch.Tensor) and logits.dim() == 2 and logits.is_cuda and logits.is_contiguous():
        tokens, vocab = logits.shape
        ld = vocab
    else:
        tokens, vocab, ld = _matrix(logits, "logits")
    icode = _b.I64
    if targets is not None:
        _check_rows(targets, "targets", None, logits.shape[:-1])
        icode = _index_code(targets, "targets")
    return _b.LogprobsProblem(tokens, vocab, _float_code(logits.dtype, "logits"), icode, logits.data_ptr(), ld,
                              None if targets is None else targets.data_ptr(), int(ignore_index), float(scale), int(top))


def token_logprobs(logits, targets=None, *, top=0, scale=1.0, ignore_index=-100, workspace=None, stream=None):
    """Log probabilities of given tokens, entropies and the most likely alternatives.

    logits: [..., vocab], bf16 or fp32 (rows may be strided); targets: int64 or int32 of
    the leading shape, or None for the distributions alone.  The logits are multiplied by
    ``scale`` (1/temperature).  Returns a ``TokenLogprobs``.  Tokens whose target is
    ``ignore_index`` have zeros (ids -1); ``TARGET_ELSEWHERE`` gives -lse, another target
    outside the vocabulary NaN.  ``top`` (up to 128) alternatives come largest first, equal
    logits by rising id.

    A vocabulary in shards: call each with its columns and the shifted targets,
    ``TARGET_ELSEWHERE`` where that is not one of its columns.  Then lse is the logsumexp of
    the shards', the log probability sum(logprobs_s + lse_s) - lse, the entropy
    lse - sum(exp(lse_s - lse)*(lse_s - entropy_s)); a shard whose lse is -inf adds nothing.
    """
    import torch
    _no_graph("token_logprobs", logits=logits)
    prob = _rows_problem(logits, targets, scale, top, ignore_index)
    need = ctypes.c_size_t(0)
    _b.check(_b.lib().dmuon_logprobs_workspace_size(ctypes.byref(prob), ctypes.byref(need)))
    shape = logits.shape[:-1]
    with _on(stream, logits, targets) as on:
        logprobs, entropy, lse = _results(shape, logits)
        if targets is None:
            logprobs = None
        ids = best = None
        if top:
            ids = logits.new_empty((*shape, top), dtype=torch.int64)
            best = torch.empty_like(ids, dtype=torch.float32)
        ws = _ws_args(on.workspace(workspace, need.value, logits.device)) if need.value else (None, 0)
        _b.check(_b.lib().dmuon_logprobs(ctypes.byref(prob), _ptr(logprobs), _ptr(entropy), _ptr(lse), _ptr(ids), _ptr(best),
                                         *ws, on.handle))
    return TokenLogprobs(logprobs, entropy, lse, ids, best)


def _check_row_grads(shape, lse, entropy, grad_logprobs, grad_entropy):
    import torch
    if grad_logprobs is None and grad_entropy is None:
        raise ValueError("grad_logprobs or grad_entropy must be given")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs entropy")
    for t, what in ((lse, "lse"), (entropy, "entropy"), (grad_logprobs, "grad_logprobs"), (grad_entropy, "grad_entropy")):
        if t is not None or what == "lse":
            _check_rows(t, what, torch.float32, shape)


def token_logprobs_backward(logits, targets, lse, entropy, grad_logprobs, grad_entropy=None, *, scale=1.0, ignore_index=-100,
                            out=None, stream=None):
    """The gradient of ``token_logprobs`` with respect to the logits.

    lse, entropy: as ``token_logprobs`` returned them (of a vocabulary in shards: the
    joined ones); grad_logprobs, grad_entropy: fp32 of the same shape, the gradients of
    each token's log probability and entropy (either may be None); contiguous, which the
    expanded ones that ``sum()`` hands to a Function's backward are not.  Returns a dense tensor
    of the logits' shape and type, or writes ``out``, which may have strided rows and may be
    ``logits`` itself.
    """
    prob = _rows_problem(logits, targets, scale, 0, ignore_index)
    _check_row_grads(logits.shape[:-1], lse, entropy, grad_logprobs, grad_entropy)
    if grad_logprobs is not None and targets is None:
        raise ValueError("grad_logprobs needs targets")
    ld = prob.vocab
    if out is not None:
        ld = _matrix(out, "out")[2]
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out must have the logits' shape and type")
    with _on(stream, logits, targets, lse, entropy, grad_logprobs, grad_entropy, out) as on:
        if out is None:
            out = logits.new_empty(logits.shape)
        _b.check(_b.lib().dmuon_logprobs_backward(ctypes.byref(prob), _ptr(lse), _ptr(entropy), _ptr(grad_logprobs),
                                                  _ptr(grad_entropy), _ptr(out), ld, on.handle))
    return out


def _linear_workspace(prob, backward, workspace, on, device):
    need = ctypes.c_size_t(0)
    _b.check(_b.lib().dmuon_linear_logprobs_workspace_size(ctypes.byref(prob), backward, ctypes.byref(need)))
    return on.workspace(workspace, need.value, device)


def linear_token_logprobs(h, w, targets, *, scale=1.0, ignore_index=-100, workspace=None, stream=None):
    """Log probabilities of given tokens and entropies of a vocabulary, logits not kept.

    h, w, targets, ``ignore_index`` and shards of the vocabulary as in
    ``linear_cross_entropy``; the logits h·wᵀ are multiplied by ``scale``.  Returns a
    ``TokenLogprobs`` without alternatives, its values as those of ``token_logprobs``.
    """
    _no_graph("linear_token_logprobs", h=h, w=w)
    prob = _ce_problem(h, w, targets, ignore_index)
    with _on(stream, h, w, targets) as on:
        logprobs, entropy, lse = _results(targets.shape, h)
        ws = _linear_workspace(prob, 0, workspace, on, h.device)
        _b.check(_b.lib().dmuon_linear_logprobs(ctypes.byref(prob), float(scale), _ptr(logprobs), _ptr(entropy), _ptr(lse),
                                                *_ws_args(ws), on.handle))
    return TokenLogprobs(logprobs, entropy, lse)


def linear_token_logprobs_backward(h, w, targets, lse, entropy, grad_logprobs, grad_entropy=None, *, scale=1.0,
                                   ignore_index=-100, grad_h=None, grad_w=None, need_h=True, need_w=True, workspace=None,
                                   stream=None):
    """Gradients of ``linear_token_logprobs`` with respect to h and w.

    lse, entropy, grad_logprobs and grad_entropy as in ``token_logprobs_backward``; grad_h,
    grad_w, ``need_h`` and ``need_w`` as in ``linear_cross_entropy_backward``.
    """
    prob = _ce_problem(h, w, targets, ignore_index)
    _check_row_grads(targets.shape, lse, entropy, grad_logprobs, grad_entropy)
    for t, what, like, need in ((grad_h, "grad_h", h, need_h), (grad_w, "grad_w", w, need_w)):
        if t is not None and not need:
            raise ValueError(f"{what} is given but not needed")
        if t is not None:
            _dense(t, what, like.dtype, like.shape)
    with _on(stream, h, w, targets, lse, entropy, grad_logprobs, grad_entropy, grad_h, grad_w) as on:
        if need_h and grad_h is None:
            grad_h = h.new_empty(h.shape)
        if need_w and grad_w is None:
            grad_w = w.new_empty(w.shape)
        ws = _linear_workspace(prob, 1, workspace, on, h.device)
        _b.check(_b.lib().dmuon_linear_logprobs_backward(ctypes.byref(prob), float(scale), _ptr(lse), _ptr(entropy),
                                                         _ptr(grad_logprobs), _ptr(grad_entropy), _ptr(grad_h), _ptr(grad_w),
                                                         *_ws_args(ws), on.handle))
    return grad_h, grad_w
