"""Refusals of the gradient-norm and clipping entry points (no GPU needed: every call is
rejected, or does nothing, before any HIP call; pointers are never dereferenced), workspace
sizes, and the argument checks of the Python face."""
import ctypes
import math

import pytest
import torch

import matrix_optimizer_muon_amd as mm
from matrix_optimizer_muon_amd import _binding as B

FAKE = 0x7F0000000000
GAP = 1 << 40
WS = FAKE + 100 * GAP
vp = ctypes.c_void_p


def at(i):
    return FAKE + i * GAP


def tensors(*changes):
    arr = (B.GradTensor * max(len(changes), 1))()
    for i, kw in enumerate(changes):
        d = dict(numel=1000, dtype=B.BF16, out_dtype=B.BF16, grad=at(2 * i + 1), out=at(2 * i + 2))
        d.update(kw)
        arr[i] = B.GradTensor(*[d[n] for n, _ in B.GradTensor._fields_])
    return arr, len(changes)


def size(t):
    out = ctypes.c_size_t(0)
    return B.lib().dmuon_grad_workspace_size(*t, ctypes.byref(out)), out.value


def prepare(t, ws=WS, nbytes=1 << 30):
    return B.lib().dmuon_grad_prepare(*t, vp(ws), nbytes, None)


def norm_run(t, norm=at(90), ws=WS, nbytes=1 << 30):
    return B.lib().dmuon_grad_norm_run(*t, vp(norm), vp(ws), nbytes, None)


def clip_run(t, max_norm=1.0, eps=1e-6, measure=1, norm=at(90), ws=WS, nbytes=1 << 30):
    return B.lib().dmuon_grad_clip_run(*t, max_norm, eps, measure, vp(norm), vp(ws), nbytes, None)


@pytest.fixture(autouse=True)
def nothing_is_enqueued(monkeypatch):
    """A call that validation lets through ends before its first launch."""
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", "plan")


@pytest.mark.parametrize("kw,code", [(dict(numel=-1), -3), (dict(numel=(1 << 41) + 1), -3), (dict(dtype=2), -4), (dict(out_dtype=5), -4),
                                     (dict(grad=None), -1), (dict(out=at(3), out_dtype=B.F32), -4)])
def test_tensors_are_refused(kw, code):
    t = tensors({}, kw)
    assert size(t)[0] == code and prepare(t) == code and norm_run(t) == code and clip_run(t) == code
    assert b"tensor 1" in B.lib().dmuon_last_error()


def test_refusals():
    t = tensors({}, dict(out_dtype=B.F32), dict(numel=0, grad=None, out=None))
    assert prepare(t) == -8 and norm_run(t) == -8 and clip_run(t) == -8 and clip_run(t, measure=0) == -8     # accepted
    assert B.lib().dmuon_grad_prepare(None, 1, None, 0, None) == -1 and B.lib().dmuon_grad_prepare(None, -1, None, 0, None) == -3
    n = size(t)[1]
    assert 0 < n <= 2048
    for call in (prepare, norm_run, clip_run):
        assert call(t, ws=None) == -6 and call(t, ws=WS + 64) == -6 and call(t, nbytes=n - 1) == -6 and call(t, ws=at(1)) == -7
        assert call(t, nbytes=n) == -8
    assert norm_run(t, norm=None) == -1 and clip_run(t, norm=None) == -1
    assert norm_run(t, norm=at(1)) == -7 and clip_run(t, norm=at(2) + 8) == -7 and clip_run(t, norm=WS) == -7
    assert clip_run(t, norm=at(1), measure=0) == -8              # read beside a gradient that is read
    assert clip_run(t, norm=at(2), measure=0) == -7
    for x in (-1.0, math.inf, math.nan):
        assert clip_run(t, max_norm=x) == -5 and clip_run(t, eps=x) == -5
    assert clip_run(t, measure=2) == -5
    assert clip_run(tensors(dict(out=None))) == -1 and norm_run(tensors(dict(out=None))) == -8
    assert prepare(tensors(dict(out=at(1)))) == -8               # in place
    assert prepare(tensors(dict(out=at(1) + 2))) == -7
    assert prepare(tensors({}, dict(grad=at(1), out=at(9)))) == -8        # one gradient read twice
    assert prepare(tensors(dict(out=at(1)), dict(grad=at(1), out=at(1)))) == -7
    assert prepare(tensors({}, dict(out=at(2) + 1998))) == -7
    assert B.lib().dmuon_grad_workspace_size(*t, None) == -1


def test_sizes():
    none = tensors()
    assert size(none) == (0, 0) and prepare(none, ws=None, nbytes=0) == 0 and clip_run(none, ws=None, nbytes=0, measure=0) == 0
    assert norm_run(none, ws=None, nbytes=0) == -8               # accepted: writes 0
    assert size(tensors(dict(numel=0))) == (0, 0)
    # a table entry and a first chunk per tensor, a sum for each of at most 2048 workgroups
    assert size(tensors(dict(numel=1 << 41)))[1] <= 2048 * 8 + 1024
    many = tensors(*[dict(numel=3, grad=at(1) + 64 * i, out=at(2) + 64 * i) for i in range(5000)])
    assert size(many)[1] <= 5000 * 44 + 2048 * 8 + 1024
    assert prepare(many) == -8
    assert size(tensors(dict(numel=1 << 40), dict(numel=1 << 40), {}))[0] == -3


@pytest.mark.parametrize("point,call,code", [("plan", prepare, -8), ("table", prepare, -8), ("grad_norm", norm_run, -8), ("grad_norm", clip_run, -8)])
def test_forced_failures(point, call, code, monkeypatch):
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", point)
    assert call(tensors({})) == code
    assert point.encode() in B.lib().dmuon_last_error()
    if call is clip_run:
        monkeypatch.setenv("DMUON_TEST_FAIL_AT", "grad_clip")
        assert clip_run(tensors({}), measure=0) == -8


def test_python_refusals():
    g = [torch.zeros(3), torch.zeros(4)]
    for call in (lambda: mm.grad_norm(g), lambda: mm.clip_grad_norm(g, 1.0), lambda: mm.ClipGradNorm(g, 1.0)):
        with pytest.raises(ValueError, match=r"grads\[0\] must be a GPU tensor"):
            call()
    for bad in (-1.0, math.inf, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            mm.clip_grad_norm(g, bad)
        with pytest.raises(ValueError, match="eps"):
            mm.ClipGradNorm(g, 1.0, eps=bad)
    with pytest.raises(ValueError, match="differ in length"):
        mm.clip_grad_norm(g, 1.0, outs=g[:1])
