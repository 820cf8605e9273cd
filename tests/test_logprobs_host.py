"""Refusals of the log-probability entry points (no GPU needed: every call is rejected, or
does nothing, before any HIP call; pointers are never dereferenced), workspace sizes, and
the argument checks of the Python face."""
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


def rows(**kw):
    d = dict(tokens=64, vocab=1000, dtype=B.BF16, index_dtype=B.I64, logits=at(1), ld=1000, targets=at(2), ignore_index=-100,
             scale=1.0, top=5)
    d.update(kw)
    return B.LogprobsProblem(*[d[n] for n, _ in B.LogprobsProblem._fields_])


def size(p):
    out = ctypes.c_size_t(0)
    rc = B.lib().dmuon_logprobs_workspace_size(ctypes.byref(p), ctypes.byref(out))
    return rc, out.value


def fwd(p, lp=at(3), H=at(4), lse=at(5), ids=at(6), best=at(7), ws=WS, nbytes=1 << 39):
    return B.lib().dmuon_logprobs(ctypes.byref(p), vp(lp), vp(H), vp(lse), vp(ids), vp(best), vp(ws), nbytes, None)


def bwd(p, lse=at(5), H=at(4), g=at(8), h=at(9), out=at(10), ld=1000):
    return B.lib().dmuon_logprobs_backward(ctypes.byref(p), vp(lse), vp(H), vp(g), vp(h), vp(out), ld, None)


@pytest.fixture(autouse=True)
def nothing_is_enqueued(monkeypatch):
    """A call that validation lets through ends before its first launch."""
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", "plan")


BAD = [(dict(dtype=7), -4), (dict(index_dtype=5), -4), (dict(tokens=-1), -3), (dict(tokens=(1 << 24) + 1), -3), (dict(vocab=0, ld=0), -3),
       (dict(vocab=(1 << 22) + 1, ld=1 << 23), -3), (dict(ld=999), -3), (dict(ld=(1 << 40) + 1), -3), (dict(tokens=256, ld=1 << 40), -3),
       (dict(scale=0.0), -5), (dict(scale=-1.0), -5), (dict(scale=math.inf), -5), (dict(scale=math.nan), -5), (dict(scale=2.0 ** -21), -5),
       (dict(scale=2.0 ** 21), -5), (dict(logits=None), -1), (dict(tokens=1 << 24, vocab=100000, ld=100000), -3)]


@pytest.mark.parametrize("kw,code", BAD)
def test_refusals(kw, code):
    p = rows(**kw)
    assert fwd(p) == code
    assert size(p)[0] == code
    assert bwd(p, ld=max(p.vocab, 1)) == code
    assert B.lib().dmuon_last_error()


def test_refusals_of_outputs():
    p = rows()
    assert fwd(p) == -8 and bwd(p) == -8                       # accepted
    assert B.lib().dmuon_logprobs(None, vp(at(3)), vp(at(4)), vp(at(5)), None, None, None, 0, None) == -1
    assert fwd(p, H=None) == -1 and fwd(p, lse=None) == -1 and fwd(p, ids=None) == -1 and fwd(p, best=None) == -1
    assert fwd(p, lp=None) == -1 and fwd(rows(targets=None)) == -1
    assert fwd(rows(targets=None), lp=None) == -8
    assert fwd(rows(top=0), ids=None, best=None) == -8
    for top in (-1, 129):
        assert fwd(rows(top=top)) == -5
    assert fwd(rows(vocab=4, ld=4)) == -5                       # more alternatives than words
    assert bwd(rows(top=-1)) == -8                              # not read
    many = rows(tokens=1 << 24, vocab=8, ld=8)                  # a wave per row: 2^30 threads
    assert fwd(many) == -8 and bwd(many, ld=8) == -8
    assert fwd(p, lp=at(4)) == -7 and fwd(p, H=at(1) + 64) == -7 and fwd(p, ids=at(7) + 8) == -7
    assert bwd(p, lse=None) == -1 and bwd(p, out=None) == -1 and bwd(p, g=None, h=None) == -1 and bwd(p, H=None) == -1
    assert bwd(rows(targets=None)) == -1
    assert bwd(rows(targets=None), g=None) == -8 and bwd(p, h=None, H=None) == -8
    assert bwd(p, ld=999) == -3 and bwd(rows(tokens=256), ld=1 << 40) == -3
    assert bwd(p, out=at(1)) == -8                              # in place
    assert bwd(p, out=at(1), ld=1001) == -7                     # not with another stride
    assert bwd(p, out=at(1) + 2) == -7 and bwd(p, out=at(8)) == -7


def test_workspace():
    assert size(rows(tokens=0, logits=None, targets=None)) == (0, 0)
    # a row per workgroup: none
    assert size(rows(tokens=4096, vocab=131072, ld=131072, top=128)) == (0, 0)
    assert fwd(rows(tokens=4096, vocab=131072, ld=131072), ws=None, nbytes=0) == -8
    # few rows, or long ones, in pieces: their statistics and candidates
    for kw in (dict(tokens=1, vocab=128000, top=20), dict(tokens=9, vocab=1 << 22, top=128), dict(tokens=1, vocab=1 << 22, top=1)):
        p = rows(ld=kw["vocab"], **kw)
        rc, n = size(p)
        assert rc == 0 and 0 < n <= p.tokens * 64 * (12 + 8 * p.top) + 512
        assert fwd(p, nbytes=n) == -8
        assert fwd(p, ws=None) == -6 and fwd(p, nbytes=n - 1) == -6 and fwd(p, ws=WS + 128) == -6
        assert fwd(p, ws=at(1)) == -7
    # a row's candidates fit the LDS of the workgroup that joins them
    for top in range(1, 129):
        for tokens in (1, 3, 40, 1 << 10):
            for vocab in (2048, 50257, 1 << 22):
                n = size(rows(tokens=tokens, vocab=vocab, ld=vocab, top=top))[1]
                assert n // tokens <= 6144 * 8 + 64 * 12 + 512
    assert B.lib().dmuon_logprobs_workspace_size(ctypes.byref(rows()), None) == -1


def test_no_rows():
    p = rows(tokens=0, logits=None, targets=None)
    assert fwd(p, lp=None, H=None, lse=None, ids=None, best=None, ws=None, nbytes=0) == 0
    assert bwd(p, lse=None, H=None, g=None, h=None, out=None) == 0


@pytest.mark.parametrize("point,call", [("plan", fwd), ("logprobs", fwd), ("plan", bwd), ("logprobs_grad", bwd)])
def test_forced_failure_before_the_first_launch(point, call, monkeypatch):
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", point)
    assert call(rows()) == -8
    assert point.encode() in B.lib().dmuon_last_error()


def refusal(call):
    with pytest.raises(ValueError) as e:
        call()
    return str(e.value)


def test_python_refusals():
    z, y, g = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    assert "GPU tensor" in refusal(lambda: mm.token_logprobs(z, y))
    assert "GPU tensor" in refusal(lambda: mm.token_logprobs_backward(z, y, g, g, g))
    leaf = z.clone().requires_grad_()
    for call in (lambda: mm.token_logprobs(leaf, y), lambda: mm.token_logprobs(leaf * 2, y)):
        assert refusal(call).startswith("logits requires gradients")
        with torch.no_grad():
            assert "GPU tensor" in refusal(call)
    assert "torch.Tensor" in refusal(lambda: mm.token_logprobs([1.0], y))


# ---- from hidden states -----------------------------------------------------------
def ce(**kw):
    d = dict(tokens=64, width=128, vocab=1000, dtype=B.BF16, index_dtype=B.I64, h=at(1), ldh=128, w=at(2), ldw=128, targets=at(3),
             ignore_index=-100)
    d.update(kw)
    return B.CeProblem(*[d[n] for n, _ in B.CeProblem._fields_])


def lsize(p, backward=0):
    out = ctypes.c_size_t(0)
    rc = B.lib().dmuon_linear_logprobs_workspace_size(ctypes.byref(p), backward, ctypes.byref(out))
    return rc, out.value


def lfwd(p, scale=1.0, lp=at(4), H=at(5), lse=at(6), ws=WS, nbytes=1 << 39):
    return B.lib().dmuon_linear_logprobs(ctypes.byref(p), scale, vp(lp), vp(H), vp(lse), vp(ws), nbytes, None)


def lbwd(p, scale=1.0, lse=at(6), H=at(5), g=at(7), e=at(8), gh=at(9), gw=at(10), ws=WS, nbytes=1 << 39):
    return B.lib().dmuon_linear_logprobs_backward(ctypes.byref(p), scale, vp(lse), vp(H), vp(g), vp(e), vp(gh), vp(gw), vp(ws),
                                                  nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), -4), (dict(index_dtype=5), -4), (dict(tokens=-1), -3), (dict(tokens=(1 << 24) + 1), -3), (dict(width=0, ldh=0, ldw=0), -3),
    (dict(vocab=0), -3), (dict(ldh=127), -3), (dict(ldw=127), -3), (dict(h=None), -1), (dict(w=None), -1), (dict(targets=None), -1),
    (dict(tokens=1 << 24, vocab=1 << 30), -3)])
def test_linear_refusals(kw, code):
    assert lfwd(ce(**kw)) == code and lbwd(ce(**kw)) == code


def test_linear_refusals_of_outputs():
    p = ce()
    assert lfwd(p) == -8 and lbwd(p) == -8
    for s in (0.0, -1.0, math.inf, math.nan, 2.0 ** -21, 2.0 ** 21):
        assert lfwd(p, s) == -5 and lbwd(p, s) == -5
    assert lfwd(p, lp=None) == -1 and lfwd(p, H=None) == -1 and lfwd(p, lse=None) == -1
    assert lfwd(p, H=at(4)) == -7 and lfwd(p, H=at(1)) == -7
    assert lbwd(p, lse=None) == -1 and lbwd(p, H=None) == -1 and lbwd(p, g=None, e=None) == -1
    assert lbwd(p, g=None) == -8 and lbwd(p, e=None, H=None) == -8 and lbwd(p, gh=None) == -8
    assert lbwd(p, gh=None, gw=None) == 0
    assert lbwd(p, gh=at(8)) == -7 and lbwd(p, gw=at(5)) == -7
    for call, n in ((lfwd, lsize(p)[1]), (lbwd, lsize(p, 1)[1])):
        assert n > 0 and call(p, nbytes=n) == -8
        assert call(p, nbytes=n - 1) == -6 and call(p, ws=None) == -6 and call(p, ws=WS + 8) == -6 and call(p, ws=at(1)) == -7
    assert lsize(p, 2)[0] == -5
    assert B.lib().dmuon_linear_logprobs_workspace_size(ctypes.byref(p), 0, None) == -1
    none = ce(tokens=0, h=None, targets=None)
    assert lsize(none) == (0, 0) and lfwd(none, lp=None, H=None, lse=None, ws=None) == 0
    assert lbwd(none, lse=None, H=None, g=None, e=None, gw=None, ws=None) == -8     # accepted


def test_linear_python_refusals():
    h, w, y, g = torch.zeros(4, 8), torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    assert "GPU tensor" in refusal(lambda: mm.linear_token_logprobs(h, w, y))
    assert "GPU tensor" in refusal(lambda: mm.linear_token_logprobs_backward(h, w, y, g, g, g))
    leaf = h.clone().requires_grad_()
    assert refusal(lambda: mm.linear_token_logprobs(leaf, w, y)).startswith("h requires gradients")
    assert refusal(lambda: mm.linear_token_logprobs(h, w.clone().requires_grad_(), y)).startswith("w requires gradients")
