"""Refusals of the training-gradient entry points (no GPU needed: every call is
rejected, or does nothing, before any HIP call; pointers are never dereferenced),
workspace sizes, and the argument checks of the Python face."""
import ctypes

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


def ce(**kw):
    d = dict(tokens=64, width=128, vocab=1000, dtype=B.BF16, index_dtype=B.I64, h=at(1), ldh=128, w=at(2), ldw=128,
             targets=at(3), ignore_index=-100)
    d.update(kw)
    return B.CeProblem(*[d[n] for n, _ in B.CeProblem._fields_])


def ce_size(p, backward=0):
    out = ctypes.c_size_t(0)
    rc = B.lib().dmuon_linear_ce_workspace_size(ctypes.byref(p), backward, ctypes.byref(out))
    return rc, out.value


def ce_fwd(p, losses=at(4), lse=at(5), ws=WS, nbytes=1 << 39):
    return B.lib().dmuon_linear_ce(ctypes.byref(p), vp(losses), vp(lse), vp(ws), nbytes, None)


def ce_bwd(p, lse=at(5), gl=at(6), gh=at(7), gw=at(8), ws=WS, nbytes=1 << 39):
    return B.lib().dmuon_linear_ce_backward(ctypes.byref(p), vp(lse), vp(gl), vp(gh), vp(gw), vp(ws), nbytes, None)


BAD_CE = [
    (dict(dtype=7), -4), (dict(index_dtype=5), -4), (dict(tokens=-1), -3), (dict(tokens=(1 << 24) + 1), -3),
    (dict(width=0, ldh=0, ldw=0), -3), (dict(width=65537, ldh=70000, ldw=70000), -3), (dict(vocab=0), -3),
    (dict(vocab=(1 << 30) + 1), -3), (dict(ldh=127), -3), (dict(ldw=127), -3), (dict(h=None), -1), (dict(w=None), -1),
    (dict(targets=None), -1), (dict(tokens=1 << 24, vocab=1 << 30), -3),
]


@pytest.mark.parametrize("kw,code", BAD_CE)
def test_ce_refuses(kw, code):
    p = ce(**kw)
    assert ce_fwd(p) == code
    assert ce_bwd(p) == code
    if code != -1 or "w" in kw:
        assert ce_size(p)[0] == code
    assert B.lib().dmuon_last_error()


def test_ce_refuses_outputs_and_workspace():
    p = ce()
    assert B.lib().dmuon_linear_ce(None, vp(at(4)), vp(at(5)), vp(WS), 1 << 39, None) == -1
    assert ce_fwd(p, losses=None) == -1
    assert ce_fwd(p, lse=None) == -1
    assert ce_fwd(p, losses=at(5)) == -7                       # losses and lse are one buffer
    assert ce_fwd(p, lse=at(1) + 256) == -7                    # inside h
    assert ce_bwd(p, lse=None) == -1
    assert ce_bwd(p, gl=None) == -1
    assert ce_bwd(p, gh=at(1)) == -7
    assert ce_bwd(p, gw=at(2) + 64) == -7
    assert ce_bwd(p, gh=None, gw=None) == 0                    # nothing wanted: nothing done
    for call, size in ((ce_fwd, ce_size(p)[1]), (ce_bwd, ce_size(p, 1)[1])):
        assert size > 0
        assert call(p, ws=None) == -6
        assert call(p, ws=WS + 128) == -6
        assert call(p, nbytes=size - 1) == -6
        assert call(p, ws=at(1) & ~255) == -7                  # the workspace meets h
    assert ce_size(p, 2)[0] == -5
    assert B.lib().dmuon_linear_ce_workspace_size(ctypes.byref(p), 0, None) == -1


def test_ce_without_tokens():
    p = ce(tokens=0, h=None, targets=None)
    assert ce_size(p) == (0, 0) and ce_size(p, 1) == (0, 0)
    assert ce_fwd(p, losses=None, lse=None, ws=None, nbytes=0) == 0
    assert ce_bwd(p, lse=None, gl=None, gw=None, ws=None, nbytes=0) == 0


def test_ce_workspace_keeps_no_logits():
    """A piece of the vocabulary at a time: far below tokens × vocab, and a copy of
    w only where the core cannot read it in place."""
    big = dict(tokens=8192, width=4096, vocab=128000, ldh=4096, ldw=4096)
    assert ce_size(ce(**big))[1] < 8192 * 4096 * 2 + 8192 * 500 * 8 + (1 << 20)
    # gradient logits of a piece (256 MiB, its rows rounded up to tiles of 256), the
    # hidden states in two orders, their gradient's fp32 sums, four numbers per token
    assert ce_size(ce(**big), 1)[1] <= (256 << 20) + 8192 * 256 * 2 + 8192 * 4096 * (2 + 2 + 4) + 8192 * 16 + 8192 * 4 + 4096
    assert ce_size(ce(**big), 1)[1] < 8192 * 128000 * 2 // 3
    aligned, shifted = ce_size(ce(**big))[1], ce_size(ce(**dict(big, w=at(2) + 2)))[1]
    assert shifted > aligned
    small = ce_size(ce(tokens=1, width=1, vocab=1, ldh=1, ldw=1))[1]
    assert 0 < small < 1 << 16


def test_ce_pieces_of_a_huge_vocabulary():
    """One token: the gradient logits' rows stay short enough for 32-bit offsets (2^20
    of 2 bytes), though 256 MiB would hold 2^27 of them."""
    assert ce_size(ce(tokens=1, width=64, vocab=1 << 27, ldh=64, ldw=64), 1)[1] < 1 << 26


@pytest.mark.parametrize("point", ["plan", "ce_pack"])
def test_forced_failure_before_the_first_launch(point, monkeypatch):
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", point)
    assert ce_fwd(ce()) == -8
    assert ce_bwd(ce()) == -8
    assert b"DMUON_TEST_FAIL_AT" in B.lib().dmuon_last_error()


def embed(ids=at(1), idt=B.I64, tokens=10, table=at(2), ldt=64, rows=100, width=64, dtype=B.BF16, scale=1.0, out=at(3)):
    return B.lib().dmuon_embedding(vp(ids), idt, tokens, vp(table), ldt, rows, width, dtype, scale, vp(out), None)


def embed_bwd(ids=at(1), idt=B.I64, tokens=10, g=at(2), ldg=64, gdt=B.BF16, rows=100, width=64, scale=1.0, pad=-1,
              out=at(3), odt=B.F32, acc=0, ws=WS, nbytes=1 << 30):
    return B.lib().dmuon_embedding_backward(vp(ids), idt, tokens, vp(g), ldg, gdt, rows, width, scale, pad, vp(out), odt,
                                            acc, vp(ws), nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(idt=3), -4), (dict(tokens=-1), -3), (dict(tokens=(1 << 30) + 1), -3), (dict(rows=-1), -3),
    (dict(rows=(1 << 30) + 1), -3), (dict(width=0), -3), (dict(width=65537), -3), (dict(scale=float("nan")), -5),
    (dict(scale=float("inf")), -5), (dict(ids=None), -1), (dict(out=None), -1), (dict(out=at(1)), -7)])
def test_embedding_refuses(kw, code):
    assert embed(**kw) == code
    assert embed_bwd(**kw) == code


def test_embedding_refuses_more():
    assert embed(dtype=9) == -4
    assert embed(ldt=63) == -3
    assert embed(table=None) == -1
    assert embed(out=at(2) + 128) == -7
    assert embed(tokens=0, ids=None, out=None) == 0
    assert embed_bwd(gdt=9) == -4
    assert embed_bwd(odt=9) == -4
    assert embed_bwd(ldg=63) == -3
    assert embed_bwd(g=None) == -1
    assert embed_bwd(acc=2) == -5
    assert embed_bwd(out=at(2) + 64) == -7
    assert embed_bwd(rows=0, out=None) == 0
    assert embed_bwd(tokens=0, ids=None, g=None, acc=1) == 0
    need = ctypes.c_size_t(0)
    assert B.lib().dmuon_embedding_backward_workspace_size(10, 100, 64, ctypes.byref(need)) == 0 and need.value > 0
    assert embed_bwd(nbytes=need.value - 1) == -6
    assert embed_bwd(ws=None) == -6
    assert embed_bwd(ws=WS + 8) == -6
    assert embed_bwd(ws=at(3)) == -7
    assert B.lib().dmuon_embedding_backward_workspace_size(10, 100, 64, None) == -1
    assert B.lib().dmuon_embedding_backward_workspace_size(0, 100, 64, ctypes.byref(need)) == 0 and need.value == 0


def quantize(x=at(1), dtype=B.BF16, rows=4, cols=64, ldx=64, q=at(2), e=at(3)):
    return B.lib().dmuon_ckpt8_quantize(vp(x), dtype, rows, cols, ldx, vp(q), vp(e), None)


def dequantize(q=at(2), e=at(3), rows=4, cols=64, out=at(1), dtype=B.BF16):
    return B.lib().dmuon_ckpt8_dequantize(vp(q), vp(e), rows, cols, vp(out), dtype, None)


@pytest.mark.parametrize("kw,code", [(dict(dtype=4), -4), (dict(rows=-1), -3), (dict(rows=(1 << 30) + 1), -3),
                                     (dict(cols=-1), -3), (dict(cols=65537), -3), (dict(q=None), -1), (dict(e=None), -1),
                                     (dict(rows=0), 0), (dict(cols=0), 0)])
def test_codec_refuses(kw, code):
    if kw.get("cols", 0) == 65537:
        assert quantize(**kw, ldx=70000) == code
    else:
        assert quantize(**kw) == code
    assert dequantize(**kw) == code


def test_codec_refuses_more():
    assert quantize(x=None) == -1
    assert quantize(ldx=63) == -3
    assert quantize(q=at(1)) == -7
    assert quantize(e=at(2) + 16) == -7
    assert dequantize(out=None) == -1
    assert dequantize(out=at(2) + 32) == -7


def wg(**kw):
    d = dict(tokens=64, n=100, k=200, grad_dtype=B.BF16, out_dtype=B.F32, grad_out=at(1), ldg=100, q=at(2), exps=at(3),
             offsets=None, groups=0, reserved=0, out=at(4))
    d.update(kw)
    return B.Ckpt8WgradProblem(*[d[n] for n, _ in B.Ckpt8WgradProblem._fields_])


def wg_run(p, ws=WS, nbytes=1 << 39):
    return B.lib().dmuon_ckpt8_wgrad(ctypes.byref(p), vp(ws), nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(grad_dtype=3), -4), (dict(out_dtype=3), -4), (dict(tokens=-1), -3), (dict(tokens=(1 << 24) + 1), -3),
    (dict(n=0, ldg=0), -3), (dict(k=0), -3), (dict(n=65537, ldg=65537), -3), (dict(k=65537), -3), (dict(ldg=99), -3),
    (dict(groups=-1), -3), (dict(groups=(1 << 20) + 1, offsets=at(6)), -3), (dict(groups=2), -1), (dict(reserved=1), -3),
    (dict(grad_out=None), -1), (dict(q=None), -1), (dict(exps=None), -1), (dict(out=None), -1), (dict(out=at(1)), -7),
    (dict(out=at(2) + 64), -7), (dict(offsets=at(4), groups=2), -7), (dict(n=65536, ldg=65536, k=65536, offsets=at(6), groups=1 << 20), -3)])
def test_wgrad_refuses(kw, code):
    assert wg_run(wg(**kw)) == code


def test_wgrad_workspace():
    need = ctypes.c_size_t(0)
    p = wg()
    assert B.lib().dmuon_ckpt8_wgrad_workspace_size(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value > 0
    assert wg_run(p, nbytes=need.value - 1) == -6
    assert wg_run(p, ws=None) == -6
    assert wg_run(p, ws=at(4)) == -7
    assert B.lib().dmuon_ckpt8_wgrad_workspace_size(ctypes.byref(p), None) == -1
    assert B.lib().dmuon_ckpt8_wgrad_workspace_size(None, ctypes.byref(need)) == -1
    assert wg_run(wg(offsets=at(6), groups=0, out=None)) == 0


# ---- the Python face ------------------------------------------------------------------
def test_python_refuses_cpu_tensors():
    x = torch.zeros(4, 8)
    y = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: mm.linear_cross_entropy(x, x, y),
                 lambda: mm.linear_cross_entropy_backward(x, x, y, y, y),
                 lambda: mm.embedding(y, x),
                 lambda: mm.embedding_backward(y, x, 10),
                 lambda: mm.checkpoint_quantize(x),
                 lambda: mm.checkpoint_dequantize(x.to(torch.int8), x.to(torch.uint8)),
                 lambda: mm.checkpoint_wgrad(x, x.to(torch.int8), x.to(torch.uint8)),
                 lambda: mm.embedding([1, 2], x), lambda: mm.linear_cross_entropy(None, x, y)):
        with pytest.raises(ValueError):
            call()
