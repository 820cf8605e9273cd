"""The largest sizes and strides that the training-gradient entry points accept, and what
lies past them (no GPU needed: a refused call makes no HIP call, an accepted one fails at
its first launch here; pointers are never dereferenced)."""
import ctypes
import os

import pytest

from matrix_optimizer_muon_amd import _binding as B
from test_training_host import at, ce, ce_bwd, ce_fwd, ce_size, embed, embed_bwd, quantize, wg, wg_run

HIP = -8                     # accepted; stopped at the point that the test names, before a launch
SHAPE = -3


@pytest.fixture
def stop(monkeypatch):
    """Accepted calls end after validation and planning, with DMUON_E_HIP."""
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", "plan")


def longest(rows, cols, es):
    """The longest stride at which rows × cols elements end within 2^48 bytes."""
    return min(((1 << 48) // es - cols) // (rows - 1), 1 << 40)


@pytest.mark.parametrize("dtype,es", [(B.BF16, 2), (B.F32, 4)])
def test_strides_past_the_largest_matrix(stop, dtype, es):
    """A product of rows, stride and element size past 63 bits wrapped, and the buffer
    then took no part in the overlap check."""
    far = 1 << 40
    # each operand alone: the longest stride is taken, one more and the largest of all refused
    for rows, cols, call in (
            (1 << 24, 128, lambda ld, n: ce_fwd(ce(tokens=n, vocab=100, dtype=dtype, ldh=ld, h=1 << 12, w=1 << 55, targets=2 << 55),
                                                losses=3 << 55, lse=4 << 55, ws=5 << 55, nbytes=1 << 50)),
            (1 << 30, 128, lambda ld, n: ce_fwd(ce(vocab=n, dtype=dtype, ldw=ld, w=1 << 12, h=1 << 55, targets=2 << 55),
                                                losses=3 << 55, lse=4 << 55, ws=5 << 55, nbytes=1 << 50)),
            (1 << 30, 64, lambda ld, n: embed(rows=n, ldt=ld, dtype=dtype, table=1 << 12, ids=1 << 55, out=2 << 55)),
            (1 << 28, 64, lambda ld, n: embed_bwd(tokens=n, ldg=ld, gdt=dtype, g=1 << 12, ids=1 << 55, out=2 << 55, ws=3 << 55,
                                                  nbytes=1 << 50)),
            (1 << 30, 64, lambda ld, n: quantize(rows=n, ldx=ld, dtype=dtype, x=1 << 12, q=1 << 55, e=2 << 55)),
            (1 << 24, 100, lambda ld, n: wg_run(wg(tokens=n, ldg=ld, grad_dtype=dtype, grad_out=1 << 12, q=1 << 55, exps=2 << 55,
                                                   out=3 << 55), ws=5 << 55, nbytes=1 << 50))):
        ok = longest(rows, cols, es)
        assert call(ok, rows) == HIP
        assert call(ok + 1, rows) == SHAPE
        assert call(far, rows) == SHAPE
        assert call(far, 1) == HIP                             # one row: no stride is taken
    # the size queries look at the strides too
    assert ce_size(ce(tokens=1 << 24, ldh=far))[0] == SHAPE
    assert ce_size(ce(vocab=1 << 30, ldw=far), 1)[0] == SHAPE


def test_a_far_reaching_buffer_takes_part_in_the_overlap_check(stop):
    """h reaches 2^44 bytes: an output inside it is refused."""
    p = ce(tokens=1 << 20, ldh=1 << 23)
    assert ce_fwd(p, losses=at(1) + (1 << 43), nbytes=1 << 50) == -7


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("dtype", [B.BF16, B.F32])
def test_sizes_at_the_limits_have_a_workspace(backward, dtype):
    """Planning at the ends of every range: no overflow, a size that fits 63 bits."""
    for kw in (dict(tokens=1 << 24, vocab=100), dict(tokens=64, vocab=1 << 30), dict(tokens=1, vocab=1 << 30, width=65536, ldh=65536, ldw=65536),
               dict(tokens=1 << 24, width=1, ldh=1, ldw=1, vocab=16256), dict(tokens=1, width=1, ldh=1, ldw=1, vocab=1),
               dict(tokens=1 << 20, width=8192, ldh=8192, ldw=8192, vocab=1 << 17)):
        rc, size = ce_size(ce(dtype=dtype, **kw), backward)
        assert rc == 0 and 0 < size < 1 << 50, kw
    out = ctypes.c_size_t(0)
    for kw in (dict(tokens=1 << 24), dict(tokens=1 << 24, n=65536, ldg=65536, k=65536), dict(tokens=1 << 24, offsets=at(6), groups=1 << 20)):
        p = wg(grad_dtype=dtype, **kw)
        assert B.lib().dmuon_ckpt8_wgrad_workspace_size(ctypes.byref(p), ctypes.byref(out)) == 0 and 0 < out.value < 1 << 55


def test_launches_of_the_table_gradient_hold_fewer_than_2_32_threads(stop):
    """Refused before anything is enqueued; they were accepted and failed at a launch
    behind the sort."""
    need = ctypes.c_size_t(0)
    for tokens, rows, width, rc in ((1 << 29, 100, 8, SHAPE), ((1 << 29) - 64, 100, 8, HIP), (1 << 28, 100, 1024, SHAPE),
                                    ((1 << 28) - 256, 100, 1024, HIP), (1 << 22, 100, 65536, SHAPE), (1000, 1 << 30, 64, HIP),
                                    (1000, 1 << 28, 65536, SHAPE)):
        got = embed_bwd(tokens=tokens, rows=rows, width=width, ldg=width, ids=1 << 40, g=1 << 50, out=1 << 52, ws=1 << 55, nbytes=1 << 50)
        assert got == rc, (tokens, rows, width)
        size = B.lib().dmuon_embedding_backward_workspace_size(tokens, rows, width, ctypes.byref(need))
        assert (size == SHAPE) == (rc == SHAPE)
    # the lookup's launch walks over its rows and takes them all
    assert embed(tokens=1 << 30, rows=1 << 30, width=8, ids=1 << 40, table=1 << 50, out=1 << 52) == HIP


def test_launches_of_the_cross_entropy_hold_fewer_than_2_32_threads(stop):
    p = ce(tokens=1 << 24, width=32768, ldh=32768, ldw=32768, vocab=100, h=1 << 46, w=1 << 50, targets=1 << 51)
    far = dict(lse=1 << 52, ws=1 << 56, nbytes=1 << 54)
    assert ce_bwd(p, gl=1 << 53, gh=1 << 54, gw=1 << 55, **far) == SHAPE
    assert ce_size(p, 1)[0] == SHAPE and ce_size(p, 0)[0] == 0
    assert ce_fwd(p, losses=1 << 53, **far) == HIP
    # few tokens: a workgroup per 64 words up to 2^30 − 64 of them, then tiles of 128
    # (8 bytes of statistics per token and either)
    few, tiles = ce_size(ce(tokens=1, vocab=(1 << 30) - 64))[1], ce_size(ce(tokens=1, vocab=1 << 30))[1]
    assert few > (1 << 27) - 64 and tiles < (1 << 26) + (1 << 16)
