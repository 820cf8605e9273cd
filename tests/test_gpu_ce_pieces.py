"""Cross entropy whose vocabulary goes through in several pieces (needs an MI355X)."""
import torch
import pytest

from test_gpu_training import U, ce_inputs, ce_reference, gen, mm, randn, within

pytestmark = pytest.mark.gpu


def test_more_tiles_than_a_launch_holds():
    """2^21 tokens × 2^17 words: 2^24 tiles of 256 threads, one too many for a launch;
    the losses are those of the two halves of the tokens to the bit."""
    m = mm()
    g = gen(3)
    T, D, V = 1 << 21, 64, 1 << 17
    h = randn(g, T, D).to(torch.bfloat16)
    w = (randn(g, V, D) * 0.2).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    m.phase_timing(True)
    m.phase_timing_read()
    losses, lse = m.linear_cross_entropy(h, w, y)
    launches = m.phase_timing_read()["ce_logits"][1]
    m.phase_timing(False)
    assert launches == 2
    half = T // 2
    for s in (slice(0, half), slice(half, T)):
        a, b = m.linear_cross_entropy(h[s], w, y[s])
        assert torch.equal(losses[s], a) and torch.equal(lse[s], b)
    z = h[-50:].double() @ w.double().T                         # and some of them the definition's
    want = torch.logsumexp(z, 1) - z.gather(1, y[-50:, None].long())[:, 0]
    assert ((losses[-50:].double() - want).abs() <= 1e-4 * (1 + want)).all()


# Copies of w (rows off the 16-byte grid, odd widths, fp32 planes) in several pieces, the
# last one shorter: the forward pass from 256 MiB of copied rows on, the backward pass from
# 256 MiB of gradient logits and rows.  The bounds are those of ce_reference.
@pytest.mark.parametrize("T,D,V,shift,dtype", [
    (70, 2048, 32000, 0, torch.float32),          # fp32, 12 KiB of planes a row: 21845 rows a piece
    (40, 1500, 95001, 1, torch.float32),          # few tokens forward (no copy), 29127 rows a piece backward
    (70, 1234, 120001, 0, torch.bfloat16),        # odd width: 104857 rows a piece forward
    (300, 2048, 70000, 1, torch.bfloat16),        # shifted rows: 65536 a piece
    (9000, 64, 6001, 0, torch.float32),           # 4944 rows a piece backward
    (9001, 72, 16500, 1, torch.bfloat16)])        # 14708 rows a piece backward
def test_several_pieces_of_a_copied_vocabulary(T, D, V, shift, dtype):
    m = mm()
    h, w, y, gl = ce_inputs(T, D + shift, V, dtype, 40 + T)
    h, w = h[:, shift:], w[:, shift:]
    m.phase_timing(True)
    m.phase_timing_read()
    losses, lse = m.linear_cross_entropy(h, w, y)
    forward = m.phase_timing_read()["ce_logits"][1]
    dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, gl)
    backward = m.phase_timing_read()["ce_logits"][1]
    m.phase_timing(False)
    assert backward > 1 and (forward > 1 or T in (40, 9000, 9001))
    tol_w = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    ref_w = torch.zeros_like(tol_w)
    for a in range(0, T, 1024):                   # some tokens at a time
        t = slice(a, a + 1024)
        ref = ce_reference(h[t], w, y[t], gl[t])
        within(losses[t], ref["loss"], ref["tol"], "loss")
        within(lse[t], ref["lse"], ref["tol"], "lse")
        ref = ce_reference(h[t], w, y[t], gl[t], lse[t])
        within(dh[t], ref["dh"], ref["tol_h"], "dh")
        ref_w += ref["dw"]
        tol_w += ref["tol_w"]
    # the parts' bounds have the summands' error and that of 1024 additions each; all T of
    # them together at most T/1024 times that, and the last rounding of the whole sum
    parts = -(-T // 1024)
    within(dw, ref_w, tol_w * parts + U[dtype] * ref_w.abs(), "dw")


@pytest.mark.parametrize("T,D,V,dtype", [(70, 2048, 32000, torch.float32), (2001, 800, 140000, torch.bfloat16)])
def test_pieces_repeat_to_the_bit(T, D, V, dtype):
    m = mm()
    h, w, y, gl = ce_inputs(T, D, V, dtype, 44)
    first = None
    for _ in range(3):
        losses, lse = m.linear_cross_entropy(h, w, y)
        got = [losses, lse, *m.linear_cross_entropy_backward(h, w, y, lse, gl)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
