"""Cross entropy whose vocabulary goes through in several pieces (needs an MI355X)."""
import torch
import pytest

from test_gpu_training import gen, mm, randn

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
