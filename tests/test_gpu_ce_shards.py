"""Cross entropy over a vocabulary in shards: each call has some rows of w and the
targets shifted to them, and the joined results are those of the whole (needs an MI355X)."""
import math

import pytest
import torch

from test_gpu_training import IGNORE, U, ce_inputs, ce_reference, mm, within

pytestmark = pytest.mark.gpu


def shard_targets(y, first, rows):
    at = torch.where(y == IGNORE, IGNORE, y - first)
    return torch.where((y != IGNORE) & ((at < 0) | (at >= rows)), mm().TARGET_ELSEWHERE, at)


@pytest.mark.parametrize("index", [torch.int64, torch.int32])
@pytest.mark.parametrize("T,D,V,cuts,dtype", [(20, 64, 900, [300], torch.bfloat16), (20, 72, 500, [77, 400], torch.float32),
                                              (300, 128, 1000, [1, 640], torch.bfloat16), (200, 64, 700, [333], torch.float32),
                                              (2001, 800, 13000, [6500], torch.bfloat16)])
def test_shards_join_to_the_whole(T, D, V, cuts, dtype, index):
    m = mm()
    h, w, y, gl = ce_inputs(T, D, V, dtype, 70 + T)
    if T > 100:
        gl[5] = 0.0                                            # left out, in whichever shard its target is
    edges = [0, *cuts, V]
    parts = [(w[a:b], shard_targets(y, a, b - a).to(index)) for a, b in zip(edges, edges[1:])]
    ref = ce_reference(h, w, y, None)
    got = [m.linear_cross_entropy(h, ws, ys) for ws, ys in parts]
    keep = y != IGNORE
    lses = torch.stack([l for _, l in got]).double()
    # a shard's lse is that of its own rows, and its loss where the target is elsewhere
    for (ws, ys), (loss, lse) in zip(parts, got):
        own = ce_reference(h, ws, torch.where(ys == m.TARGET_ELSEWHERE, 0, ys).long(), None)
        within(lse, own["lse"], own["tol"], "shard's lse")
        away = ys == m.TARGET_ELSEWHERE
        assert torch.equal(loss[away], lse[away]) and not loss[~keep].any() and not lse[~keep].any()
    lse = torch.where(keep, torch.logsumexp(lses, 0), 0.0)
    loss = torch.where(keep, lse - (lses - torch.stack([l for l, _ in got]).double()).sum(0), 0.0)
    # the shards' own errors, each within the whole's bound, and the roundings of their values
    tol = (len(parts) + 1) * (ref["tol"] + 2.0 ** -22 * (ref["lse"].abs() + 20))
    within(lse, ref["lse"], tol, "lse")
    within(loss, ref["loss"], tol, "loss")
    joined = lse.float()
    ref = ce_reference(h, w, y, gl, joined)
    dh = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(dh)                                # what the shards' results were rounded at
    for (ws, ys), a in zip(parts, edges):
        gh, gw = m.linear_cross_entropy_backward(h, ws, ys, joined, gl)
        rows = slice(a, a + ws.shape[0])
        within(gw, ref["dw"][rows], ref["tol_w"][rows], "dw")
        dh += gh.double()
        size += gh.double().abs()
        assert not gh[~keep].any()
    # every shard's own bound sums to the whole's, but for the roundings of the shards' results
    within(dh, ref["dh"], ref["tol_h"] * len(parts) + U[dtype] * size, "dh")


def test_elsewhere_may_be_the_ignored_index_and_other_targets_stay_out():
    m = mm()
    h, w, y, gl = ce_inputs(100, 64, 300, torch.bfloat16, 71, ignored=0.0)
    a = y.clone()
    a[3] = m.TARGET_ELSEWHERE
    losses, lse = m.linear_cross_entropy(h, w, a, ignore_index=m.TARGET_ELSEWHERE)
    dh, _ = m.linear_cross_entropy_backward(h, w, a, lse, gl, ignore_index=m.TARGET_ELSEWHERE)
    assert losses[3] == 0 and lse[3] == 0 and not dh[3].any()
    for other in (m.TARGET_ELSEWHERE + 1, m.TARGET_ELSEWHERE - 1, -1, 300):
        a[3] = other
        losses, lse = m.linear_cross_entropy(h, w, a)
        dh, _ = m.linear_cross_entropy_backward(h, w, a, lse, gl)
        assert math.isnan(losses[3]) and math.isfinite(lse[3]) and not dh[3].any()


@pytest.mark.parametrize("T,dtype", [(20, torch.bfloat16), (300, torch.bfloat16), (200, torch.float32)])
def test_no_target_here_at_all(T, dtype):
    """A shard that holds none of the targets: the gradient of Σ g·lse."""
    m = mm()
    h, w, y, gl = ce_inputs(T, 64, 500, dtype, 72, ignored=0.0)
    none = torch.full_like(y, m.TARGET_ELSEWHERE)
    losses, lse = m.linear_cross_entropy(h, w, none)
    assert torch.equal(losses, lse)
    dh, dw = m.linear_cross_entropy_backward(h, w, none, lse, gl)
    p = torch.exp(h.double() @ w.double().T - lse.double()[:, None]) * gl.double()[:, None]
    # as in ce_reference, for rows of probabilities
    e = p * ((64 + 16) * 2.0 ** -23 * (h.double().abs() @ w.double().abs().T) + 2.0 ** -20 + 2.0 ** -22 * 40) + 2.0 ** -126
    e = e + (U[dtype] if dtype == torch.bfloat16 else 2.0 ** -22) * (p + e)
    for got, want, err, n in ((dh, p @ w.double(), (e + (500 + 64) * 2.0 ** -23 * (p + e)) @ w.double().abs(), 500),
                              (dw, p.T @ h.double(), (e + (T + 64) * 2.0 ** -23 * (p + e)).T @ h.double().abs(), T)):
        tol = err + (n + 2) * 2.0 ** -126
        within(got, want, tol + U[dtype] * (want.abs() + tol))
