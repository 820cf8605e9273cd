"""Log probabilities and entropies from hidden states, and their gradients, against fp64
(needs an MI355X).

Tolerances are worst-case bounds, element by element.  A logit summed from D products is
off by ez = (D + 16)·2^-23·Σ|h||w| (each addition by at most 2^-24 of the running sum of
magnitudes, doubled for the matrix core's alignment), times the scale; then, with
k1 = Σ p·|x − X| and k2 = Σ p·(x − X)²:

* exp, log, the sums over the vocabulary: soft = (100 + V/4096)·2^-24 relative, and
  3·2^-24·k1 from the exponents;
* the log probability moves by at most twice the largest ez of its row, the entropy by
  2·max ez·(k1 + 1) (its derivative is −p·(log p + H));
* dz from a probability off by (ez + 2^-20)·p and an l off by ez; rounded to bf16 once
  (2^-8; three planes for fp32: 2^-22); sums of V or T products: (V + 64)·2^-23.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
IGNORE = -100
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])


def mm():
    import matrix_optimizer_muon_amd
    return matrix_optimizer_muon_amd


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def within(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    ok = (got - want).abs() <= tol + 1e-300
    ok |= torch.isnan(want) | (got == want)
    bad = (~ok).sum().item()
    assert bad == 0, f"{what}: {bad} of {want.numel()} elements outside, worst {torch.nan_to_num((got - want).abs() / (tol + 1e-300)).max().item():.3g}"


def forward_reference(h, w, y, scale):
    T, D = h.shape
    V = w.shape[0]
    kept = y != IGNORE
    inside = kept & (y >= 0) & (y < V)
    hd, wd = torch.where(kept[:, None], h.double(), 0.0), w.double()
    x = hd @ wd.T * scale
    ex = (D + 16) * 2.0 ** -23 * (hd.abs() @ wd.abs().T) * scale + 2.0 ** -24 * x.abs()
    ez = ex.amax(1)
    lse = torch.logsumexp(x, 1)
    log_p = x - lse[:, None]
    p = log_p.exp()
    H = -torch.special.xlogy(p, p).sum(1)
    far = (x.amax(1, keepdim=True) - x)
    k1, k2 = (p * far).sum(1), (p * far * far).sum(1)
    soft = (100 + V / 4096) * 2.0 ** -24
    at = torch.where(inside, y, 0).long()[:, None]
    lp = torch.where(inside, log_p.gather(1, at)[:, 0], torch.where(y == -2 ** 31, -lse, math.nan))
    tol = 2 * ez + soft + 3 * 2.0 ** -24 * k1 + 2.0 ** -22 * (lse.abs() + log_p.gather(1, at)[:, 0].abs())
    t_H = 2 * ez * (k1 + 1) + soft * (1 + 2 * k1) + 6 * 2.0 ** -24 * (k1 + k2) + 2.0 ** -22 * (lse - x.amax(1) + k1)
    zero = lambda v: torch.where(kept, v, 0.0)  # noqa: E731
    return {"logprobs": zero(lp), "lse": zero(lse), "entropy": zero(H), "tol": tol, "t_entropy": t_H, "x": x, "ex": ex}


def gradient_reference(h, w, y, r, f, g, e, scale):
    t, (T, D), V = h.dtype, h.shape, w.shape[0]
    zero = torch.zeros(T, dtype=torch.float64, device=h.device)
    g = zero if g is None else g.double()
    e = zero if e is None else e.double()
    inside = (y >= 0) & (y < V)
    use = (y != IGNORE) & (inside | (y == -2 ** 31)) & ~((g == 0) & (e == 0))
    l = f["x"] - r.lse.double()[:, None]
    H = (r.entropy.double() if e.any() else zero)[:, None]
    p = l.exp()
    inner = g[:, None] + e[:, None] * (l + H)
    d = -p * inner
    d.scatter_add_(1, torch.where(inside, y, 0).long()[:, None], torch.where(inside, g, 0.0)[:, None])
    dz = torch.where(use[:, None], d * scale, 0.0)
    e_l = f["ex"] + 2.0 ** -23 * l.abs()
    mag = g.abs()[:, None] + e.abs()[:, None] * (l.abs() + H.abs())
    err = p * (e_l + 2.0 ** -20) * (mag + e.abs()[:, None]) + 2.0 ** -22 * (p * mag + d.abs()) + 2.0 ** -126 * (1 + mag)
    u = U[t] if t == torch.bfloat16 else 2.0 ** -22
    err = torch.where(use[:, None], scale * (u * (d.abs() + err) + err) * (1 + 2.0 ** -20), 0.0)
    hd, wd = torch.where(use[:, None], h.double(), 0.0), w.double()
    out = []
    for want, e_sum, mags, n in ((dz @ wd, err @ wd.abs(), (dz.abs() + err) @ wd.abs(), V), (dz.T @ hd, err.T @ hd.abs(), (dz.abs() + err).T @ hd.abs(), T)):
        tol = e_sum + (n + 64) * 2.0 ** -23 * mags + (n + 2) * 2.0 ** -126
        out.append((want, tol + U[t] * (want.abs() + tol)))
    return out


def check(h, w, y, g, e, scale=1.0, what=""):
    m = mm()
    f = forward_reference(h, w, y.long(), scale)
    r = m.linear_token_logprobs(h, w, y, scale=scale)
    assert r.top_ids is None
    within(r.logprobs, f["logprobs"], f["tol"], what + " logprobs")
    within(r.lse, f["lse"], f["tol"], what + " lse")
    within(r.entropy, f["entropy"], f["t_entropy"], what + " entropy")
    (dh, th), (dw, tw) = gradient_reference(h, w, y.long(), r, f, g, e, scale)
    got_h, got_w = m.linear_token_logprobs_backward(h, w, y, r.lse, r.entropy, g, e, scale=scale)
    assert got_h.dtype == h.dtype and got_w.dtype == w.dtype
    within(got_h, dh, th, what + " dh")
    within(got_w, dw, tw, what + " dw")
    return r, got_h, got_w


def inputs(T, D, V, dtype, seed, ignored=0.2, index=torch.int64):
    g = gen(seed)
    h = randn(g, T, D).to(dtype)
    w = (randn(g, V, D) * (1.5 / math.sqrt(D))).to(dtype)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.where(torch.rand(T, generator=g, device="cuda") < ignored, IGNORE, y).to(index)
    return h, w, y, randn(g, T) / T, -0.05 * torch.rand(T, generator=g, device="cuda") / T


SIZES = [(1, 1, 1), (1, 64, 2), (3, 7, 5), (2, 64, 257), (17, 100, 255), (33, 65, 300), (64, 128, 1000), (255, 64, 256), (256, 192, 511),
         (257, 256, 513), (300, 320, 2049), (600, 72, 700), (4100, 800, 3333)]


@TYPES
@pytest.mark.parametrize("T,D,V", SIZES)
def test_sizes(T, D, V, dtype):
    check(*inputs(T, D, V, dtype, 1000 + T, ignored=0.0 if T < 4 else 0.2), what=f"{T}x{D}x{V}")


@TYPES
@pytest.mark.parametrize("scale", [2.0 ** -10, 0.7, 3.0])
@pytest.mark.parametrize("T", [20, 300])
def test_scale(T, scale, dtype):
    check(*inputs(T, 96, 777, dtype, 5), scale=scale)


@TYPES
@pytest.mark.parametrize("T", [24, 280])
def test_targets_and_weights(T, dtype):
    h, w, y, g, e = inputs(T, 128, 700, dtype, 6, index=torch.int32)
    y[1::8] = -1
    y[2::8] = 700
    y[3::8] = -2 ** 31
    e[4::8] = 0
    g[4::16] = 0
    g[5::16] = 0
    r, dh, dw = check(h, w, y, g, e)
    # ignored rows are not read, whatever they hold
    h2 = h.clone()
    h2[y == IGNORE] = math.nan
    for s, t in zip((*r[:3], dh, dw), [t for v in check_only(h2, w, y, g, e) for t in v]):
        assert torch.equal(torch.nan_to_num(s, 7.0), torch.nan_to_num(t, 7.0))
    # one gradient alone; one result alone
    check(h, w, y, g, None)
    check(h, w, y, None, e)
    a, b = mm().linear_token_logprobs_backward(h, w, y, r.lse, r.entropy, g, e, need_w=False)
    assert torch.equal(a, dh) and b is None
    a, b = mm().linear_token_logprobs_backward(h, w, y, r.lse, r.entropy, g, e, need_h=False)
    assert a is None and torch.equal(b, dw)
    # no token at all
    none = torch.full_like(y, IGNORE)
    r = mm().linear_token_logprobs(h, w, none)
    for t in (*r[:3], *mm().linear_token_logprobs_backward(h, w, none, r.lse, r.entropy, g, e)):
        assert not t.any()


def check_only(h, w, y, g, e):
    r = mm().linear_token_logprobs(h, w, y)
    return r[:3], mm().linear_token_logprobs_backward(h, w, y, r.lse, r.entropy, g, e)


@TYPES
@pytest.mark.parametrize("T", [20, 200])
def test_agrees_with_the_loss(T, dtype):
    """Without an entropy's weight the gradients are the negated loss's.  The statistics of
    the tiles are joined with other roundings: 10 of 2^-24 of the sums in ten steps, of
    logarithms below 16."""
    m = mm()
    h, w, y, g, _ = inputs(T, 256, 1500, dtype, 7)
    losses, lse = m.linear_cross_entropy(h, w, y)
    r = m.linear_token_logprobs(h, w, y)
    assert (r.lse - lse).abs().max() <= 2.0 ** -18 and (r.logprobs + losses).abs().max() <= 2.0 ** -18
    a = m.linear_cross_entropy_backward(h, w, y, lse, -g)
    b = m.linear_token_logprobs_backward(h, w, y, lse, None, g)
    for s, t in zip(a, b):       # p and the target's 1 in one rounding more or less: two roundings of dz
        assert torch.linalg.norm((s - t).double()) <= 2 * U[dtype] * torch.linalg.norm(s.double()) + 2.0 ** -20 * torch.linalg.norm(s.double())


@TYPES
@pytest.mark.parametrize("T", [30, 300])
def test_words_masked_out_and_infinite_states(T, dtype):
    """A word whose weights give −∞ has probability 0 and adds nothing to the entropy; a row
    of −∞ alone has none; a NaN stays in its row."""
    m = mm()
    h, w, y, g, e = inputs(T, 64, 600, dtype, 8, ignored=0.0)
    h[:, 0] = h[:, 0].abs() + 0.5
    w[:, 0] = 0
    masked = torch.arange(600, device="cuda") % 3 == 0
    y = y // 3 * 3 + 1
    w2 = w.clone()
    w2[masked] = 0
    w2[masked, 0] = -math.inf
    r = m.linear_token_logprobs(h, w2, y)
    keep = (~masked).nonzero()[:, 0]
    f = forward_reference(h, w[keep], torch.searchsorted(keep, y), 1.0)
    within(r.logprobs, f["logprobs"], f["tol"], "logprobs")
    within(r.entropy, f["entropy"], f["t_entropy"], "entropy")
    dh, dw = m.linear_token_logprobs_backward(h, w2, y, r.lse, r.entropy, g, e)
    assert not dw[masked].any() and torch.isfinite(dw).all()
    # rows of −∞ alone
    w3 = torch.zeros_like(w)
    w3[:, 0] = -math.inf
    r = m.linear_token_logprobs(h, w3, y)
    assert (r.lse == -math.inf).all() and (r.logprobs == -math.inf).all() and not r.entropy.any()
    dh, dw = m.linear_token_logprobs_backward(h, w3, y, r.lse, r.entropy, g, e)
    assert not dw.any()
    # NaN
    h[3, 5] = math.nan
    r = m.linear_token_logprobs(h, w, y)
    assert torch.equal(torch.isnan(r.lse).nonzero()[:, 0], torch.tensor([3], device="cuda"))
    assert torch.isnan(r.entropy[3]) and torch.isnan(r.logprobs[3]) and torch.isfinite(r.entropy).sum() == T - 1
    dh, _ = m.linear_token_logprobs_backward(h, w, y, r.lse, r.entropy, g, e)
    assert torch.isnan(dh[3]).all() and torch.isnan(dh).sum() == 64


@TYPES
def test_strided_rows_and_pieces(dtype):
    """Rows off the 16-byte grid, and a vocabulary in several pieces."""
    h, w, y, g, e = inputs(150, 67, 9000, dtype, 9)
    hb, wb = torch.full((150, 71), math.nan, device="cuda", dtype=dtype), torch.full((9000, 70), math.nan, device="cuda", dtype=dtype)
    hb[:, 3:70], wb[:, 1:68] = h, w
    a, b = check_only(h, w, y, g, e), check_only(hb[:, 3:70], wb[:, 1:68], y, g, e)
    for s, t in zip((*a[0], *a[1]), (*b[0], *b[1])):
        assert torch.equal(s, t)
    h, w, y, g, e = inputs(20000, 64, 10000, dtype, 10)
    f, r = forward_reference(h[:64], w, y[:64], 1.0), mm().linear_token_logprobs(h, w, y)
    within(r.entropy[:64], f["entropy"], f["t_entropy"], "entropy")
    dh, dw = mm().linear_token_logprobs_backward(h, w, y, r.lse, r.entropy, g, e)
    y2 = torch.where(torch.arange(20000, device="cuda") < 64, y, IGNORE)       # the same tokens in one piece
    dh2, _ = mm().linear_token_logprobs_backward(h, w, y2, r.lse, r.entropy, g, e)
    small = [t[:64] for t in (h, y, g, e)]
    r64 = type(r)(*(t[:64] if t is not None else None for t in r))
    (want, tol), _ = gradient_reference(small[0], w, small[1], r64, f, small[2], small[3], 1.0)
    within(dh[:64], want, tol, "dh in pieces")
    within(dh2[:64], want, tol, "dh of the first tokens")


def test_shards():
    h, w, y, g, e = inputs(120, 96, 2000, torch.float32, 11)
    m = mm()
    cuts = [0, 300, 1111, 2000]
    shifted = [torch.where(y == IGNORE, IGNORE, torch.where((y >= a) & (y < b), y - a, m.TARGET_ELSEWHERE)) for a, b in zip(cuts, cuts[1:])]
    parts = [m.linear_token_logprobs(h, w[a:b], t) for a, b, t in zip(cuts, cuts[1:], shifted)]
    kept = y != IGNORE
    lses = torch.stack([p.lse for p in parts]).double()
    lse = torch.logsumexp(lses, 0)
    H = lse - sum(torch.exp(s - lse) * (s - p.entropy.double()) for s, p in zip(lses, parts))
    lp = sum(p.logprobs.double() + p.lse.double() for p in parts) - lse
    f = forward_reference(h, w, y, 1.0)
    zero = lambda v: torch.where(kept, v, 0.0)  # noqa: E731
    within(zero(lp), f["logprobs"], 4 * f["tol"] + 2.0 ** -20, "logprobs")
    within(zero(H), f["entropy"], 4 * f["t_entropy"] + 4 * f["tol"] + 2.0 ** -18, "entropy")
    r = type(parts[0])(None, zero(H).float(), zero(lse).float())
    (dh, th), (dw, tw) = gradient_reference(h, w, y, r, f, g, e, 1.0)
    outs = [m.linear_token_logprobs_backward(h, w[a:b], t, r.lse, r.entropy, g, e) for a, b, t in zip(cuts, cuts[1:], shifted)]
    within(sum(o[0].double() for o in outs), dh, 3 * th, "dh")
    within(torch.cat([o[1] for o in outs]), dw, 3 * tw, "dw")


def test_gradients_against_differences():
    """Central differences of Σ g·logprob + e·entropy in fp64 along random directions: the
    step of 2^-12 leaves its square times the third derivative, below 2^-10 of the
    gradient's scale here, and the fp32 gradient its rounding."""
    h, w, y, g, e = inputs(12, 16, 30, torch.float32, 12)
    e = e * 20
    r = mm().linear_token_logprobs(h, w, y, scale=1.5)
    dh, dw = mm().linear_token_logprobs_backward(h, w, y, r.lse, r.entropy, g, e, scale=1.5)
    kept = y != IGNORE

    def f(h, w):
        lp = torch.log_softmax(h @ w.T * 1.5, 1)
        v = g.double() * lp.gather(1, y.clamp(min=0)[:, None])[:, 0] - e.double() * (lp.exp() * lp).sum(1)
        return torch.where(kept, v, 0.0).sum().item()
    rng = gen(13)
    for _ in range(10):
        a, b = randn(rng, *h.shape).double(), randn(rng, *w.shape).double()
        s = 2.0 ** -12
        num = (f(h.double() + s * a, w.double() + s * b) - f(h.double() - s * a, w.double() - s * b)) / (2 * s)
        want = (dh.double() * a).sum().item() + (dw.double() * b).sum().item()
        size = (torch.linalg.norm(dh.double()) * torch.linalg.norm(a) + torch.linalg.norm(dw.double()) * torch.linalg.norm(b)).item()
        assert abs(num - want) <= 2.0 ** -10 * size


@TYPES
def test_same_bits_streams_and_graphs(dtype):
    m = mm()
    h, w, y, g, e = inputs(300, 128, 3001, dtype, 14)
    r, grads = check_only(h, w, y, g, e)
    want = (*r, *grads)
    for _ in range(2):
        a, b = check_only(h, w, y, g, e)
        for s, t in zip(want, (*a, *b)):
            assert torch.equal(s, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = m.linear_token_logprobs(h, w, y, stream=side)
    b = m.linear_token_logprobs_backward(h, w, y, r[2], r[1], g, e, stream=side)
    for _ in range(10):
        torch.empty_like(w).fill_(3.0)
    side.synchronize()
    for s, t in zip(want, (*a[:3], *b)):
        assert torch.equal(s, t)
    h2, _, y2, _, _ = inputs(300, 128, 3001, dtype, 15, ignored=0.7)
    other = check_only(h2, w, y2, g, e)
    hs, ys = h.clone(), y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = m.linear_token_logprobs(hs, w, ys)
        b = m.linear_token_logprobs_backward(hs, w, ys, a.lse, a.entropy, g, e)
    for hx, yx, ref in ((h, y, want), (h2, y2, (*other[0], *other[1])), (h, y, want)):
        hs.copy_(hx)
        ys.copy_(yx)
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip((*a[:3], *b), ref):
            assert torch.equal(s, t)
        check_only(h2, w, y, g, e)
