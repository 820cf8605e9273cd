"""Training-gradient operators against plain fp64 implementations (needs an MI355X).

Tolerances are worst-case bounds, element by element, from the arithmetic:

* a product of K bf16 (or fp32) pairs summed in fp32 is off by at most
  (K + 16)·2^-23·Σ|a||b| (each addition rounds by at most 2^-24 of the running sum
  of magnitudes; the factor 2 covers the matrix core's internal alignment);
* a rounding to bf16 is off by 2^-8 of the value, to fp32 by 2^-24;
* exp, log and the sums of the softmax: (100 + V/4096)·2^-24 relative, on top of the
  error of the logits, which passes to lse and loss as it is;
* 2^-126 is the smallest normal fp32 and bf16 value: a probability, a product, a sum
  or a result below it may become 0, so each of those adds up to 2^-126.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
IGNORE = -100


def mm():
    import matrix_optimizer_muon_amd
    return matrix_optimizer_muon_amd


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def within(got, want, tol, what=""):
    """Every element of got within tol of want (fp64), NaN and inf in the same places."""
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    ok = (got - want).abs() <= tol + 1e-300
    ok |= torch.isnan(want) | (got == want)
    bad = (~ok).sum().item()
    worst = ((got - want).abs() / (tol + 1e-300))[~torch.isnan(want)].max().item() if want.numel() else 0.0
    assert bad == 0, f"{what}: {bad} of {want.numel()} elements outside, worst {worst:.3g} of the bound"


# ---------------------------------------------------------------------------
# cross entropy
# ---------------------------------------------------------------------------
def ce_reference(h, w, y, g, lse=None):
    """fp64: losses, lse, dh, dw and their bounds."""
    t = h.dtype
    keep = y != IGNORE
    inside = keep & (y >= 0) & (y < w.shape[0])
    V, D = w.shape
    T = h.shape[0]
    hd = torch.where(keep[:, None], h.double(), 0.0)
    wd = w.double()
    z = hd @ wd.T
    dz_logit = (D + 16) * 2.0 ** -23 * (hd.abs() @ wd.abs().T)
    ez = dz_logit.amax(1)
    ref_lse = torch.where(keep, torch.logsumexp(z, 1), 0.0)
    at = torch.where(inside, y, 0)[:, None]
    loss = torch.where(keep, torch.where(inside, ref_lse - z.gather(1, at)[:, 0], math.nan), 0.0)
    soft = (100 + V / 4096) * 2.0 ** -24
    tol = 2 * ez + soft + 2.0 ** -22 * (ref_lse.abs() + torch.nan_to_num(loss).abs())
    out = {"loss": loss, "lse": ref_lse, "tol": tol}
    if g is None:
        return out
    use = inside & (g != 0)
    hd = torch.where(use[:, None], h.double(), 0.0)
    L = (ref_lse if lse is None else lse.double())[:, None]
    p = torch.exp(z - L)
    d = p.clone()
    d.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    gd = torch.where(use, g.double(), 0.0)[:, None]
    dz = torch.where(use[:, None], d * gd, 0.0)
    # p off by the logits' error, exp's, and the fp32 difference with the target
    e_p = p * (dz_logit + 2.0 ** -20 + 2.0 ** -23 * (z.abs() + L.abs())) + 2.0 ** -23 * d.abs()
    u = U[t] if t == torch.bfloat16 else 2.0 ** -22
    e_p = e_p + 2.0 ** -126                                          # exp below the normal range gives 0
    e = torch.where(use[:, None], (u * (d.abs() + e_p) + e_p) * gd.abs() * (1 + 2.0 ** -20), 0.0)
    out["dh"], out["dw"] = dz @ wd, dz.T @ hd
    s_h, s_w = (dz.abs() + e) @ wd.abs(), (dz.abs() + e).T @ hd.abs()
    out["tol_h"] = e @ wd.abs() + (V + 64) * 2.0 ** -23 * s_h + (V + 2) * 2.0 ** -126
    out["tol_w"] = e.T @ hd.abs() + (T + 64) * 2.0 ** -23 * s_w + (T + 2) * 2.0 ** -126
    out["tol_h"] += U[t] * (out["dh"].abs() + out["tol_h"])
    out["tol_w"] += U[t] * (out["dw"].abs() + out["tol_w"])
    return out


def ce_inputs(T, D, V, dtype, seed, ignored=0.2, index=torch.int64):
    g = gen(seed)
    h = randn(g, T, D).to(dtype)
    w = (randn(g, V, D) * (1.5 / math.sqrt(D))).to(dtype)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.where(torch.rand(T, generator=g, device="cuda") < ignored, IGNORE, y).to(index)
    gl = (torch.rand(T, generator=g, device="cuda") + 0.5) / T
    return h, w, y, gl


def check_ce(h, w, y, gl, what=""):
    m = mm()
    ref = ce_reference(h, w, y.long(), gl)
    losses, lse = m.linear_cross_entropy(h, w, y)
    within(losses, ref["loss"], ref["tol"], what + " loss")
    within(lse, ref["lse"], ref["tol"], what + " lse")
    ref = ce_reference(h, w, y.long(), gl, lse)
    dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, gl)
    assert dh.dtype == h.dtype and dw.dtype == w.dtype
    within(dh, ref["dh"], ref["tol_h"], what + " dh")
    within(dw, ref["dw"], ref["tol_w"], what + " dw")
    return losses, lse, dh, dw


CE_SIZES = [(1, 1, 1), (1, 64, 2), (3, 7, 5), (2, 64, 257), (17, 100, 255), (33, 65, 300), (64, 128, 1000),
            (255, 64, 256), (256, 192, 511), (257, 256, 513), (300, 320, 2049), (600, 72, 700)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,D,V", CE_SIZES)
def test_ce_sizes(T, D, V, dtype):
    h, w, y, gl = ce_inputs(T, D, V, dtype, 1000 + T, ignored=0.0 if T < 4 else 0.2)
    check_ce(h, w, y, gl, f"{T}x{D}x{V}")


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_ce_masks(index):
    m = mm()
    h, w, y, gl = ce_inputs(300, 128, 700, torch.bfloat16, 7, index=index)
    # every row ignored
    none = torch.full_like(y, IGNORE)
    losses, lse = m.linear_cross_entropy(h, w, none)
    dh, dw = m.linear_cross_entropy_backward(h, w, none, lse, gl)
    for t in (losses, lse, dh, dw):
        assert not t.any()
    # one row left
    one = none.clone()
    one[137] = 5
    check_ce(h, w, one, gl, "one row")
    # targets outside the vocabulary: loss NaN, no gradient
    out = y.clone()
    out[3], out[4], out[299] = 700, -7, 2 ** 31 - 1
    check_ce(h, w, out, gl, "outside")
    # weights of zero leave a token out, negative ones count
    g2 = gl.clone()
    g2[::3] = 0
    g2[1::3] *= -1
    check_ce(h, w, y, g2, "weights")
    # another ignore_index
    y2 = torch.where(y == IGNORE, 9, torch.where(y == 9, 10, y))
    a = m.linear_cross_entropy(h, w, y2, ignore_index=9)
    y3 = torch.where(y == 9, 10, y)
    b = m.linear_cross_entropy(h, w, y3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_ce_ignored_rows_may_hold_anything():
    m = mm()
    h, w, y, gl = ce_inputs(200, 96, 400, torch.bfloat16, 11)
    clean = [t.clone() for t in check_ce(h, w, y, gl)]
    dirty = h.clone()
    rows = torch.nonzero(y == IGNORE)[:, 0]
    dirty[rows[0::3]] = math.nan
    dirty[rows[1::3]] = math.inf
    dirty[rows[2::3]] = torch.finfo(torch.bfloat16).min
    losses, lse = m.linear_cross_entropy(dirty, w, y)
    gl2 = gl.clone()
    gl2[rows] = math.nan
    dh, dw = m.linear_cross_entropy_backward(dirty, w, y, lse, gl2)
    for a, b in zip(clean, (losses, lse, dh, dw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_ce_nan_stays_in_its_token(dtype):
    m = mm()
    h, w, y, gl = ce_inputs(64, 64, 300, dtype, 12, ignored=0.0)
    ref, _ = m.linear_cross_entropy(h, w, y)
    h[5, 3] = math.nan
    losses, lse = m.linear_cross_entropy(h, w, y)
    assert torch.isnan(losses[5]) and torch.isnan(lse[5])
    keep = torch.arange(64, device="cuda") != 5
    assert torch.equal(losses[keep], ref[keep])


def test_ce_extreme_logits():
    """Logits of ±1000: the largest is subtracted before exp; probabilities of 0 and 1."""
    g = gen(13)
    h = randn(g, 40, 64) * 30
    w = randn(g, 500, 64) * 5
    y = torch.randint(0, 500, (40,), generator=g, device="cuda")
    for t in (torch.bfloat16, torch.float32):
        hh, ww = h.to(t), w.to(t)
        z = hh.double() @ ww.double().T
        y[::2] = z.argmax(1)[::2]
        check_ce(hh, ww, y, torch.full((40,), 1 / 40, device="cuda"), str(t))


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 2.0 ** 100])
def test_ce_gradient_weights_of_any_magnitude(scale):
    h, w, y, gl = ce_inputs(100, 64, 300, torch.float32, 14)
    check_ce(h, w, y, gl * scale, f"{scale}")


def test_ce_gradient_weights_that_are_not_finite():
    """An infinite or NaN weight reaches its own token's gradient and the vocabulary
    rows (all of them: every row takes part in every token), no other token's."""
    m = mm()
    h, w, y, gl = ce_inputs(40, 64, 300, torch.bfloat16, 31, ignored=0.0)
    _, lse = m.linear_cross_entropy(h, w, y)
    for bad in (math.inf, -math.inf, math.nan):
        g = gl.clone()
        g[7] = bad
        dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, g)
        ref = ce_reference(h, w, y, torch.where(g.isfinite(), g, 0.0), lse)
        keep = torch.arange(40, device="cuda") != 7
        within(dh[keep], ref["dh"][keep], ref["tol_h"][keep], f"dh beside {bad}")
        assert not dh[7].isfinite().any() and not dw.isfinite().any()
        only = torch.full_like(gl, bad)
        dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, only)
        assert not dh.isfinite().any() and not dw.isfinite().any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_ce_strides_and_alignment(dtype):
    """Strided rows, rows off the 16-byte grid, and a view whose last row ends the
    allocation: the same bits as dense copies."""
    m = mm()
    for T, D, V, pad, off in ((70, 64, 300, 64, 0), (70, 64, 300, 8, 8), (70, 64, 300, 3, 1), (70, 256, 300, 256, 256),
                              (70, 50, 300, 13, 2)):
        g = gen(T + pad)
        hb, wb = randn(g, T * (D + pad)).to(dtype), (randn(g, V * (D + pad)) * 0.1).to(dtype)
        # the view starts `off` elements in, so that its last row ends the buffer
        # (off + D ≤ D + pad) or leaves pad − off behind it
        h = hb.view(T, D + pad)[:, off:off + D]
        w = wb.view(V, D + pad)[:, pad:pad + D]
        y = torch.randint(0, V, (T,), generator=g, device="cuda")
        gl = torch.full((T,), 1 / T, device="cuda")
        a = m.linear_cross_entropy(h, w, y)
        b = m.linear_cross_entropy(h.contiguous(), w.contiguous(), y)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        ga = m.linear_cross_entropy_backward(h, w, y, a[1], gl)
        gb = m.linear_cross_entropy_backward(h.contiguous(), w.contiguous(), y, b[1], gl)
        assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])
        check_ce(h, w, y, gl, "strided")


def test_ce_batched_shapes_outputs_and_skips():
    m = mm()
    h, w, y, gl = ce_inputs(96, 64, 300, torch.bfloat16, 15)
    ref = m.linear_cross_entropy(h, w, y)
    got = m.linear_cross_entropy(h.view(4, 24, 64), w, y.view(4, 24))
    assert got[0].shape == (4, 24) and torch.equal(got[0].view(-1), ref[0])
    dh, dw = m.linear_cross_entropy_backward(h, w, y, ref[1], gl)
    packed = torch.full((96 * 64 + 300 * 64 + 7,), 3.0, dtype=torch.bfloat16, device="cuda")
    vh, vw = packed[:96 * 64].view(4, 24, 64), packed[96 * 64 + 3:96 * 64 + 3 + 300 * 64].view(300, 64)   # unaligned
    oh, ow = m.linear_cross_entropy_backward(h.view(4, 24, 64), w, y.view(4, 24), ref[1].view(4, 24), gl.view(4, 24),
                                             grad_h=vh, grad_w=vw)
    assert oh is vh and ow is vw and torch.equal(vh.reshape(-1), dh.view(-1)) and torch.equal(vw, dw)
    assert (packed[96 * 64:96 * 64 + 3] == 3).all() and (packed[-4:] == 3).all()
    only_h = m.linear_cross_entropy_backward(h, w, y, ref[1], gl, need_w=False)
    only_w = m.linear_cross_entropy_backward(h, w, y, ref[1], gl, need_h=False)
    assert only_h[1] is None and torch.equal(only_h[0], dh)
    assert only_w[0] is None and torch.equal(only_w[1], dw)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ey, ef = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    assert m.linear_cross_entropy(e, w, ey)[0].shape == (0,)
    eh, ew = m.linear_cross_entropy_backward(e, w, ey, ef, ef)
    assert eh.shape == (0, 64) and ew.shape == (300, 64) and not ew.any()


def test_ce_many_pieces():
    """Tokens × vocabulary above the piece budget: several pieces, the hidden-state
    gradient added up over them, split K for the others."""
    h, w, y, gl = ce_inputs(9000, 64, 33000, torch.bfloat16, 16)
    m = mm()
    losses, lse = m.linear_cross_entropy(h, w, y)
    dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, gl)
    for part in (slice(0, 300), slice(8700, 9000)):
        ref = ce_reference(h[part], w, y[part], gl[part], lse[part])
        within(losses[part], ref["loss"], ref["tol"], "loss")
        within(dh[part], ref["dh"], ref["tol_h"], "dh")
    # dw in fp64 over all tokens, some vocabulary rows
    use = y != IGNORE
    rows = torch.cat([torch.arange(0, 300), torch.arange(32700, 33000)]).cuda()
    hd = torch.where(use[:, None], h.double(), 0.0)
    p = torch.exp(hd @ w[rows].double().T - lse.double()[:, None])
    d = p - (y[:, None] == rows[None]).double()
    d = torch.where(use[:, None], d * gl.double()[:, None], 0.0)
    tol = 2.0 ** -7 * (d.abs().T @ hd.abs())
    within(dw[rows], d.T @ hd, tol + 2.0 ** -8 * (d.T @ hd).abs(), "dw")


@pytest.mark.parametrize("T,D,V,dtype", [(2001, 800, 6500, torch.bfloat16), (1999, 780, 6501, torch.bfloat16),
                                         (2049, 1024, 6400, torch.bfloat16), (2001, 136, 6500, torch.float32)])
def test_ce_large_tiles(T, D, V, dtype):
    """Enough work for the 256 × 256 tiles in the logits and in both products."""
    h, w, y, gl = ce_inputs(T, D, V, dtype, 60)
    check_ce(h, w, y, gl, f"{T}x{D}x{V}")


@pytest.mark.parametrize("T", [1, 15, 16, 17, 32, 33, 49, 64, 65])
@pytest.mark.parametrize("D,V,shift", [(32, 64, 0), (264, 1000, 0), (333, 65, 0), (2056, 130, 0), (320, 700, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ce_few_tokens(T, D, V, shift, dtype):
    """Widths and vocabularies around the fragments' sizes, rows off the 16-byte grid."""
    h, w, y, gl = ce_inputs(T, D + shift, V, dtype, 100 + T)
    if T > 1:
        y[T // 2] = V + 3                                        # no target: NaN loss, lse as ever
    check_ce(h[:, shift:], w[:, shift:], y, gl, f"{T} tokens")


@pytest.mark.parametrize("kept", [0, 1, 130, 256, 700, 2099])
@pytest.mark.parametrize("D,V,dtype", [(200, 5000, torch.bfloat16), (520, 9000, torch.bfloat16), (136, 2500, torch.float32)])
def test_ce_few_of_many_tokens(D, V, dtype, kept):
    """Tiles and K splits are planned for every token; those that take part share them."""
    T = 2100
    h, w, y, gl = ce_inputs(T, D, V, dtype, 23, ignored=0.0)
    out = torch.randperm(T, generator=gen(24), device="cuda")[kept:]
    y[out] = IGNORE
    check_ce(h, w, y, gl, f"{kept} of {T}")


def test_ce_gradient_against_differences():
    """Directional derivatives of the fp64 loss: (L(+δ) − L(−δ))/2δ against ⟨grad, direction⟩ (fp32 gradients)."""
    m = mm()
    h, w, y, _ = ce_inputs(50, 40, 130, torch.float32, 17)
    n = (y != IGNORE).sum()
    gl = torch.full((50,), 1.0, device="cuda") / n
    _, lse = m.linear_cross_entropy(h, w, y)
    dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, gl)

    def loss(hd, wd):
        z = hd @ wd.T
        l = torch.logsumexp(z, 1) - z.gather(1, torch.where(y == IGNORE, 0, y)[:, None])[:, 0]
        return torch.where(y == IGNORE, 0.0, l).sum() / n

    g = gen(18)
    for grad, which in ((dh, 0), (dw, 1)):
        v = randn(g, *grad.shape).double()
        step = 1e-5
        pts = [[h.double(), w.double()], [h.double(), w.double()]]
        pts[0][which] = pts[0][which] + step * v
        pts[1][which] = pts[1][which] - step * v
        diff = (loss(*pts[0]) - loss(*pts[1])) / (2 * step)
        # the difference's own error is O(step²·‖v‖³): under 1e-6 of the scale here
        assert abs((grad.double() * v).sum() - diff) <= 1e-5 * (grad.double() * v).abs().sum()


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (5, 10, 7), (64, 100, 64), (300, 50, 264), (1000, 3000, 513)])
def test_embedding_lookup(T, V, D, dtype):
    m = mm()
    g = gen(T)
    table = randn(g, V, D + 8).to(dtype)
    ids = torch.randint(-2, V + 2, (T,), generator=g, device="cuda")
    for tab in (table[:, :D].contiguous(), table[:, 8:8 + D], table[:, 3:3 + D]):
        for idx in (ids, ids.int()):
            got = m.embedding(idx, tab, scale=1.7)
            inside = (ids >= 0) & (ids < V)
            want = torch.where(inside[:, None], tab[ids.clamp(0, V - 1)].float() * 1.7, 0.0).to(dtype)
            assert torch.equal(got, want)
    assert m.embedding(ids[:0], table).shape == (0, D + 8)
    assert torch.equal(m.embedding(ids.view(1, -1, 1).clamp(0, V - 1), table), table[ids.clamp(0, V - 1)].view(1, -1, 1, D + 8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,ld,shift", [(12, 12, 0), (684, 684, 0), (4, 20, 4), (20, 24, 2), (6, 8, 2), (2, 2, 0), (8, 9, 0), (9, 16, 0), (16, 24, 4)])
def test_embedding_lookup_alignments(D, ld, shift, dtype):
    """Rows that allow 8, 4, 2 or 1 elements at a time, by their width, stride and start."""
    m = mm()
    g = gen(D + ld)
    flat = randn(g, 500 * ld + shift).to(dtype)
    table = flat[shift:].view(500, ld)[:, :D]
    ids = torch.randint(-1, 501, (3000,), generator=g, device="cuda")
    want = torch.where(((ids >= 0) & (ids < 500))[:, None], table[ids.clamp(0, 499)].float() * 0.75, 0.0).to(dtype)
    assert torch.equal(m.embedding(ids, table, scale=0.75), want)
    room = torch.full((3000 * D + 8,), 5.0, device="cuda").to(dtype)      # an output off the grid, its surroundings kept
    out = room[shift:shift + 3000 * D].view(3000, D)
    assert torch.equal(m.embedding(ids, table, scale=0.75, out=out), want)
    assert (room[:shift] == 5).all() and (room[shift + 3000 * D:] == 5).all()


def embed_reference(ids, grad, V, scale, pad, out):
    use = (ids >= 0) & (ids < V)
    if pad is not None:
        use &= ids != pad
    at = torch.where(use, ids.long(), V)
    gd = torch.where(use[:, None], grad.double(), 0.0)
    want = torch.zeros(V + 1, grad.shape[1], dtype=torch.float64, device="cuda").index_add_(0, at, gd)[:V]
    mag = torch.zeros(V + 1, grad.shape[1], dtype=torch.float64, device="cuda").index_add_(0, at, gd.abs())[:V]
    n = torch.bincount(at, minlength=V + 1)[:V, None]
    s = torch.tensor(scale, dtype=torch.float32).double().item()
    tol = abs(s) * mag * (n + 2) * 2.0 ** -24
    return want * s, tol + U[out] * (abs(s) * want.abs() + tol)


@pytest.mark.parametrize("gdt,odt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                     (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (31, 7, 5), (32, 1, 8), (33, 40, 64), (1500, 300, 100), (5000, 70000, 16)])
def test_embedding_gradient(T, V, D, gdt, odt):
    m = mm()
    g = gen(T + V)
    ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    grad = randn(g, T, D).to(gdt)
    for pad in (None, 0, V + 5):
        want, tol = embed_reference(ids, grad, V, 0.3, pad, odt)
        got = m.embedding_backward(ids, grad, V, scale=0.3, padding_id=pad, out_dtype=odt)
        assert got.dtype == odt
        within(got, want, tol, f"pad {pad}")
        assert torch.equal(m.embedding_backward(ids.int(), grad, V, scale=0.3, padding_id=pad, out_dtype=odt), got)


@pytest.mark.parametrize("T", [63, 64, 1023, 1024, 1025, 2079, 33000, 70001])
def test_embedding_gradient_of_one_frequent_id(T):
    """The same id everywhere (and almost everywhere): the sums of every level."""
    m = mm()
    g = gen(T)
    D = 24
    grad = randn(g, T, D)
    ids = torch.full((T,), 3, device="cuda")
    want, tol = embed_reference(ids, grad, 5, 1.0, None, torch.float32)
    within(m.embedding_backward(ids, grad, 5), want, tol, "all")
    ids[::7] = 1
    ids[5::1000] = 4
    want, tol = embed_reference(ids, grad, 5, 1.0, None, torch.float32)
    within(m.embedding_backward(ids, grad, 5), want, tol, "most")


@pytest.mark.parametrize("T,V", [(1024, 9), (1025, 9), (4097, 300), (8192, 1000), (8193, 1000), (16385, 40000), (65536, 2000),
                                 (65537, 2000), (9000, 524285), (9000, 524286), (9000, 524287), (9000, 600000)])
def test_embedding_gradient_sorts(T, V):
    """Token counts and table sizes at the borders of the sorts' variants; ids at both ends of the table and outside."""
    m = mm()
    g = gen(T + V)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    ids[::5] = torch.randint(V - 2, V + 1, ids[::5].shape, generator=g, device="cuda")
    ids[1::7] = torch.randint(-1, 2, ids[1::7].shape, generator=g, device="cuda")
    grad = randn(g, T, 8)
    want, tol = embed_reference(ids, grad, V, 1.0, None, torch.float32)
    within(m.embedding_backward(ids, grad, V), want, tol)


def test_embedding_gradient_accumulates_and_leaves_other_rows():
    m = mm()
    g = gen(3)
    T, V, D = 200, 1000, 72
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    for odt in (torch.bfloat16, torch.float32):
        grad = randn(g, T, D).to(torch.bfloat16)
        held = randn(g, V, D).to(odt)
        held[17] = math.nan
        ids = torch.where(ids == 17, 18, ids)
        out = held.clone()
        assert m.embedding_backward(ids, grad, V, scale=2.0, out=out, accumulate=True) is out
        seen = torch.zeros(V, dtype=torch.bool, device="cuda")
        seen[ids] = True
        assert torch.equal(out[~seen].view(torch.uint8), held[~seen].view(torch.uint8))
        want, _ = embed_reference(ids, grad, V, 2.0, None, odt)
        _, tol = embed_reference(ids, grad, V, 2.0, None, torch.float32)
        total = (held.double() + want)[seen]
        within(out[seen], total, tol[seen] + (U[odt] + 2.0 ** -24) * (total.abs() + tol[seen]), "sum")
        # overwritten, a stale NaN does not survive
        assert not m.embedding_backward(ids, grad, V, out=held.clone()).isnan().any()


def test_embedding_gradient_strides_nan_and_order():
    m = mm()
    g = gen(4)
    T, V, D = 400, 60, 40
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    big = randn(g, T, D + 11)
    for off in (0, 8, 3, 11):
        v = big[:, off:off + D]
        assert torch.equal(m.embedding_backward(ids, v, V), m.embedding_backward(ids, v.contiguous(), V))
    grad = big[:, :D].contiguous()
    grad[7] = math.nan
    got = m.embedding_backward(ids, grad, V)
    assert got[ids[7]].isnan().all()
    keep = torch.arange(V, device="cuda") != ids[7]
    assert not got[keep].isnan().any()
    assert not m.embedding_backward(ids, grad, V, padding_id=int(ids[7])).isnan().any()
    a = m.embedding_backward(ids, grad[:, :8].contiguous(), V)
    for _ in range(3):
        assert torch.equal(torch.nan_to_num(m.embedding_backward(ids, grad[:, :8].contiguous(), V)), torch.nan_to_num(a))
    assert m.embedding_backward(ids[:0], grad[:0], 9).eq(0).all()


# ---------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------
def p2(e):
    """2^e in fp64, exactly (from its bits; a library power need not be exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def ckpt_reference(x):
    """q, exps from the definition, in fp64."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    xd = torch.nn.functional.pad(x.double(), (0, blocks * 32 - cols)).view(rows, blocks, 32)
    finite = torch.isfinite(xd).all(2)
    most = torch.where(finite, xd.abs().amax(2), 0.0)
    b = torch.where(most >= 2.0 ** -126, torch.frexp(most)[1] + 126, 0)
    up = (most * p2(133 - b) >= 127.5) & (b > 0) & (b < 254)
    b = b + up
    q = torch.clamp(torch.round(xd * p2(133 - b)[..., None]), -127, 127)
    q = torch.where((b > 0)[..., None] & finite[..., None], q, 0.0)
    b = torch.where(finite, b, 255)
    return q.view(rows, blocks * 32)[:, :cols].to(torch.int8), b.to(torch.uint8)


def ckpt_values(q, b):
    v = q.double() * p2(b.int() - 133).repeat_interleave(32, 1)[:, :q.shape[1]]
    return torch.where(b.repeat_interleave(32, 1)[:, :q.shape[1]] == 255, math.nan, v)


def check_codec(x):
    m = mm()
    q, b = m.checkpoint_quantize(x)
    rq, rb = ckpt_reference(x)
    assert torch.equal(b, rb)
    ok = (rb != 255).repeat_interleave(32, 1)[:, :x.shape[1]]
    assert torch.equal(q[ok], rq[ok])
    for t in (torch.bfloat16, torch.float32):
        y = m.checkpoint_dequantize(q, b, dtype=t)
        v = ckpt_values(q, b)
        assert torch.equal(y.double()[ok], v[ok]) and y[~ok].isnan().all()
    # within half a step of the input
    half = p2(b.int() - 134).repeat_interleave(32, 1)[:, :x.shape[1]]
    fine = ok & (b != 0).repeat_interleave(32, 1)[:, :x.shape[1]] & (b != 254).repeat_interleave(32, 1)[:, :x.shape[1]]
    assert ((v - x.double()).abs() <= half)[fine].all()
    return q, b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 31), (5, 32), (7, 33), (64, 64), (100, 1000), (33, 4099)])
def test_checkpoint_codec(T, K, dtype):
    g = gen(T + K)
    x = (randn(g, T, K) * torch.exp(4 * randn(g, T, 1))).to(dtype)
    q, b = check_codec(x)
    wide = torch.cat([x, x, x], 1)
    for off in (0, K, 8):
        v = wide[:, off:off + K]
        m = mm()
        a = m.checkpoint_quantize(v)
        c = m.checkpoint_quantize(v.contiguous())
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    assert mm().checkpoint_quantize(x[:0])[0].shape == (0, K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_checkpoint_special_values(dtype):
    big = torch.finfo(dtype).max
    tiny = 2.0 ** -126
    rows = [[0.0] * 32, [1.0] + [0.0] * 31, [127.4 / 64] + [1.0] * 31, [127.6 / 64] + [1.0] * 31, [-127.6 / 64] * 32,
            [big] * 32, [-big] + [1.0] * 31, [tiny] * 32, [tiny / 2] * 32, [tiny * 1.999] + [0.0] * 31,
            [math.nan] + [1.0] * 31, [1.0] * 31 + [math.inf], [-math.inf] * 32, [0.5, 1.5, 2.5, -0.5, -2.5] + [64.0] * 27,
            [2.0 ** -120] * 32, [2.0 ** 120, 1.0] + [0.0] * 30]
    x = torch.tensor(rows, device="cuda", dtype=torch.float64).to(dtype)
    check_codec(x)
    check_codec(torch.cat([x, x.flip(0)[:, :5]], 1))


def wgrad_reference(grad, q, b, out, offsets=None):
    xd, gd = ckpt_values(q, b), grad.double()
    groups = [(0, q.shape[0])] if offsets is None else list(zip(offsets, offsets[1:]))
    want, tol = [], []
    for s, e in groups:
        w = gd[s:e].T @ xd[s:e]
        t = (max(e - s, 0) + 64) * 2.0 ** -23 * (gd[s:e].abs().T @ xd[s:e].abs())
        want.append(w)
        tol.append(t + U[out] * (w.abs() + t))
    return (want[0], tol[0]) if offsets is None else (torch.stack(want), torch.stack(tol))


@pytest.mark.parametrize("gdt,odt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                     (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (2, 64, 32), (31, 65, 33), (300, 256, 256), (257, 300, 520), (5000, 40, 72)])
def test_wgrad(T, N, K, gdt, odt):
    m = mm()
    g = gen(T + N + K)
    x, grad = randn(g, T, K), randn(g, T, N).to(gdt)
    q, b = m.checkpoint_quantize(x)
    want, tol = wgrad_reference(grad, q, b, odt)
    got = m.checkpoint_wgrad(grad, q, b, out_dtype=odt)
    assert got.dtype == odt
    within(got, want, tol)
    # strided and shifted rows: the same bits
    wide = torch.cat([grad, torch.ones_like(grad[:, :1]).expand(T, 5), grad], 1)[:, N + 5:]
    assert torch.equal(m.checkpoint_wgrad(wide, q, b, out_dtype=odt), got)


@pytest.mark.parametrize("offsets", [[0, 0, 0, 300], [0, 100, 100, 101, 290], [5, 40, 72, 72, 250], [0, 300], [300, 300, 300]])
def test_wgrad_groups(offsets):
    m = mm()
    g = gen(sum(offsets))
    T, N, K = 300, 136, 264
    x, grad = randn(g, T, K), randn(g, T, N).to(torch.bfloat16)
    # rows outside every group may hold anything
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    inside[offsets[0]:offsets[-1]] = True
    grad[~inside] = math.nan
    x[~inside] = math.inf
    q, b = m.checkpoint_quantize(x)
    want, tol = wgrad_reference(grad, q, b, torch.float32, offsets)
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got = m.checkpoint_wgrad(grad, q, b, offsets=at, out_dtype=torch.float32)
    within(got, want, tol)
    assert torch.equal(m.checkpoint_wgrad(grad, q, b, offsets=at, out_dtype=torch.bfloat16), got.to(torch.bfloat16))


@pytest.mark.parametrize("T,N,K,gdt,odt", [(3001, 1500, 1700, torch.bfloat16, torch.float32), (2999, 1501, 1703, torch.bfloat16, torch.bfloat16),
                                           (500, 4000, 4100, torch.bfloat16, torch.bfloat16), (1100, 1500, 1700, torch.float32, torch.float32)])
def test_wgrad_large_tiles(T, N, K, gdt, odt):
    """Enough work for the 256 × 256 tiles, with K splits and without."""
    m = mm()
    g = gen(T + N + K)
    x, grad = randn(g, T, K), randn(g, T, N).to(gdt)
    q, b = m.checkpoint_quantize(x)
    want, tol = wgrad_reference(grad, q, b, odt)
    within(m.checkpoint_wgrad(grad, q, b, out_dtype=odt), want, tol)


def test_wgrad_large_tiles_in_groups():
    """Uneven and empty groups whose rows start and end inside stages; rows outside hold NaN."""
    m = mm()
    g = gen(77)
    T, N, K = 3001, 1496, 1704
    offsets = [3, 700, 700, 701, 1900, 2990]
    x, grad = randn(g, T, K), randn(g, T, N).to(torch.bfloat16)
    for gone in (slice(0, 3), slice(2990, T)):
        grad[gone] = math.nan
        x[gone] = math.inf
    q, b = m.checkpoint_quantize(x)
    want, tol = wgrad_reference(grad, q, b, torch.float32, offsets)
    at = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    within(m.checkpoint_wgrad(grad, q, b, offsets=at, out_dtype=torch.float32), want, tol)


def test_wgrad_offsets_out_of_range_are_clamped():
    m = mm()
    g = gen(9)
    T, N, K = 100, 64, 64
    grad = randn(g, T, N).to(torch.bfloat16)
    q, b = m.checkpoint_quantize(randn(g, T, K))
    at = torch.tensor([-50, 40, 30, 2 ** 30, 60], dtype=torch.int32, device="cuda")
    got = m.checkpoint_wgrad(grad, q, b, offsets=at, out_dtype=torch.float32)
    want, tol = wgrad_reference(grad, q, b, torch.float32, [0, 40, 40])
    within(got[:2], want, tol)
    want, tol = wgrad_reference(grad, q, b, torch.float32, [30, 100])
    within(got[2:3], want, tol)
    assert not got[3].any()
    assert m.checkpoint_wgrad(grad, q, b, offsets=at[:1]).shape == (0, N, K)
    assert not m.checkpoint_wgrad(grad[:0], q[:0], b[:0]).any()


# ---------------------------------------------------------------------------
# streams, graphs, determinism, refusals
# ---------------------------------------------------------------------------
def one_of_each(seed=21):
    """Every operator once, as closures over fixed inputs."""
    m = mm()
    h, w, y, gl = ce_inputs(300, 128, 1000, torch.bfloat16, seed)
    _, lse = m.linear_cross_entropy(h, w, y)
    g = gen(seed)
    ids = torch.randint(0, 50, (600,), generator=g, device="cuda")
    grad = randn(g, 600, 72).to(torch.bfloat16)
    x = randn(g, 600, 200).to(torch.bfloat16)
    q, b = m.checkpoint_quantize(x)
    at = torch.tensor([0, 10, 300, 600], dtype=torch.int32, device="cuda")
    table = randn(g, 50, 72).to(torch.bfloat16)
    return [lambda **k: m.linear_cross_entropy(h, w, y, **k),
            lambda **k: m.linear_cross_entropy_backward(h, w, y, lse, gl, **k),
            lambda **k: (m.embedding(ids, table, scale=3.0, **k),),
            lambda **k: (m.embedding_backward(ids, grad, 50, **k),),
            lambda **k: m.checkpoint_quantize(x, **k),
            lambda **k: (m.checkpoint_dequantize(q, b, **k),),
            lambda **k: (m.checkpoint_wgrad(grad, q, b, **k),),
            lambda **k: (m.checkpoint_wgrad(grad, q, b, offsets=at, **k),)]


def test_deterministic_and_on_another_stream():
    calls = one_of_each()
    ref = [c() for c in calls]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for c, r in zip(calls, ref):
        for a, b in zip(c(), r):
            assert torch.equal(a, b)
        got = c(stream=st)
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(4)]     # the current stream allocates behind it
        st.synchronize()
        for a, b in zip(got, r):
            assert torch.equal(a, b)
        del junk


def test_two_streams_at_once():
    a, b = one_of_each(31), one_of_each(32)
    ra, rb = [c() for c in a], [c() for c in b]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ga, gb = [], []
    for c1, c2 in zip(a, b):
        ga.append(c1(stream=s1))
        gb.append(c2(stream=s2))
    torch.cuda.synchronize()
    for got, want in ((ga, ra), (gb, rb)):
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_graph_replays():
    """Every operator in one captured graph, replayed with changed inputs and eager
    work in between; each replay equals the eager results."""
    m = mm()
    h, w, y, gl = ce_inputs(300, 128, 1000, torch.bfloat16, 41)
    g = gen(42)
    ids = torch.randint(0, 50, (300,), generator=g, device="cuda")
    x = randn(g, 300, 128).to(torch.bfloat16)

    def run():
        losses, lse = m.linear_cross_entropy(h, w, y)
        dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, gl)
        q, b = m.checkpoint_quantize(x)
        return [losses, lse, dh, dw, m.embedding(ids, w), m.embedding_backward(ids, dh, 50), q, b,
                m.checkpoint_dequantize(q, b), m.checkpoint_wgrad(dh, q, b)]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for k in range(3):
        h.copy_(randn(g, 300, 128).to(torch.bfloat16))
        x.copy_(randn(g, 300, 128).to(torch.bfloat16))
        y[k * 50:(k + 1) * 50] = IGNORE
        ids.copy_(torch.randint(0, 50, (300,), generator=g, device="cuda"))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,D,V,dtype", [(20, 264, 1000, torch.bfloat16), (40, 100, 700, torch.float32),
                                         (2100, 520, 9000, torch.bfloat16), (2100, 136, 2500, torch.float32)])
def test_graph_replays_with_other_tokens_taking_part(T, D, V, dtype):
    """A captured loss and gradient: how many tokens count is read on the device, from
    all of them to none."""
    m = mm()
    h, w, y, gl = ce_inputs(T, D, V, dtype, 51, ignored=0.0)
    all_y = y.clone()

    def run():
        losses, lse = m.linear_cross_entropy(h, w, y)
        return [losses, lse, *m.linear_cross_entropy_backward(h, w, y, lse, gl)]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for kept in (T // 3, 0, T, 1):
        y.copy_(all_y)
        y[kept:] = IGNORE
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b), kept
        assert not held[2][kept:].any() and not held[0][kept:].any()


@pytest.mark.parametrize("phase", ["ce_pack", "ce_logits", "ce_rows", "ce_grads", "embed", "embed_grad", "ckpt_codec", "ckpt_wgrad"])
def test_forced_failures(phase, monkeypatch):
    calls = one_of_each()
    ref = [c() for c in calls]
    torch.cuda.synchronize()
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", phase)
    failed = 0
    for c in calls:
        try:
            c()
        except RuntimeError as e:
            assert phase in str(e)
            failed += 1
    assert failed >= 1
    monkeypatch.delenv("DMUON_TEST_FAIL_AT")
    for c, r in zip(calls, ref):
        assert all(torch.equal(a, b) for a, b in zip(c(), r))


def test_debug_sync_and_phase_timing(monkeypatch):
    m = mm()
    calls = one_of_each()
    ref = [c() for c in calls]
    monkeypatch.setenv("DMUON_DEBUG_SYNC", "1")
    m.phase_timing(True)
    m.phase_timing_read()
    for c, r in zip(calls, ref):
        assert all(torch.equal(a, b) for a, b in zip(c(), r))
    m.phase_timing(False)
    seen = m.phase_timing_read()
    for p in ("ce_pack", "ce_logits", "ce_rows", "ce_grads", "embed", "embed_grad", "ckpt_codec", "ckpt_wgrad"):
        assert seen[p][1] >= 1 and seen[p][0] > 0


def test_python_refusals():
    m = mm()
    h = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(10, 16, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(8, dtype=torch.int64, device="cuda")
    f = torch.zeros(8, device="cuda")
    q, b = m.checkpoint_quantize(h)
    bad = [lambda: m.linear_cross_entropy(h.half(), w.half(), y), lambda: m.linear_cross_entropy(h, w.float(), y),
           lambda: m.linear_cross_entropy(h, w[:, :8], y), lambda: m.linear_cross_entropy(h, w, y.float()),
           lambda: m.linear_cross_entropy(h, w, y[:7]), lambda: m.linear_cross_entropy(h.t(), w, y),
           lambda: m.linear_cross_entropy(h[:1].expand(8, 16), w, y), lambda: m.linear_cross_entropy(h, w[None], y),
           lambda: m.linear_cross_entropy(h, w[:0], y), lambda: m.linear_cross_entropy(h, w, y.cpu()),
           lambda: m.linear_cross_entropy(h, w, y, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: m.linear_cross_entropy_backward(h, w, y, f[:7], f), lambda: m.linear_cross_entropy_backward(h, w, y, f, f.double()),
           lambda: m.linear_cross_entropy_backward(h, w, y, f, f, grad_h=h), lambda: m.linear_cross_entropy_backward(h, w, y, f, f, grad_w=w.float()),
           lambda: m.linear_cross_entropy_backward(h, w, y, f, f, grad_h=torch.empty_like(h), need_h=False),
           lambda: m.embedding(y.float(), w), lambda: m.embedding(y, w[None]), lambda: m.embedding(y, w.half()),
           lambda: m.embedding(y, w, out=h.float()), lambda: m.embedding(y[::2], w), lambda: m.embedding(y, w, scale=math.nan),
           lambda: m.embedding_backward(y, h[:7], 10), lambda: m.embedding_backward(y, h, -1),
           lambda: m.embedding_backward(y, h, 10, accumulate=True), lambda: m.embedding_backward(y, h, 10, out_dtype=torch.float16),
           lambda: m.embedding_backward(y, h, 10, out=w, out_dtype=torch.float32), lambda: m.embedding_backward(y, h, 10, padding_id=-1),
           lambda: m.embedding_backward(y, h, 9, out=w), lambda: m.embedding_backward(y, h[0].expand(8, 16), 10),
           lambda: m.checkpoint_quantize(h.half()), lambda: m.checkpoint_quantize(h[0]),
           lambda: m.checkpoint_dequantize(q, b[:, :0]), lambda: m.checkpoint_dequantize(q.float(), b),
           lambda: m.checkpoint_dequantize(q, b, dtype=torch.float16), lambda: m.checkpoint_wgrad(h[:7], q, b),
           lambda: m.checkpoint_wgrad(h, q, b, offsets=y), lambda: m.checkpoint_wgrad(h, q, b, offsets=y.int()[:0]),
           lambda: m.checkpoint_wgrad(h, q, b, out=h)]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", k)


# ---------------------------------------------------------------------------
# together: one training step's gradients, then the two optimizer routes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("tied", [False, True])
def test_a_training_step(tied):
    """Embedding → one linear layer whose input is kept in 8 bits → cross entropy;
    the table's (and head's) gradient goes to the AdamW step, the layer's to the
    Muon step, and both steps equal the oracle's on these gradients."""
    import numpy as np
    import oracle
    from matrix_optimizer_muon_amd.workloads import HYPER
    m = mm()
    g = gen(50)
    T, V, D = 300, 500, 128
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.where(torch.rand(T, generator=g, device="cuda") < 0.1, IGNORE, ids.roll(-1))
    bf = torch.bfloat16
    masters = {"table": randn(g, V, D) * 0.05, "lin": randn(g, D, D) * 0.1, "head": randn(g, V, D) * 0.1}
    p = {k: v.to(bf) for k, v in masters.items()}
    head = p["table"] if tied else p["head"]
    scale = math.sqrt(D)
    # forward
    x = m.embedding(ids, p["table"], scale=scale)
    q, b = m.checkpoint_quantize(x)
    h = (x.float() @ p["lin"].float().T).to(bf)
    losses, lse = m.linear_cross_entropy(h, head, y)
    n = (y != IGNORE).sum()
    gl = torch.ones(T, device="cuda") / n
    # backward
    dh, dhead = m.linear_cross_entropy_backward(h, head, y, lse, gl)
    dlin = m.checkpoint_wgrad(dh, q, b)
    dx = (dh.float() @ p["lin"].float()).to(bf)
    if tied:
        before = dhead.clone()
        dtable = m.embedding_backward(ids, dx, V, scale=scale, out=dhead, accumulate=True)
    else:
        dtable = m.embedding_backward(ids, dx, V, scale=scale)
    # against fp64, each operator on its own inputs
    ref = ce_reference(h, head, y, gl, lse)
    within(losses, ref["loss"], ref["tol"], "loss")
    within(dh, ref["dh"], ref["tol_h"], "dh")
    within(before if tied else dhead, ref["dw"], ref["tol_w"], "dhead")
    want, tol = wgrad_reference(dh, q, b, bf)
    within(dlin, want, tol, "dlin")
    want, tol = embed_reference(ids, dx, V, scale, None, torch.float32)
    if tied:
        want = want + before.double()
    within(dtable, want, tol + (U[bf] + 2.0 ** -24) * (want.abs() + tol), "dtable")
    # the steps
    mom = torch.zeros_like(masters["lin"])
    W = masters["lin"].clone()
    out = torch.empty_like(W)
    m.muon_step([dlin], [mom], [W], ns_outs=[out], param_outs=[p["lin"]])
    B, O, _ = oracle.muon_step(dlin.float().cpu().numpy(), np.zeros((D, D), np.float32), masters["lin"].cpu().numpy(), lr=HYPER["lr"],
                               mu=HYPER["mu"], wd=HYPER["wd"], eps=HYPER["eps"], a=HYPER["a"], b=HYPER["b"], c=HYPER["c"],
                               steps=HYPER["steps"])
    assert np.linalg.norm(out.cpu().numpy() - O) <= 2e-2 * np.linalg.norm(O)
    assert torch.equal(p["lin"], W.to(bf))
    P, G = [masters["table"]], [dtable]
    if not tied:
        P, G = P + [masters["head"]], G + [dhead]
    M, S = [torch.zeros_like(t) for t in P], [torch.zeros_like(t) for t in P]
    old = [t.cpu().numpy().copy() for t in P]
    m.adamw_step(P, G, M, S, step=1)
    hp = {k: float(np.float32(v)) for k, v in dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.01).items()}
    for o, t, gr in zip(old, P, G):
        pr, _, _ = oracle.adamw_step(o, gr.float().cpu().numpy(), np.zeros_like(o), np.zeros_like(o), step=1, **hp)
        assert np.linalg.norm(t.cpu().numpy() - pr) <= 1e-6 * np.linalg.norm(pr)
