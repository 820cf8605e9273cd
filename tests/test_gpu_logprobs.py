"""Log probabilities from logits, entropies, alternatives and their gradient against plain
fp64 implementations (needs an MI355X).

Tolerances are worst-case bounds from the arithmetic.  With x = scale·z, X the row's
largest x, p the probabilities, k1 = Σ p·|x − X| and k2 = Σ p·(x − X)²:

* an exponent (z − m)·(scale·log2 e) is off by 3·2^-24 of itself (the difference or the
  reference, the product, the constant), exp2 by 2^-23 of its result; the reference's own
  rounding, at most 1/2, is common to all terms;
* a thread adds up n ≤ 64 + V/256 terms of one sign and multiplies its sums at most n/8
  times when its largest grows (4·2^-24 each), the others join in ten more steps: the sum S
  is off by soft = (2n + 128)·2^-24 of itself, plus 3·2^-24·k1 of it from the exponents;
* log S, its products and differences: 2^-22 of each term;
* the entropy's sum Σ (x − X)·p has the same n steps, and 3·2^-24·k2 from the exponents;
* a result below 2^-126 may become 0, a rounding to bf16 is off by 2^-8 of the value.
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
    """Every element of got within tol of want (fp64), NaN and inf in the same places."""
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    ok = (got - want).abs() <= tol + 1e-300
    ok |= torch.isnan(want) | (got == want)
    bad = (~ok).sum().item()
    assert bad == 0, f"{what}: {bad} of {want.numel()} elements outside, worst {torch.nan_to_num((got - want).abs() / (tol + 1e-300)).max().item():.3g}"


def reference(z, y, scale=1.0, top=0, ignore=IGNORE):
    """fp64 results and their bounds; rows of -inf alone, ignored rows and targets elsewhere
    as documented."""
    T, V = z.shape
    kept = torch.ones(T, dtype=torch.bool, device=z.device) if y is None else y != ignore
    x = torch.where(kept[:, None], z.double() * scale, 0.0)
    big = x.amax(1, keepdim=True)
    none = big[:, 0] == -math.inf
    d = torch.where(none[:, None], -math.inf, x - big)
    e = torch.exp(d)
    S = e.sum(1)
    dist = torch.where(e > 0, -d, 0.0)
    dist = torch.where(torch.isnan(d), math.nan, dist)
    p = e / S[:, None]
    k1, k2 = (p * dist).sum(1), (p * dist * dist).sum(1)
    logS = torch.log(S)
    n = 64 + V / 256
    e_s = (2 * n + 128) * 2.0 ** -24 + 3 * 2.0 ** -24 * k1 + 2.0 ** -22 * logS.abs()
    lse = torch.where(none, -math.inf, big[:, 0] + logS)
    H = torch.where(none, 0.0, logS + k1)
    log_p = torch.where(none[:, None], -math.inf, d - logS[:, None])
    t_lp = e_s[:, None] + 2.0 ** -22 * (torch.nan_to_num(d, 0.0, 0.0, 0.0).abs() + torch.nan_to_num(log_p, 0.0, 0.0, 0.0).abs())
    out = {"lse": torch.where(kept, lse, 0.0), "t_lse": e_s + 2.0 ** -23 * torch.nan_to_num(lse, 0.0, 0.0, 0.0).abs(),
           "entropy": torch.where(kept, H, 0.0),
           "t_entropy": e_s * (1 + k1) + (2 * n + 128) * 2.0 ** -24 * k1 + 3 * 2.0 ** -24 * k2 + 2.0 ** -22 * (logS.abs() + k1)}
    if y is not None:
        inside = (y >= 0) & (y < V)
        at = torch.where(inside, y, 0).long()[:, None]
        lp = torch.where(inside, log_p.gather(1, at)[:, 0], torch.where(y == -2 ** 31, -lse, math.nan))
        out["logprobs"] = torch.where(kept, lp, 0.0)
        out["t_logprobs"] = torch.where(inside, t_lp.gather(1, at)[:, 0], out["t_lse"])
    if top:
        order = torch.sort(torch.nan_to_num(z.double(), -math.inf, math.inf, -math.inf), dim=1, descending=True, stable=True).indices[:, :top]
        out["ids"] = torch.where(kept[:, None], order, -1)
        out["best"] = torch.where(kept[:, None], log_p.gather(1, order), 0.0)
        out["t_best"] = t_lp.gather(1, order)
    return out


def check(z, y, scale=1.0, top=0, what="", **kw):
    ref = reference(z, y, scale, top)
    r = mm().token_logprobs(z, y, top=top, scale=scale, **kw)
    within(r.lse, ref["lse"], ref["t_lse"], what + " lse")
    within(r.entropy, ref["entropy"], ref["t_entropy"], what + " entropy")
    if y is None:
        assert r.logprobs is None
    else:
        within(r.logprobs, ref["logprobs"], ref["t_logprobs"], what + " logprobs")
    if top:
        assert r.top_ids.dtype == torch.int64
        assert torch.equal(r.top_ids, ref["ids"]), what + " ids"
        within(r.top_logprobs, ref["best"], ref["t_best"], what + " best")
    else:
        assert r.top_ids is None and r.top_logprobs is None
    return r


def grad_reference(z, y, lse, H, g, h, scale=1.0, ignore=IGNORE):
    """fp64 gradient and its bound, from the same lse and entropy."""
    T, V = z.shape
    zero = torch.zeros(T, dtype=torch.float64, device=z.device)
    g, h = zero if g is None else g.double(), zero if h is None else h.double()
    inside = torch.zeros(T, dtype=torch.bool, device=z.device) if y is None else (y >= 0) & (y < V)
    part = torch.ones_like(inside) if y is None else (y != ignore) & (inside | (y == -2 ** 31))
    part = part & ~((g == 0) & (h == 0)) & (lse != -math.inf)
    L, H = lse.double()[:, None], (zero if H is None else H.double())[:, None]
    l = z.double() * scale - L
    p = torch.exp(l)
    far = p < 2.0 ** -200
    l = torch.where(far & ~torch.isnan(l), 0.0, l)
    inner = g[:, None] + h[:, None] * (l + H)
    d = torch.where(far, 0.0, -p * inner)
    hot = torch.zeros_like(d)
    if y is not None:
        hot.scatter_(1, torch.where(inside, y, 0).long()[:, None], torch.where(inside, g, 0.0)[:, None])
    want = torch.where(part[:, None], scale * (d + hot), 0.0)
    mag = g.abs()[:, None] + h.abs()[:, None] * (l.abs() + H.abs())
    tol = scale * (p * mag * (3 * l.abs() + 12) * 2.0 ** -24 + 2.0 ** -22 * (d.abs() + hot.abs()) + 2.0 ** -126 * (2 + mag))
    return want, torch.nan_to_num(tol) + U[z.dtype] * torch.nan_to_num(want).abs() + 2.0 ** -126


def check_grad(z, y, g, h, scale=1.0, what="", **kw):
    r = mm().token_logprobs(z, y, scale=scale)
    want, tol = grad_reference(z, y, r.lse, r.entropy, g, h, scale)
    got = mm().token_logprobs_backward(z, y, r.lse, r.entropy, g, h, scale=scale, **kw)
    assert got.dtype == z.dtype
    within(got, want, tol, what + " gradient")
    return got


def inputs(T, V, dtype, seed, ignored=0.0, index=torch.int64, spread=2.5):
    g = gen(seed)
    z = (randn(g, T, V) * spread).to(dtype)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.where(torch.rand(T, generator=g, device="cuda") < ignored, IGNORE, y).to(index)
    return z, y, randn(g, T) / T, -0.01 * torch.rand(T, generator=g, device="cuda") / T


SIZES = [(1, 1), (1, 2), (3, 5), (6, 63), (7, 100), (5, 255), (4, 256), (3, 257), (9, 1000), (2, 2047), (2, 2048), (5, 2049),
         (3, 4096), (3, 4097), (1, 8192), (3, 20000), (70, 32000), (2100, 300), (2049, 2300), (9, 131072), (2, 131080), (1, 300007)]


@TYPES
@pytest.mark.parametrize("T,V", SIZES)
def test_sizes(T, V, dtype):
    z, y, g, h = inputs(T, V, dtype, 100 + T + V, ignored=0.0 if T < 4 else 0.2)
    for top in sorted({0, 1, min(V, 5), min(V, 64), min(V, 128)}):
        check(z, y, top=top, what=f"{T}x{V} top {top}")
    check_grad(z, y, g, h, what=f"{T}x{V}")


# where the kernels change: a unit, a wave's row with and without alternatives, a
# workgroup's row, and rows enough for waves over longer ones
BORDERS = [(3, 8), (3, 9), (5, 15), (5, 16), (5, 17), (4, 511), (4, 512), (4, 513), (4, 1025), (4, 2056), (3, 4095), (3, 4103), (2, 8192), (2, 8193),
           (2, 12288), (2, 12289), (600, 4100), (512, 12288), (511, 12288), (513, 12289), (1024, 20000), (1023, 20000), (1, 131073), (17, 40007),
           (1024, 4097), (1024, 8191), (1023, 8193)]


@TYPES
@pytest.mark.parametrize("T,V", BORDERS)
def test_borders_between_the_kernels(T, V, dtype):
    z, y, g, h = inputs(T, V, dtype, 900 + T + V, ignored=0.0 if T < 6 else 0.2)
    for top in sorted({0, 3, min(V, 32), min(V, 33), min(V, 128)}):
        check(z, y, 0.9, top=top, what=f"{T}x{V} top {top}")
    check_grad(z, y, g, h, 0.9, what=f"{T}x{V}")


@TYPES
@pytest.mark.parametrize("V", [100, 9000, 40000])
def test_large_logits(V, dtype):
    """Logits whose exponents have no fraction bits left, beside each other and alone."""
    for size in (1e4, 1e8, 1e9, 1e20, 2e38):
        z, y, g, h = inputs(6, V, dtype, 40)
        z = (z.float() * 1e-3 * size).clamp(-size, size).to(dtype)
        z[1] = torch.where(torch.arange(V, device="cuda") % 5 == 0, z[1].abs().max(), z[1])      # equal largest ones
        z[2] = -z[2].abs()
        z[3, ::2] = -math.inf
        y[3] = 1
        check(z, y, top=20, what=f"{size}")
        check_grad(z, y, g, h, what=f"{size}")


@TYPES
@pytest.mark.parametrize("scale", [2.0 ** -20, 0.7, 1.25, 1000.0])
def test_scale(scale, dtype):
    z, y, g, h = inputs(33, 5000, dtype, 7)
    check(z, y, scale, top=9, what="scaled")
    check_grad(z, y, g, h, scale, what="scaled")


@TYPES
def test_targets_none_int32_and_leading_dims(dtype):
    z, y, g, h = inputs(24, 3001, dtype, 8, ignored=0.3)
    check(z, None, top=4)
    check_grad(z, None, None, h)
    a, b = check(z, y, top=4), check(z, y.int(), top=4)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    r = mm().token_logprobs(z.view(4, 6, -1), y.view(4, 6), top=4)
    assert r.logprobs.shape == r.lse.shape == (4, 6) and r.top_ids.shape == (4, 6, 4)
    for s, t in zip(a, r):
        assert torch.equal(s, t.view(s.shape))
    r = mm().token_logprobs(z.view(4, 6, -1), y.view(4, 6))
    d = mm().token_logprobs_backward(z.view(4, 6, -1), y.view(4, 6), r.lse, r.entropy, g.view(4, 6), h.view(4, 6))
    assert torch.equal(d.view(24, -1), check_grad(z, y, g, h))
    # either gradient alone
    check_grad(z, y, g, None)
    check_grad(z, y, None, h)


@TYPES
def test_targets_outside(dtype):
    z, y, g, h = inputs(40, 777, dtype, 9)
    y[::4] = IGNORE
    y[1::8] = -1
    y[2::8] = 777
    y[3::8] = -2 ** 31
    y[5] = 2 ** 40
    r = check(z, y, top=3)
    assert torch.isnan(r.logprobs[1]) and r.logprobs[3] == -r.lse[3]
    d = check_grad(z, y, g, h)
    assert not d[1].any() and not d[5].any() and d[3].any()
    # ignored rows are not read: what they hold is no matter
    z2 = z.clone()
    z2[::4] = math.nan
    for s, t in zip(r, mm().token_logprobs(z2, y, top=3)):
        assert torch.equal(torch.nan_to_num(s, 7.0), torch.nan_to_num(t, 7.0))
    assert torch.equal(check_grad(z2, y, g, h), d)
    # rows of zero gradients neither
    g[7], h[7] = 0.0, 0.0
    z2[7] = math.nan
    r = mm().token_logprobs(z, y)
    d = mm().token_logprobs_backward(z2, y, r.lse, r.entropy, g, h)
    assert not d[7].any() and not torch.isnan(d).any()
    every = torch.full_like(y, IGNORE)
    r = check(z, every, top=3)
    assert not r.lse.any() and (r.top_ids == -1).all()
    assert not check_grad(z, every, g, h).any()


def patterns(V, dtype, seed):
    """Rows at which a selection can go wrong."""
    g = gen(seed)
    at = torch.arange(V, device="cuda")
    base = randn(g, V) * 2.5
    rows = [torch.zeros(V, device="cuda"),                                  # all equal
            torch.full((V,), -math.inf, device="cuda"),
            torch.where(at % 997 == 5, base, -math.inf),                    # most words masked out
            torch.where(at == V - 1, 1.0, -math.inf),
            (base * 2).round() / 2,                                         # many equal values
            at / V * 10, -at / V * 10,                                      # in order
            torch.where(at // 8 % 256 < 100, base + 40, base),              # all large ones in 100 threads
            torch.where(at // 8 % 256 < 3, 20.0 + at % 7, base),            # ... equal ones in 3
            torch.full((V,), torch.finfo(dtype).min, device="cuda"),        # the lowest value
            torch.where(at % 2 == 0, torch.finfo(dtype).min, base),
            torch.where(at == V // 2, torch.finfo(dtype).max, base),
            torch.where(at % 3 == 0, -0.0, 0.0),
            torch.where(at < 10, 3.0, -5.0), torch.where(at >= V - 10, 3.0, -5.0),
            torch.where(at % 64 == 0, 1e-30, 0.0)]
    return torch.stack([r.float().to(dtype) for r in rows])


@TYPES
@pytest.mark.parametrize("V", [200, 2000, 2048, 50257, 131072, 140001])
def test_patterns(V, dtype):
    z = patterns(V, dtype, 11)
    T = z.shape[0]
    y = torch.arange(T, device="cuda") % V
    g, h = torch.linspace(-1, 1, T, device="cuda"), torch.full((T,), 0.1, device="cuda")
    for top in (1, 20, 64, 128):
        r = check(z, y, top=top, what=f"top {top}")
    assert r.lse[1] == -math.inf and r.logprobs[1] == -math.inf and r.entropy[1] == 0
    assert r.top_ids[1].tolist() == list(range(128))
    d = check_grad(z, y, g, h)
    assert not d[1].any()
    # many rows: each in one piece where it fits
    many = z.repeat(160, 1)
    ids = mm().token_logprobs(many, None, top=128).top_ids
    assert torch.equal(ids, r.top_ids.repeat(160, 1))


@TYPES
@pytest.mark.parametrize("V", [50, 3000, 131072])
def test_nan_and_infinity(V, dtype):
    z, y, g, h = inputs(8, V, dtype, 12)
    z[1, V // 3] = math.nan
    z[2, V // 2] = math.inf
    z[3, 7] = z[3, 9] = math.inf
    z[4] = math.nan
    r = check(z, y, top=20)
    for t in (r.logprobs, r.entropy, r.lse, r.top_logprobs[:, 0]):
        assert torch.equal(torch.isnan(t), torch.tensor([0, 1, 1, 1, 1, 0, 0, 0], device="cuda").bool())
    assert r.top_ids[3, :2].tolist() == [7, 9] and r.top_ids[4].tolist() == list(range(20))
    d = mm().token_logprobs_backward(z, y, r.lse, r.entropy, g, h)
    assert torch.isnan(d[1:5]).all() and not torch.isnan(d[0]).any() and not torch.isnan(d[5:]).any()
    # weights that are not finite stay in their row
    r = mm().token_logprobs(z[5:], y[5:])
    d = mm().token_logprobs_backward(z[5:], y[5:], r.lse, r.entropy, torch.tensor([math.nan, 1.0, math.inf], device="cuda"))
    assert torch.isnan(d[0]).all() and torch.isfinite(d[1]).all() and not torch.isfinite(d[2]).all()


@TYPES
@pytest.mark.parametrize("V,pad,shift", [(50257, 47, 0), (4097, 1, 1), (333, 3, 5), (2048, 8, 3)])
def test_strides_and_alignment(V, pad, shift, dtype):
    """Padded rows that start at any element; the gradient into strided rows, whose gaps
    stay as they were, and in place."""
    T = 21
    z, y, g, h = inputs(T, V, dtype, 13)
    buf = torch.full((T * (V + pad) + shift,), math.nan, device="cuda", dtype=dtype)
    view = buf[shift:].view(T, V + pad)[:, :V]
    view.copy_(z)
    check(z, y, top=11)
    check(view, y, top=11)                  # sums in another order: the units lie on the 16-byte grid
    check_grad(view, y, g, h)
    a = mm().token_logprobs(z, y)
    d = mm().token_logprobs_backward(z, y, a.lse, a.entropy, g, h)
    assert torch.equal(mm().token_logprobs_backward(view, y, a.lse, a.entropy, g, h), d)
    out = torch.full((T * (V + pad) + shift,), 5.0, device="cuda", dtype=dtype)
    dst = out[shift:].view(T, V + pad)[:, :V]
    assert mm().token_logprobs_backward(z, y, a.lse, a.entropy, g, h, out=dst) is dst
    assert torch.equal(dst, d)
    dst.fill_(5.0)
    assert (out == 5.0).all()
    got = mm().token_logprobs_backward(view, y, a.lse, a.entropy, g, h, out=view)
    assert torch.equal(got, d)
    view.fill_(math.nan)
    assert torch.isnan(buf).all()


@TYPES
@pytest.mark.parametrize("V", [4099, 65543])
def test_beyond_the_caches(V, dtype):
    """More than 256 MiB of logits, rows of every alignment."""
    T = (257 << 20) // (V * dtype.itemsize) + 8
    z, y, g, h = inputs(T, V, dtype, 60, ignored=0.1)
    z[5, 3:] = -math.inf
    z[6] = -math.inf
    for top in (0, 20, 64, 65):
        check(z, y, top=top, what=f"{T}x{V} top {top}")
    check_grad(z, y, g, h, what=f"{T}x{V}")


@TYPES
@pytest.mark.parametrize("V,ld", [(3, 8), (4, 8), (7, 16), (8, 8), (9, 16), (2049, 2056), (8193, 8200), (10007, 10008), (16390, 16392), (16390, 16400)])
def test_gradient_of_aligned_rows(V, ld, dtype):
    """Rows that start on 16 bytes and do not end there, also in place; what lies between stays."""
    z, y, g, h = inputs(37, V, dtype, 61 + V, ignored=0.2)
    want = check_grad(z, y, g, h, 0.9)
    buf = torch.full((37, ld), 7.0, device="cuda", dtype=dtype)
    rows = buf[:, :V]
    rows.copy_(z)
    check(rows, y, 0.9, top=2)
    first = mm().token_logprobs(z, y, scale=0.9)
    assert mm().token_logprobs_backward(rows, y, first.lse, first.entropy, g, h, scale=0.9, out=rows) is rows
    assert torch.equal(rows, want)
    assert (buf[:, V:] == 7.0).all()
    rows.copy_(z)
    assert torch.equal(mm().token_logprobs_backward(rows, y, first.lse, first.entropy, g, h, scale=0.9), want)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    V, ld = 1000, 2 ** 30 + 24
    buf = torch.zeros(3 * ld, device="cuda", dtype=torch.bfloat16)
    z = buf.view(3, ld)[:, :V]
    want, y, g, h = inputs(3, V, torch.bfloat16, 14)
    z.copy_(want)
    a, b = check(want, y, top=5), mm().token_logprobs(z, y, top=5)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    d = check_grad(want, y, g, h)
    a = mm().token_logprobs(want, y)
    assert torch.equal(mm().token_logprobs_backward(z, y, a.lse, a.entropy, g, h, out=z), d)


@TYPES
def test_shards(dtype):
    """A vocabulary in three shards against the whole."""
    z, y, g, h = inputs(50, 9000, dtype, 15, ignored=0.2)
    whole = mm().token_logprobs(z, y, top=30)
    cuts = [0, 1000, 4097, 9000]
    parts, shifted = [], []
    for a, b in zip(cuts, cuts[1:]):
        t = torch.where((y >= a) & (y < b), y - a, mm().TARGET_ELSEWHERE)
        shifted.append(torch.where(y == IGNORE, IGNORE, t))
        parts.append(mm().token_logprobs(z[:, a:b], shifted[-1], top=30))
    kept = y != IGNORE
    lse_s = torch.stack([p.lse for p in parts]).double()
    lse = torch.logsumexp(lse_s, 0)
    lp = sum(p.logprobs.double() + p.lse.double() for p in parts) - lse
    H = lse - sum(torch.exp(s - lse) * (s - p.entropy.double()) for s, p in zip(lse_s, parts))
    ref = reference(z, y)
    for got, name in ((lp, "logprobs"), (H, "entropy"), (lse, "lse")):
        # three parts, each off by its own bound and by the rounding of its lse
        within(torch.where(kept, got, 0.0), ref[name], 4 * ref["t_" + name] + 2.0 ** -20 * (1 + ref["lse"].abs()), name)
    val = torch.cat([p.top_logprobs + p.lse[:, None] for p in parts], 1)
    ids = torch.cat([p.top_ids + a for p, a in zip(parts, cuts)], 1)
    best = torch.gather(ids, 1, torch.topk(z.float().gather(1, ids.clamp(0, 8999)), 30, 1).indices)
    rows = kept.nonzero()[:, 0]
    assert torch.equal(torch.sort(z[rows].float().gather(1, best[rows]), 1).values, torch.sort(z[rows].float().gather(1, whole.top_ids[rows]), 1).values)
    assert val.shape == ids.shape
    lse32, H32 = torch.where(kept, lse, 0.0).float(), torch.where(kept, H, 0.0).float()
    joined = torch.cat([mm().token_logprobs_backward(z[:, a:b], t, lse32, H32, g, h) for a, b, t in zip(cuts, cuts[1:], shifted)], 1)
    want, tol = grad_reference(z, y, lse32, H32, g, h)
    within(joined, want, tol, "gradient")


def test_gradient_against_differences():
    """Central differences of f = Σ g·logprob + h·entropy, computed in fp64 from the
    formulas, with respect to single logits: a step of 2^-10 leaves third derivatives (at
    most 6 of the weights here) times 2^-20/6."""
    z, y, g, h = inputs(6, 40, torch.float32, 16)
    h = h * 100
    scale = 1.25
    r = mm().token_logprobs(z, y, scale=scale)
    d = mm().token_logprobs_backward(z, y, r.lse, r.entropy, g, h, scale=scale).double()

    def f(z):
        lp = torch.log_softmax(z * scale, 1)
        return (g.double() * lp.gather(1, y[:, None])[:, 0] - h.double() * (lp.exp() * lp).sum(1)).sum()
    step = 2.0 ** -10
    bound = 8 * scale ** 3 * step ** 2 * (g.abs() + h.abs() * 10).double() + 2.0 ** -18 * (g.abs() + h.abs() * 10).double()
    for t in range(6):
        for v in range(0, 40, 3):
            up, down = z.double().clone(), z.double().clone()
            up[t, v] += step
            down[t, v] -= step
            assert abs((f(up) - f(down)).item() / (2 * step) - d[t, v].item()) <= bound[t].item()


def test_same_bits_streams_and_graphs():
    m = mm()
    z, y, g, h = inputs(40, 33000, torch.bfloat16, 17, ignored=0.2)
    call = lambda: (*m.token_logprobs(z, y, top=20), m.token_logprobs_backward(z, y, lse, H, g, h))  # noqa: E731
    lse, H = m.token_logprobs(z, y).lse, m.token_logprobs(z, y).entropy
    want = call()
    for _ in range(3):
        for s, t in zip(want, call()):
            assert torch.equal(s, t)
    # on another stream than the current one, while that allocates and writes
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = m.token_logprobs(z, y, top=20, stream=side)
    d = m.token_logprobs_backward(z, y, lse, H, g, h, stream=side)
    for _ in range(10):
        torch.empty_like(z).fill_(3.0)
    side.synchronize()
    for s, t in zip(want, (*r, d)):
        assert torch.equal(s, t)
    # captured, replayed with other inputs and eager work between
    z2, y2, _, _ = inputs(40, 33000, torch.bfloat16, 18, ignored=0.5)
    other = m.token_logprobs(z2, y2, top=20)
    zs, ys = z.clone(), y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = m.token_logprobs(zs, ys, top=20)
        d = m.token_logprobs_backward(zs, ys, lse, H, g, h)
    for src, tgt, ref in ((z, y, want[:5]), (z2, y2, other), (z, y, want[:5])):
        zs.copy_(src)
        ys.copy_(tgt)
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip(r, ref):
            assert torch.equal(s, t)
        m.token_logprobs(z2, y2, top=7)
    assert torch.equal(d, want[5])


def test_no_rows_and_workspace():
    m = mm()
    z = torch.zeros(0, 100, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(0, dtype=torch.int64, device="cuda")
    r = m.token_logprobs(z, y, top=5)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 5)
    assert m.token_logprobs_backward(z, y, r.lse, r.entropy, r.logprobs, r.lse).shape == (0, 100)
    z, y, _, _ = inputs(3, 40000, torch.float32, 19)
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")     # its contents do not matter
    for s, t in zip(m.token_logprobs(z, y, top=9), m.token_logprobs(z, y, top=9, workspace=ws)):
        assert torch.equal(s, t)
    with pytest.raises(ValueError, match="WORKSPACE"):
        m.token_logprobs(z, y, top=9, workspace=ws[:256])


@pytest.mark.parametrize("phase", ["logprobs", "logprobs_grad"])
def test_forced_failures_and_debug_sync(phase, monkeypatch):
    m = mm()
    z, y, g, h = inputs(3, 20000, torch.bfloat16, 20)
    r = m.token_logprobs(z, y, top=3)
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", phase)
    with pytest.raises(RuntimeError, match="forced failure"):
        m.token_logprobs(z, y)
        m.token_logprobs_backward(z, y, r.lse, r.entropy, g, h)
    monkeypatch.delenv("DMUON_TEST_FAIL_AT")
    monkeypatch.setenv("DMUON_DEBUG_SYNC", "1")
    for s, t in zip(r, m.token_logprobs(z, y, top=3)):
        assert torch.equal(s, t)
