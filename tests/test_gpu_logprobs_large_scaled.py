"""Gradients of large logits whose scaled values fp32 cannot hold exactly (needs an MI355X).
The lse they are computed from is rounded to fp32, so x − lse of a row's largest may come out
above 0, by up to half a step of lse: from |lse| = 2^16 on a probability stays at most 1."""
import pytest
import torch
from test_gpu_logprobs import IGNORE, TYPES, U, gen, mm, randn, within

pytestmark = pytest.mark.gpu

SCALES = [0.7, 1.25, 3.3]
SIZES = [1e4, 1e6, 1e8, 1e10, 1e20, 1e37]


def rows(T, V, size, dtype, seed):
    g = gen(seed)
    z = (randn(g, T, V) * 0.2 * size).clamp(-size, size)
    z[1] = z[1].abs().amax()
    z[2] = -z[2].abs()
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[3] = IGNORE
    y[4] = z[4].argmax()
    z[5] = -size                            # nothing but the mask's value
    return z.to(dtype), y, randn(g, T) / T, -0.01 * torch.rand(T, generator=g, device="cuda") / T


def reference(x, y, lse, H, g, h, scale):
    """dz and its bound: the formula in fp64 from the same lse, with p ≤ 1 where that is large."""
    l = x - lse.double()[:, None]
    l = torch.where(lse.abs()[:, None] < 2.0 ** 16, l, l.clamp(max=0.0))
    p = torch.exp(l)
    l = torch.where(p > 0, l, 0.0)
    inner = g.double()[:, None] + h.double()[:, None] * (l + H.double()[:, None])
    hot = torch.zeros_like(x).scatter_(1, y.clamp(min=0)[:, None], g.double()[:, None])
    part = (y != IGNORE)[:, None]
    mag = g.double().abs()[:, None] + h.double().abs()[:, None] * (l.abs() + H.double().abs()[:, None])
    tol = scale * (p * mag * (3 * l.abs() + 12) * 2.0 ** -24 + 2.0 ** -22 * ((p * inner).abs() + hot.abs()) + 2.0 ** -126 * (2 + mag))
    return torch.where(part, scale * (hot - p * inner), 0.0), tol


@TYPES
@pytest.mark.parametrize("V", [1, 5, 300, 9000, 20000])
@pytest.mark.parametrize("size", SIZES)
def test_from_logits(V, size, dtype):
    z, y, g, h = rows(20, V, size, dtype, 50 + V)
    for scale in SCALES:
        scale = torch.tensor(scale).item()
        r = mm().token_logprobs(z, y, scale=scale)
        d = mm().token_logprobs_backward(z, y, r.lse, r.entropy, g, h, scale=scale)
        want, tol = reference(z.double() * scale, y, r.lse, r.entropy, g, h, scale)
        within(d, want, tol + U[dtype] * want.abs() + 2.0 ** -126, f"{size} scale {scale}")


@TYPES
@pytest.mark.parametrize("T", [20, 300])
@pytest.mark.parametrize("size", SIZES[:-1])
def test_from_hidden_states(T, size, dtype):
    """Logits that are exact: weights in one column, hidden states a power of 2 there."""
    V, D = 700, 8
    w1 = randn(gen(61), V).to(dtype)
    y = torch.randint(0, V, (T,), generator=gen(62), device="cuda")
    y[3] = IGNORE
    g, h = randn(gen(63), T) / T, torch.full((T,), -0.01 / T, device="cuda")
    w = torch.zeros(V, D, device="cuda", dtype=dtype)
    w[:, 0] = w1
    hs = torch.zeros(T, D, device="cuda", dtype=dtype)
    hs[:, 0] = 2.0 ** torch.tensor(float(size)).log2().round().item()
    for scale in SCALES:
        scale = torch.tensor(scale).item()
        r = mm().linear_token_logprobs(hs, w, y, scale=scale)
        gh, gw = mm().linear_token_logprobs_backward(hs, w, y, r.lse, r.entropy, g, h, scale=scale)
        assert torch.isfinite(gh).all() and torch.isfinite(gw).all(), f"{size} scale {scale}"
        x = hs[:, :1].double() * w1.double() * scale
        dz, tol = reference(x, y, r.lse, r.entropy, g, h, scale)
        # dz relative to the largest weight in bf16, the sums' order and the results' rounding
        u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -21
        off = tol + u * dz.abs()
        want = dz @ w.double()
        within(gh, want, off @ w.double().abs() + 2 * u * want.abs() + 2.0 ** -100, f"{size} scale {scale} grad_h")
        want = dz.T @ hs.double()
        within(gw, want, off.T @ hs.double().abs() + 2 * u * want.abs() + 2.0 ** -100, f"{size} scale {scale} grad_w")
