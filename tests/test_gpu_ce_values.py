"""Cross entropy where single values decide: logits that are exact in fp32, from 1e4 to
the end of the type, and tokens certain of their target (needs an MI355X).

The logits of these inputs are products of two numbers with 8 significant bits (every
other product of the sum is 0), so they carry no rounding and the bounds can be those
of the softmax alone:

* exp(z − m) is off by 2^-22 of its value (the difference rounds by 2^-24 of itself and
  is at most 88 where the exponential counts; the instruction by an ulp), a sum of n
  of them in fp32 by n·2^-24; a token's sum has at most 160 + V/512 terms in a row
  (a lane's 64, the exchanges, the tiles' statistics);
* log of the sum is then off by as much absolutely, plus 2^-23 of its own value (at most
  16), and losses and lse are rounded once more.
"""
import math

import pytest
import torch

from test_gpu_training import IGNORE, U, gen, mm, randn, within

pytestmark = pytest.mark.gpu

SIZES = [(16, 64, 500), (100, 64, 900), (100, 70, 333), (2001, 800, 6500)]      # few tokens, 128 tiles (two widths), 256 tiles
TYPES = [(torch.bfloat16, *s) for s in SIZES] + [(torch.float32, *s) for s in SIZES[:3]] + [(torch.float32, 2001, 136, 6500)]


def eight_bits(g, *shape):
    """±(128 … 255)/128, uniformly."""
    x = torch.randint(128, 256, shape, generator=g, device="cuda").float() / 128
    return torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.5, -x, x)


def exact_inputs(T, D, V, dtype, top, seed):
    """h holds one number per token, w anything but in that column: z = h[:, 0]·w[:, 0],
    all |z| < 4·2^k with 2^k the power of two below top/4."""
    g = gen(seed)
    k = int(math.floor(math.log2(top / 4)))
    h = torch.zeros(T, D, device="cuda")
    h[:, 0] = eight_bits(g, T) * 2.0 ** (k // 2)
    w = randn(g, V, D)
    w[:, 0] = eight_bits(g, V) * 2.0 ** (k - k // 2)
    h, w = h.to(dtype), w.to(dtype)
    z = h[:, :1].double() * w[:, 0].double()[None]
    assert torch.equal(z.float().double(), z)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::2] = z.argmax(1)[::2]                                  # certain of their target
    return h, w, y, z


@pytest.mark.parametrize("top", [40.0, 1e4, 1e10, 1e30, 3.4e38])
@pytest.mark.parametrize("dtype,T,D,V", TYPES)
def test_exact_logits_of_any_size(dtype, T, D, V, top):
    m = mm()
    h, w, y, z = exact_inputs(T, D, V, dtype, top, T + int(math.log2(top)))
    losses, lse = m.linear_cross_entropy(h, w, y)
    most = z.amax(1)
    logs = torch.log(torch.exp(z - most[:, None]).sum(1))
    want = (most - z.gather(1, y[:, None])[:, 0]) + logs
    tol = (160 + V / 512 + 4) * 2.0 ** -24 + 16 * 2.0 ** -23
    within(losses, torch.where(want > torch.finfo(torch.float32).max, math.inf, want), tol + 2.0 ** -22 * want, "loss")
    within(lse, most + logs, tol + 2.0 ** -23 * (most + logs).abs(), "lse")
    assert (losses >= 0).all()
    # the gradients, from the lse they are given
    gl = torch.full((T,), 1 / T, device="cuda")
    dh, dw = m.linear_cross_entropy_backward(h, w, y, lse, gl)
    d = z - lse.double()[:, None]
    p = torch.exp(d)
    dz = p.clone()
    dz.scatter_add_(1, y[:, None], torch.full_like(dz[:, :1], -1))
    # p: as above; a difference with 1 and the products' roundings; dz in bf16 (fp32: three planes, 2^-22)
    e = p * (2.0 ** -22 + 2.0 ** -22 * d.abs().clamp(max=200)) + 2.0 ** -126 + 2.0 ** -23 * dz.abs()
    e = (e + (U[dtype] if dtype == torch.bfloat16 else 2.0 ** -22) * (dz.abs() + e)) / T * (1 + 2.0 ** -20)
    dz = dz * gl.double()[:, None]
    for got, want, s, n, what in ((dh, dz @ w.double(), (dz.abs() + e) @ w.double().abs(), V, "dh"),
                                  (dw, dz.T @ h.double(), (dz.abs() + e).T @ h.double().abs(), T, "dw")):
        err = e @ w.double().abs() if what == "dh" else e.T @ h.double().abs()
        tol = err + (n + 64) * 2.0 ** -23 * s + (n + 2) * 2.0 ** -126
        within(got, want, tol + U[dtype] * (want.abs() + tol), what)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_loss_is_never_negative(dtype):
    """Tokens certain of their target, logits of 10 to 60: a loss of 0 or just above it,
    the same whether few tokens or many are asked for."""
    m = mm()
    g = gen(5)
    T, D, V = 300, 64, 700
    h, w = randn(g, T, D), randn(g, V, D) * 0.01
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    w[:, 0] = 0
    h[:, 0] = torch.rand(T, generator=g, device="cuda") * 50 + 10
    w[5, 0] = 1
    y[:] = 5                                                   # z of the target 10 … 60, of the others about 0
    h, w = h.to(dtype), w.to(dtype)
    losses, lse = m.linear_cross_entropy(h, w, y)
    assert (losses >= 0).all() and (losses[h[:, 0] > 30] < 1e-6).all()
    few, few_lse = m.linear_cross_entropy(h[:16], w, y[:16])
    # both sum V exponentials below 1 beside the target's 1, in different orders
    assert ((few - losses[:16]).abs() <= 2 * 2.0 ** -24 * (200 + 16) * (1 + losses[:16])).all()
    assert ((few_lse - lse[:16]).abs() <= 2.0 ** -22 * lse[:16].abs()).all()
