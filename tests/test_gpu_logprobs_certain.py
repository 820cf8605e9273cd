"""Rows that are certain of a word, or nearly (needs an MI355X): a probability is not above 1,
an entropy not below 0, and what is small keeps its digits.

Bounds.  The reference M = m·scale·log2 e of the largest logit m is off by r, at most half a
step of M: |r| ≤ 2^-24·|M|.  The largest word's term is R = 2^r as computed, in the sum s and
in the divisor: s/R is 1 exactly where no other term is left, so log S is 0 there.  With other
terms the sum S loses at most all of them, or a half step of 2^-24 per addition.  The second
sum holds r·R beside them, and each of its additions rounds to half a step of that.  A term
below 2^-126 may become 0."""
import math

import pytest
import torch
from test_gpu_logprobs import TYPES, gen, mm, randn

pytestmark = pytest.mark.gpu

# a wave's row (short and long), a workgroup's, pieces by workgroups
VOCABS = [1, 5, 12, 200, 3000, 9000, 20000, 140001]
SCALES = [1.0, 0.7, 1.25, 3.3]
LOG2E = 1.4426950408889634


def values(n, dtype, seed):
    g = gen(seed)
    z = torch.cat([randn(g, n) * 3, randn(g, n) * 30, randn(g, n) * 3000, torch.tensor([2.5, -2.5, 0.1, 7.3, 30.7, -0.0, 1e-30], device="cuda")])
    return z.to(dtype)


@TYPES
@pytest.mark.parametrize("V", VOCABS)
def test_one_word_left(V, dtype):
    """A grammar's forced token: log probability and log of the sum 0, entropy 0."""
    v = values(40, dtype, 1)
    T = v.numel()
    at = (torch.arange(T, device="cuda") * 7919) % V
    z = torch.full((T, V), -math.inf, device="cuda", dtype=dtype)
    z.scatter_(1, at[:, None], v[:, None])
    for scale in SCALES:
        for top in (0, 1, min(V, 64)):
            r = mm().token_logprobs(z, at, top=top, scale=scale)
            assert not r.logprobs.any(), f"scale {scale}: log probability of a certain word {r.logprobs.abs().max().item()}"
            assert torch.equal(r.lse, v.float() * scale)
            assert (r.entropy >= 0).all(), f"scale {scale}: entropy {r.entropy.min().item()}"
            assert (r.entropy.double() <= 2.0 ** -48 * LOG2E * (v.double() * scale).abs()).all()
            if top:
                assert torch.equal(r.top_ids[:, 0], at) and not r.top_logprobs[:, 0].any()


@TYPES
@pytest.mark.parametrize("V", VOCABS[2:])
@pytest.mark.parametrize("gap", [10.0, 20.0, 25.0, 30.0, 45.0, 80.0])
def test_a_word_far_ahead(V, gap, dtype):
    T = 60
    g = gen(int(gap) + V)
    lead = (randn(g, T) * 20).to(dtype)
    z = (lead.float()[:, None] - gap - torch.rand(T, V, generator=g, device="cuda")).to(dtype)
    at = torch.randint(0, V, (T,), generator=g, device="cuda")
    z.scatter_(1, at[:, None], lead[:, None])
    n = 64 + max(V / 256, min(V, 12288) / 64)
    for scale in SCALES:
        x = z.double() * scale
        d = x - x.amax(1, keepdim=True)
        e = torch.exp(d)
        rest = e.sum(1) - 1
        k1, k2 = (-d * e).sum(1) / (1 + rest), (d * d * e).sum(1) / (1 + rest)
        u = 2.0 ** -24
        s_off = torch.minimum(rest, (2 * n + 128) * u * (1 + rest)) + 8 * u * rest + 3 * u * k1
        M = LOG2E * x.amax(1).abs()
        h_off = s_off * (1 + k1) + (2 * n + 160) * u * k1 + 3 * u * k2 + (2 * n + 128) * u * u * M + V * 2.0 ** -126 * d.abs().amax(1)
        want = torch.log1p(rest) + k1
        r = mm().token_logprobs(z, at, top=3 if V > 3 else 1, scale=scale)
        off = (r.entropy.double() - want).abs() / h_off
        assert (r.entropy >= 0).all() and (off <= 1).all(), f"scale {scale}: entropy {r.entropy.min().item()}, {off.max().item():.2f} of the bound"
        off = (r.logprobs.double() + torch.log1p(rest)).abs() / (s_off + 4 * u * torch.log1p(rest))
        assert (r.logprobs <= 0).all() and (off <= 1).all(), f"scale {scale}: log probability {r.logprobs.max().item()}, {off.max().item():.2f} of the bound"
        assert (r.top_logprobs <= 0).all() and torch.equal(r.top_ids[:, 0], at)


@TYPES
@pytest.mark.parametrize("V", VOCABS)
def test_signs(V, dtype):
    """Rows of every spread, equal largest words among them."""
    g = gen(3 + V)
    for spread in (0.0, 0.01, 1.0, 5.0, 40.0, 1000.0, 1e8):
        z = (randn(g, 100, V) * spread).to(dtype)
        z[1] = z[1].amax()
        y = z.float().argmax(1)
        for scale in SCALES:
            r = mm().token_logprobs(z, y, top=min(V, 5), scale=scale)
            assert (r.entropy >= 0).all() and (r.logprobs <= 0).all() and (r.top_logprobs <= 0).all(), f"spread {spread} scale {scale}"


@TYPES
@pytest.mark.parametrize("T", [5, 40, 200, 700])
def test_signs_from_hidden_states(T, dtype):
    """The other face: few tokens, and tiles of both sizes."""
    g = gen(4 + T)
    for spread in (0.0, 1.0, 30.0, 1000.0):
        w = randn(g, 5000, 32).to(dtype)
        h = (randn(g, T, 32) * spread / 5).to(dtype)
        y = (h.float() @ w.float().T).argmax(1)
        for scale in SCALES:
            r = mm().linear_token_logprobs(h, w, y, scale=scale)
            assert (r.entropy >= 0).all() and (r.logprobs <= 0).all(), f"spread {spread} scale {scale}"
