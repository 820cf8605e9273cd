"""Alternatives of rows cut into pieces that a wave takes each and a second launch joins
(needs an MI355X): ties, masks, signed zeros and lists that overflow, in that route."""
import math

import pytest
import torch
from test_gpu_logprobs import TYPES, gen, mm, patterns, randn, reference, within

pytestmark = pytest.mark.gpu


def check_ids(z, tops, what):
    """ids and log probabilities against the reference, for which −0 and 0 are one value."""
    for top in tops:
        ref = reference(z + 0.0, None, top=top)
        r = mm().token_logprobs(z, top=top)
        assert torch.equal(r.top_ids, ref["ids"]), f"{what} top {top}"
        within(r.top_logprobs, ref["best"], ref["t_best"], f"{what} top {top}")


def zeros_of_both_signs(V, piece, dtype, seed):
    """Rows whose largest value is 0, as −0, +0 or both, within units and across pieces."""
    at = torch.arange(V, device="cuda")
    base = randn(gen(seed), V)
    first = at < piece
    zero, minus = torch.zeros(V, device="cuda"), torch.full((V,), -0.0, device="cuda")
    rows = [minus,
            torch.where(at % 2 == 0, minus, zero),
            torch.where(at % 8 < 4, minus, zero), torch.where(at % 8 < 4, zero, minus),
            torch.where(first, minus, zero), torch.where(first, zero, minus),
            torch.where(first & (at % 4 == 0), -1.0, torch.where(first, minus, zero)),
            torch.where(at % 4 == 0, -1.0, minus),
            torch.where(at // piece % 2 == 0, torch.where(at % 4 == 0, -1.0, minus), zero),
            torch.where(at % 4 == 3, minus, -2.0), torch.where(at % 3 == 1, minus, -math.inf),
            base * 0.0, base.clamp(max=0.0) * (base > 0), torch.where(base < -1, base, base * 0.0)]
    return torch.stack([r.to(dtype) for r in rows])


# rows × words, words of a piece: up to 64, 128, 256 units each, and more
ROUTES = [(70, 32000, 2000), (72, 50257, 2016), (150, 50257, 3592), (500, 12500, 2504), (500, 12289, 2464)]


@TYPES
@pytest.mark.parametrize("T,V,piece", ROUTES)
def test_zeros(T, V, piece, dtype):
    z = zeros_of_both_signs(V, piece, dtype, 70)
    check_ids(z.repeat(-(-T // z.shape[0]), 1)[:T], (20, 33, 64, 128), f"{T}x{V}")


@TYPES
@pytest.mark.parametrize("V", [300, 1000, 2000, 4000, 9000, 20000, 140001])
def test_zeros_in_other_routes(V, dtype):
    """Few rows, and rows enough for one piece each."""
    z = zeros_of_both_signs(V, 2000, dtype, 71)
    check_ids(z, (20, 33, 64, 128), f"{V}")
    many = z.repeat(80, 1)
    ids = mm().token_logprobs(many, top=128).top_ids
    assert torch.equal(ids, mm().token_logprobs(z, top=128).top_ids.repeat(80, 1))


@TYPES
@pytest.mark.parametrize("T,V,piece", ROUTES)
def test_patterns(T, V, piece, dtype):
    z = patterns(V, dtype, 72)
    z = z.repeat(-(-T // z.shape[0]), 1)[:T]
    check_ids(z, (1, 20, 33, 64, 128), f"{T}x{V}")
