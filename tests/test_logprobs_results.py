"""What the log-probability functions return, in the hands of autograd (needs an MI355X)."""
import pytest
import torch

import matrix_optimizer_muon_amd as mm

pytestmark = pytest.mark.gpu


def inputs(hidden):
    g = torch.Generator(device="cuda").manual_seed(2)
    y = torch.randint(0, 50, (12,), generator=g, device="cuda")
    if hidden:
        return (torch.randn(12, 16, generator=g, device="cuda"), torch.randn(50, 16, generator=g, device="cuda")), y
    return (torch.randn(12, 50, generator=g, device="cuda"),), y


def score(inputs, y, **kw):
    return (mm.linear_token_logprobs if len(inputs) == 2 else mm.token_logprobs)(*inputs, y, **kw)


@pytest.mark.parametrize("hidden", [False, True], ids=["logits", "hidden"])
def test_results_are_tensors_of_their_own(hidden):
    x, y = inputs(hidden)
    r = [t for t in score(x, y, **({} if hidden else {"top": 4})) if t is not None]
    before = [t.clone() for t in r]
    assert len({t.untyped_storage().data_ptr() for t in r}) == len(r)
    r[0].fill_(3.0)
    assert not any(t._is_view() for t in r)
    assert [t._version for t in r] == [1] + [0] * (len(r) - 1)
    for t, b in zip(r[1:], before[1:]):
        assert torch.equal(t, b)


@pytest.mark.parametrize("hidden", [False, True], ids=["logits", "hidden"])
def test_results_changed_in_place(hidden):
    """A Function that returns them as they are: its caller may mask them in place."""
    class Score(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, *x):
            r = score(x, y)
            ctx.save_for_backward(y, r.lse, r.entropy, *x)
            return r.logprobs, r.entropy.clone()

        @staticmethod
        def backward(ctx, g, e):
            y, lse, entropy, *x = ctx.saved_tensors
            back = mm.linear_token_logprobs_backward if len(x) == 2 else mm.token_logprobs_backward
            d = back(*x, y, lse, entropy, g.contiguous(), e.contiguous())
            return (None, *(d if len(x) == 2 else (d,)))

    x, y = inputs(hidden)
    keep = (torch.arange(12, device="cuda") % 3 > 0).float()
    leaves = [t.clone().requires_grad_() for t in x]
    lp, H = Score.apply(y, *leaves)
    lp.mul_(keep)
    H.add_(1.0)
    (lp + H).sum().backward()
    plain = [t.clone().requires_grad_() for t in x]
    lp, H = Score.apply(y, *plain)
    (lp * keep + H).sum().backward()
    for a, b in zip(leaves, plain):
        assert torch.equal(a.grad, b.grad)


@pytest.mark.parametrize("hidden", [False, True], ids=["logits", "hidden"])
def test_expanded_gradients_are_refused(hidden):
    """What sum() hands to a Function's backward has strides of 0: made contiguous first."""
    x, y = inputs(hidden)
    r = score(x, y)
    back = mm.linear_token_logprobs_backward if hidden else mm.token_logprobs_backward
    g = torch.ones((), device="cuda").expand(12)
    for args in ((g, None), (None, g)):
        with pytest.raises(ValueError, match="contiguous"):
            back(*x, y, r.lse, r.entropy, *args)
    back(*x, y, r.lse, r.entropy, g.contiguous(), g.contiguous())
