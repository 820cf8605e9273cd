"""The training operators beside autograd: the forward calls record nothing, so they refuse
inputs that require gradients where autograd would; as the halves of a
``torch.autograd.Function`` their gradients flow."""
import pytest
import torch

import matrix_optimizer_muon_amd as mm


def refusal(call):
    with pytest.raises(ValueError) as e:
        call()
    return str(e.value)


def test_inputs_that_require_gradients_are_refused():
    h, w = torch.zeros(4, 8, requires_grad=True), torch.zeros(5, 8)
    y = torch.zeros(4, dtype=torch.int64)
    head = w.clone().requires_grad_()
    for call, name in ((lambda: mm.linear_cross_entropy(h, w, y), "h"), (lambda: mm.linear_cross_entropy(h.detach(), head, y), "w"),
                       (lambda: mm.linear_cross_entropy(h * 2, w, y), "h"), (lambda: mm.embedding(y, head), "table")):
        assert refusal(call).startswith(f"{name} requires gradients")
        # not where nothing is recorded (the refusal is then another one: CPU tensors)
        with torch.no_grad():
            assert "GPU tensor" in refusal(call)
    assert "GPU tensor" in refusal(lambda: mm.linear_cross_entropy(h.detach(), w, y))
    # what is kept for the backward pass, and the backward calls themselves, are not recorded anyway
    for call in (lambda: mm.checkpoint_quantize(h), lambda: mm.embedding_backward(y, h, 5),
                 lambda: mm.linear_cross_entropy_backward(h, head, y, y, y)):
        assert "GPU tensor" in refusal(call)


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table):
        ctx.save_for_backward(ids)
        ctx.rows = table.shape[0]
        return mm.embedding(ids, table)

    @staticmethod
    def backward(ctx, grad):
        return None, mm.embedding_backward(ctx.saved_tensors[0], grad, ctx.rows)


class Linear(torch.autograd.Function):
    """x·Wᵀ whose input is kept in 8 bits."""
    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(w, *mm.checkpoint_quantize(x))
        return x @ w.T

    @staticmethod
    def backward(ctx, grad):
        w, q, exps = ctx.saved_tensors
        return grad @ w, mm.checkpoint_wgrad(grad, q, exps)


class CrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, y):
        losses, lse = mm.linear_cross_entropy(h, w, y)
        ctx.save_for_backward(h, w, y, lse)
        return losses

    @staticmethod
    def backward(ctx, grad):
        h, w, y, lse = ctx.saved_tensors
        return (*mm.linear_cross_entropy_backward(h, w, y, lse, grad.contiguous()), None)


@pytest.mark.gpu
def test_as_autograd_functions():
    """Embedding → linear → cross entropy in fp32 through loss.backward(), against torch's
    own graph in fp64 on what the checkpoint holds."""
    g = torch.Generator(device="cuda").manual_seed(3)
    V, D, T = 200, 96, 150
    leaf = lambda *s, k=0.3: (torch.randn(*s, generator=g, device="cuda") * k).requires_grad_()
    table, lin, head = leaf(V, D), leaf(D, D, k=0.1), leaf(V, D)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = ids.roll(-1).clone()
    y[::7] = -100
    n = (y != -100).sum()
    x = Embedding.apply(ids, table)
    loss = CrossEntropy.apply(Linear.apply(x, lin), head, y).sum() / n
    loss.backward()
    # the same in fp64; the linear layer's weight gradient sees the checkpoint's values
    t64, l64, h64 = (p.detach().double().requires_grad_() for p in (table, lin, head))
    q, exps = mm.checkpoint_quantize(x.detach())
    kept = mm.checkpoint_dequantize(q, exps, dtype=torch.float32).double()
    x64 = t64[ids]
    hid = x64 @ l64.detach().T + (kept @ l64.T - kept @ l64.detach().T)     # value x·Wᵀ, gradients by each route
    want = torch.nn.functional.cross_entropy(hid @ h64.T, y, ignore_index=-100)
    want.backward()
    # sums of at most 200 fp32 products at every step, four steps deep: (4·200)·2^-23 of
    # their magnitudes, which cancel to no less than a tenth here
    assert abs(loss.item() - want.item()) <= 1e-3 * abs(want.item())
    for got, ref in ((table, t64), (lin, l64), (head, h64)):
        assert got.grad.shape == got.shape
        assert torch.linalg.norm(got.grad.double() - ref.grad) <= 1e-3 * torch.linalg.norm(ref.grad)
