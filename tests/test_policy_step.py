"""One step of policy-gradient training out of the library's parts: embedding, log
probabilities and entropies from hidden states (and from logits) as autograd Functions,
the clipped gradients, and the two optimizer routes."""
import pytest
import torch

import matrix_optimizer_muon_amd as mm


class Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table):
        ctx.save_for_backward(ids)
        ctx.rows = table.shape[0]
        return mm.embedding(ids, table)

    @staticmethod
    def backward(ctx, grad):
        return None, mm.embedding_backward(ctx.saved_tensors[0], grad, ctx.rows)


class LinearLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, y, scale):
        r = mm.linear_token_logprobs(h, w, y, scale=scale)
        ctx.save_for_backward(h, w, y, r.lse, r.entropy)
        ctx.scale = scale
        return r.logprobs, r.entropy

    @staticmethod
    def backward(ctx, g, e):
        h, w, y, lse, entropy = ctx.saved_tensors
        return (*mm.linear_token_logprobs_backward(h, w, y, lse, entropy, g.contiguous(), e.contiguous(), scale=ctx.scale), None, None)


class Logprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, y, scale):
        r = mm.token_logprobs(z, y, scale=scale)
        ctx.save_for_backward(z, y, r.lse, r.entropy)
        ctx.scale = scale
        return r.logprobs, r.entropy

    @staticmethod
    def backward(ctx, g, e):
        z, y, lse, entropy = ctx.saved_tensors
        return mm.token_logprobs_backward(z, y, lse, entropy, g.contiguous(), e.contiguous(), scale=ctx.scale), None, None


def policy_loss(logprobs, entropy, old, advantage, n):
    """Clipped ratio with an entropy bonus, a mean over the n tokens that count."""
    ratio = torch.exp(logprobs - old)
    gain = torch.minimum(ratio * advantage, ratio.clamp(0.8, 1.2) * advantage)
    return -(gain + 0.01 * entropy).sum() / n


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True], ids=["hidden", "logits"])
def test_step(kept):
    g = torch.Generator(device="cuda").manual_seed(5)
    V, D, T, scale = 300, 64, 130, 1.25
    leaf = lambda *s, k: (torch.randn(*s, generator=g, device="cuda") * k).requires_grad_()  # noqa: E731
    table, lin, head = leaf(V, D, k=0.5), leaf(D, D, k=0.2), leaf(V, D, k=0.3)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::9] = -100
    n = (y != -100).sum()
    advantage = torch.randn(T, generator=g, device="cuda") * (y != -100)

    def forward(params, emb, logp):
        table, lin, head = params
        return logp(emb(ids, table) @ lin.T, head)

    own = (lambda h, w: Logprobs.apply(h @ w.T, y, scale)) if kept else (lambda h, w: LinearLogprobs.apply(h, w, y, scale))

    def plain(h, w):
        lp = torch.log_softmax(h @ w.T * scale, 1)
        keep = y != -100
        return torch.where(keep, lp.gather(1, y.clamp(min=0)[:, None])[:, 0], 0.0), torch.where(keep, -(lp.exp() * lp).sum(1), 0.0)

    params = [table, lin, head]
    exact = [p.detach().double().requires_grad_() for p in params]
    with torch.no_grad():
        old = plain(table[ids].double() @ lin.double().T, head.double())[0].float() + 0.1 * torch.randn(T, generator=g, device="cuda")
    loss = policy_loss(*forward(params, Embedding.apply, own), old, advantage, n)
    want = policy_loss(*forward(exact, lambda i, t: t[i], plain), old.double(), advantage.double(), n)
    loss.backward()
    want.backward()
    # sums of at most 300 fp32 products at every step, four steps deep: (4·300)·2^-23 of
    # magnitudes that cancel to no less than a tenth here; a ratio within 2^-20 of the clip's
    # border would change sides, which the draw avoids
    ratio = torch.exp(plain(exact[0].detach()[ids] @ exact[1].detach().T, exact[2].detach())[0] - old.double())
    assert min((ratio - 0.8).abs().min(), (ratio - 1.2).abs().min()) > 2.0 ** -16
    assert abs(loss.item() - want.item()) <= 2e-3 * abs(want.item())
    for p, q in zip(params, exact):
        assert torch.linalg.norm(p.grad.double() - q.grad) <= 2e-3 * torch.linalg.norm(q.grad)

    # the gradients clipped to a third of their norm, into a packed bf16 buffer for the steps
    grads = [p.grad for p in params]
    norm = mm.grad_norm(grads)
    want_norm = sum((p.grad ** 2).sum() for p in exact).sqrt()
    assert abs(norm.double() - want_norm) <= 2e-3 * want_norm
    limit = norm.item() / 3
    flat = torch.empty(sum(p.numel() for p in params), dtype=torch.bfloat16, device="cuda")
    outs = [t.view(p.shape) for t, p in zip(flat.split([p.numel() for p in params]), params)]
    clip = mm.ClipGradNorm(grads, limit, outs=outs)
    assert torch.equal(clip(), norm)
    for o, p in zip(outs, params):          # two roundings to fp32, one to bf16
        ref = p.grad.double() * (limit / (norm.double() + 1e-6))
        assert ((o.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * ref.abs()).all()
    # both routes take them as they are: the same steps from copies give the same bits
    results = []
    for source in (outs, [o.clone() for o in outs]):
        masters, momenta = [lin.detach().clone()], [torch.zeros_like(lin)]
        mm.muon_step([source[1]], momenta, masters, lr=0.02)
        vecs = [table.detach().clone(), head.detach().clone()]
        state = [[torch.zeros_like(v) for v in vecs] for _ in range(2)]
        mm.adamw_step(vecs, [source[0], source[2]], *state, step=1, lr=1e-3)
        results.append((*masters, *momenta, *vecs))
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert not torch.equal(results[0][0], lin.detach()) and not torch.equal(results[0][2], table.detach())


@pytest.mark.gpu
def test_distilled_alternatives():
    """A teacher's alternatives as another model's targets: a call per rank."""
    g = torch.Generator(device="cuda").manual_seed(6)
    teacher, student = (torch.randn(20, 500, generator=g, device="cuda") * 2 for _ in range(2))
    top = mm.token_logprobs(teacher, top=8)
    assert top.logprobs is None
    got = torch.stack([mm.token_logprobs(student, top.top_ids[:, k].contiguous()).logprobs for k in range(8)], 1)
    want = torch.log_softmax(student.double(), 1).gather(1, top.top_ids)
    assert (got.double() - want).abs().max() <= 2.0 ** -18       # sums of 500 terms, values below 16
    assert torch.equal(top.top_ids, torch.sort(teacher, dim=1, descending=True, stable=True).indices[:, :8])


def test_the_parts_refuse_what_autograd_would_record():
    z, w, y = torch.zeros(4, 8, requires_grad=True), torch.zeros(5, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: mm.token_logprobs(z, y), lambda: mm.linear_token_logprobs(z, w, y)):
        with pytest.raises(ValueError, match="requires gradients"):
            call()
