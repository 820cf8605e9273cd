"""The cases by which the operators of policy-gradient steps are measured.

Between a model's logits and the optimizer routes stand:

* ``tokens``: log probabilities of given tokens with the entropy and the most likely
  alternatives, from logits in memory, and the gradient (``token_logprobs`` and its
  backward pass);
* ``linear``: the same log probabilities and entropies straight from hidden states and
  the head's weight, logits never kept, and the gradients (``linear_token_logprobs`` and
  its backward pass);
* ``clip``: the global norm of all gradients and the clipped gradients
  (``ClipGradNorm``).

``run`` computes a case in its plain form (elementary torch operations in fp32; sums of
squares in fp64) or, where ``own`` is true, through the package.
"""
import itertools
import math

import torch

own = False

IGNORE = -100
EPS = 1e-6                       # added to the norm before the division


def listed():
    return [
        # one decoding step of one request: the sampled token and 20 alternatives
        {"name": "tokens 1 of 128000", "op": "tokens", "pass": "forward", "T": 1, "V": 128000, "pad": 0, "type": "bf16", "top": 20, "scale": 1.0, "ignored": 0.0, "masked": 0.0},
        # one step of a batch of requests at a temperature, fp32 logits, words masked out by a grammar
        {"name": "tokens 64 of 32000", "op": "tokens", "pass": "forward", "T": 64, "V": 32000, "pad": 0, "type": "f32", "top": 5, "scale": 1.25, "ignored": 0.0, "masked": 0.5},
        # rollouts scored by the policy that made them: no alternatives
        {"name": "tokens 8192 of 128000", "op": "tokens", "pass": "forward", "T": 8192, "V": 128000, "pad": 0, "type": "bf16", "top": 0, "scale": 1.0, "ignored": 0.0, "masked": 0.0},
        # a teacher's 64 most likely words per position, rows padded to a multiple of 64 words
        {"name": "tokens 2001 of 50257", "op": "tokens", "pass": "forward", "T": 2001, "V": 50257, "pad": 47, "type": "bf16", "top": 64, "scale": 1.0, "ignored": 0.1, "masked": 0.0},
        # the gradient of a policy loss with an entropy bonus
        {"name": "tokens grad 4096 of 128000", "op": "tokens", "pass": "grad", "T": 4096, "V": 128000, "pad": 0, "type": "bf16", "top": 0, "scale": 1.0, "ignored": 0.25, "masked": 0.0},
        # a small fp32 model, nothing a multiple of anything
        {"name": "tokens grad fp32", "op": "tokens", "pass": "grad", "T": 517, "V": 10007, "pad": 0, "type": "f32", "top": 0, "scale": 0.5, "ignored": 0.1, "masked": 0.0},
        # a few positions scored from their hidden states: W is read once
        {"name": "linear 16 tokens", "op": "linear", "pass": "forward", "T": 16, "D": 2048, "V": 32000, "type": "bf16", "scale": 1.0, "ignored": 0.0},
        # a batch of rollouts scored without keeping logits
        {"name": "linear 4096 tokens", "op": "linear", "pass": "forward", "T": 4096, "D": 4096, "V": 32000, "type": "bf16", "scale": 1.0, "ignored": 0.0},
        # a policy-gradient batch: prompts masked out, an odd vocabulary
        {"name": "linear grad masked", "op": "linear", "pass": "grad", "T": 4001, "D": 2048, "V": 50257, "type": "bf16", "scale": 1.0, "ignored": 0.4},
        # an fp32 model (parity runs) at a temperature
        {"name": "linear grad fp32", "op": "linear", "pass": "grad", "T": 517, "D": 1000, "V": 10007, "type": "f32", "scale": 1.25, "ignored": 0.1},
        # the norm weights of a 32-layer model: many short vectors
        {"name": "clip 65 vectors", "op": "clip", "tensors": 65, "least": 4096, "most": 4096, "type": "bf16", "out": "bf16", "max": 0.1},
        # the matrices of four large layers and their experts' tensor
        {"name": "clip 5 matrices", "op": "clip", "tensors": 5, "least": 184549376, "most": 234881024, "type": "bf16", "out": "bf16", "max": 1.0},
    ]


LARGEST = {"tokens": 8192 * 128000 * 2, "linear": 4096 * 4096 * 32000, "clip": 4400000000}     # bytes, products, bytes


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size of [lo, hi], spread over its logarithm: a multiple of 64 or any."""
    n = _log(rng, lo, hi)
    return max(lo, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["tokens", "tokens", "linear", "clip"])
    f32 = rng.random() < 0.3
    case = {"op": op, "type": "f32" if f32 else "bf16"}
    if op == "clip":
        # equal tensors or sizes spread between two ends
        out = rng.choice(["bf16", "f32"])
        while True:
            n, most = _log(rng, 1, 600), _size(rng, 64, 1 << 28)
            if n * most * (_bytes(case["type"]) + _bytes(out)) <= LARGEST["clip"]:
                break
        least = most if rng.random() < 0.3 else max(1, most // _log(rng, 1, 10000))
        return {**case, "tensors": n, "least": least, "most": most, "out": out, "max": rng.choice([0.01, 1.0, 100.0])}
    case.update({"pass": rng.choice(["forward", "grad"]), "scale": rng.choice([1.0, 1.0, 0.5, 1.25]), "ignored": rng.choice([0.0, 0.1, 0.5, 0.9])})
    if op == "tokens":
        while True:
            T, V = _size(rng, 1, 8192), _size(rng, 100, 131072)
            if T * V >= 20000 and T * V * _bytes(case["type"]) * (2 if case["pass"] == "grad" else 1) <= LARGEST["tokens"]:
                break
        top = rng.choice([0, 1, 5, 20, 64]) if case["pass"] == "forward" else 0
        return {**case, "T": T, "V": V, "pad": rng.choice([0, 0, 1, -V % 64]), "top": top, "masked": rng.choice([0.0, 0.0, 0.5, 0.99])}
    while True:
        T, D, V = _size(rng, 1, 8192), _size(rng, 64, 4096), _size(rng, 1000, 131072)
        if T * V >= 100000 and T * D * V * (6 if f32 else 1) * (3 if case["pass"] == "grad" else 1) <= LARGEST["linear"]:
            break
    return {**case, "T": T, "D": D, "V": V}


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _bytes(name):
    return 4 if name == "f32" else 2


def _tokens(n, vocab, gen):
    """Token ids with natural frequencies (rank-frequency law), ranks scattered over the ids."""
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab + 1.0)).long() - 1
    step = 7919 if vocab % 7919 else 7927
    return torch.clamp(rank, 0, vocab - 1) * step % vocab


def _sizes(case):
    """Elements of each tensor, spread evenly over the logarithm between the two ends."""
    n, lo, hi = case["tensors"], math.log(case["least"]), math.log(case["most"])
    return [case["most"]] + [int(round(math.exp(hi - (hi - lo) * i / (n - 1)))) for i in range(1, n)]


def _places(case):
    """Where each tensor lies in a packed buffer, every one at a multiple of 64 elements, and the buffer's size."""
    return [0, *itertools.accumulate((n + 63) // 64 * 64 for n in _sizes(case))]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    normal = lambda *shape, type=None: torch.randn(*shape, generator=gen, device="cuda", dtype=type)
    uniform = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")
    op, t = case["op"], _dtype(case["type"])
    s = {"op": op}
    if op == "clip":
        s["grads"] = [normal(n, type=t).mul_(1e-3) for n in _sizes(case)]
        s["flat"] = torch.zeros(_places(case)[-1], device="cuda", dtype=_dtype(case["out"]))      # a packed buffer
        s["outs"] = [s["flat"][a:a + n] for a, n in zip(_places(case), _sizes(case))]
        s["max"] = case["max"]
        if own:
            import matrix_optimizer_muon_amd as mm
            s["clip"] = mm.ClipGradNorm(s["grads"], case["max"], outs=s["outs"], eps=EPS)
        return s
    T, V = case["T"], case["V"]
    s.update({"pass": case["pass"], "scale": case["scale"]})
    y = _tokens(T, V, gen)
    s["targets"] = torch.where(uniform(T) < case["ignored"], IGNORE, y)
    if op == "tokens":
        z = normal(T, V + case["pad"], type=t).mul_(2.5)
        z.scatter_add_(1, y[:, None], (uniform(T, 1) * 15).to(t))                 # a model that knows its tokens more or less
        if case["masked"]:
            for a in range(0, T, 1024):
                z[a:a + 1024].masked_fill_(uniform(*z[a:a + 1024].shape) < case["masked"], -math.inf)
            z.scatter_(1, y[:, None], 3.0)
        s["logits"] = z[:, :V]
        s["top"] = case["top"]
    else:
        D = case["D"]
        w = normal(V, D) * 0.02
        lean = uniform(T, 1) * 10 / (D * 4e-4)
        s["h"] = (normal(T, D) * min(1.0, 64 / math.sqrt(D)) + lean * w[y]).to(t)
        s["w"] = w.to(t)
    if case["pass"] == "grad":
        # advantages of either sign and a constant entropy bonus, as means over the tokens that count
        valid = s["targets"] != IGNORE
        n = valid.sum().clamp(min=1)
        s["grad_logprobs"] = normal(T) / n
        s["grad_entropy"] = torch.full((T,), -0.01, device="cuda") / n
        s["lse"], s["entropy"] = (torch.zeros(T, device="cuda") for _ in range(2))
        for a in range(0, T, 1024):
            x = (s["logits"][a:a + 1024].float() if op == "tokens" else s["h"][a:a + 1024].float() @ s["w"].float().T) * s["scale"]
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            s["lse"][a:a + 1024] = lse
            s["entropy"][a:a + 1024] = -torch.where(p > 0, p * (x - lse[:, None]), 0.0).sum(1)
        s["lse"], s["entropy"] = (torch.where(valid, v, 0.0) for v in (s["lse"], s["entropy"]))
    return s


def _run_own(s):
    import matrix_optimizer_muon_amd as mm
    if s["op"] == "clip":
        return s["clip"](), s["flat"]
    kw = {"scale": s["scale"], "ignore_index": IGNORE}
    if s["op"] == "tokens":
        if s["pass"] == "grad":
            return mm.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["entropy"], s["grad_logprobs"], s["grad_entropy"], **kw)
        r = mm.token_logprobs(s["logits"], s["targets"], top=s["top"], **kw)
        return (r.logprobs, r.entropy, r.lse) + ((r.top_ids, r.top_logprobs) if s["top"] else ())
    if s["pass"] == "grad":
        return mm.linear_token_logprobs_backward(s["h"], s["w"], s["targets"], s["lse"], s["entropy"], s["grad_logprobs"], s["grad_entropy"], **kw)
    r = mm.linear_token_logprobs(s["h"], s["w"], s["targets"], **kw)
    return r.logprobs, r.entropy, r.lse


def _top(z, k):
    """Places of the k largest of each row, ties to the lowest: one whole number per entry
    orders by value, then by place."""
    bits = (z + 0.0).view(torch.int32).long()                                     # −0 as 0
    order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
    key = (order << 32) + (z.shape[1] - 1 - torch.arange(z.shape[1], device=z.device))
    return z.shape[1] - 1 - (torch.topk(key, k, dim=1).values & 0xffffffff)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "clip":
        norm = torch.sqrt(sum((g.double() * g.double()).sum() for g in s["grads"])).float()
        coef = torch.clamp(s["max"] / (norm + EPS), max=1.0)
        for g, out in zip(s["grads"], s["outs"]):
            out.copy_(g.float() * coef)
        return norm, s["flat"]
    y = s["targets"]
    valid = y != IGNORE
    at = torch.where(valid, y, 0)[:, None]
    if s["op"] == "tokens":
        z = s["logits"].float()
    else:
        h, w = s["h"].float(), s["w"].float()
        z = h @ w.T
    x = z * s["scale"]
    if s["pass"] == "grad":
        log_p = x - s["lse"][:, None]
        p = torch.exp(log_p)
        d = p * torch.where(p > 0, log_p + s["entropy"][:, None], 0.0) * -s["grad_entropy"][:, None] - p * s["grad_logprobs"][:, None]
        d.scatter_add_(1, at, s["grad_logprobs"][:, None])
        d = torch.where(valid[:, None], d * s["scale"], 0.0)
        return d.to(s["logits"].dtype) if s["op"] == "tokens" else ((d @ w).to(s["h"].dtype), (d.T @ h).to(s["w"].dtype))
    most = x.amax(1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(1)
    lse = most[:, 0] + torch.log(total)
    entropy = torch.log(total) - torch.where(e > 0, e * (x - most), 0.0).sum(1) / total
    out = [x.gather(1, at)[:, 0] - lse, entropy, lse]
    out = [torch.where(valid, v, 0.0) for v in out]
    if s["op"] == "tokens" and s["top"]:
        ids = _top(z, s["top"])
        out += [torch.where(valid[:, None], ids, -1), torch.where(valid[:, None], x.gather(1, ids) - lse[:, None], 0.0)]
    return tuple(out)


def work(case):
    b = _bytes(case["type"])
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": n * (b + _bytes(case["out"])), "flops": 3 * n}
    T, V = case["T"], case["V"]
    n = T * (1 - case["ignored"])                                                  # rows that take part
    if case["op"] == "tokens":
        if case["pass"] == "grad":
            return {"bytes": (n + T) * V * b + T * 24, "flops": 8 * n * V}
        return {"bytes": n * V * b + T * (20 + 12 * case["top"]), "flops": 7 * n * V}
    D = case["D"]
    if case["pass"] == "grad":
        return {"bytes": (n + V + T + V) * D * b + T * 24, "flops": 6 * n * D * V}
    return {"bytes": (n + V) * D * b + T * 20, "flops": 2 * n * D * V}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]]))
        flat = torch.zeros(_places(case)[-1], device="cuda", dtype=torch.float64)
        for a, g in zip(_places(case), s["grads"]):
            flat[a:a + len(g)] = g.double() * min(1.0, s["max"] / (norm.item() + EPS))
        return norm, flat
    keep = torch.nonzero(s["targets"] != IGNORE)[:, 0]
    T, linear, grad = len(s["targets"]), s["op"] == "linear", s["pass"] == "grad"
    real = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")
    if linear:
        w = s["w"].double()
    if grad:
        dz = None if linear else real(T, case["V"])
        dh, dw = (real(T, case["D"]), torch.zeros_like(w)) if linear else (None, None)
    else:
        top = s.get("top", 0)
        logprobs, entropy, lse = real(T), real(T), real(T)
        ids, best = torch.full((T, top), -1, device="cuda"), real(T, top)
    for i in range(0, len(keep), 512):
        r = keep[i:i + 512]
        mine = torch.arange(len(r), device="cuda")
        z = torch.mm(s["h"][r].double(), w.T) if linear else s["logits"][r].double()
        y = s["targets"][r]
        if grad:
            log_p = (z * s["scale"]).sub_(s["lse"][r].double()[:, None])
            p = log_p.exp()
            g, ge = s["grad_logprobs"][r].double()[:, None], s["grad_entropy"][r].double()[:, None]
            d = -p * g - ge * (torch.special.xlogy(p, p) + p * s["entropy"][r].double()[:, None])
            d[mine, y] += g[:, 0]
            d *= s["scale"]
            if linear:
                dh[r] = torch.mm(d, w)
                dw.addmm_(d.T, s["h"][r].double())
            else:
                dz[r] = d
            continue
        log_p = torch.log_softmax(z * s["scale"], 1)
        p = log_p.exp()
        logprobs[r] = log_p[mine, y]
        entropy[r] = torch.special.entr(p).sum(1)
        lse[r] = torch.logsumexp(z * s["scale"], 1)
        if top:
            order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]
            ids[r] = order
            best[r] = log_p.gather(1, order)
    if grad:
        return (dh, dw) if linear else dz
    return (logprobs, entropy, lse) + ((ids, best) if top else ())
