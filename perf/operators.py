"""The cases by which the training-gradient operators are measured.

Three operators produce the gradients that the optimizer routes consume:

* ``ce``: softmax cross entropy of hidden states against a large vocabulary
  (``linear_cross_entropy`` and its backward pass; the head's gradient);
* ``embed``: embedding lookup with a scale and its gradient (``embedding``,
  ``embedding_backward``; the table's gradient);
* ``ckpt``: activation checkpoints in 8 bits and the weight gradient computed
  from them (``checkpoint_quantize`` / ``checkpoint_dequantize`` /
  ``checkpoint_wgrad``; the gradients of the Muon matrices).

``run`` computes a case in its plain form (elementary torch operations in fp32)
or, where ``own`` is true, through the package.
"""
import math

import numpy as np
import torch

own = False

IGNORE = -100
BLOCK = 32                       # columns that share one exponent of a checkpoint


def listed():
    return [
        # scoring a few positions of a short prompt against a 32k vocabulary: W is read once
        {"name": "ce loss 16 tokens", "op": "ce", "pass": "loss", "T": 16, "D": 2048, "V": 32000, "type": "bf16", "ignored": 0.0, "weights": False},
        # evaluation of a batch: losses only
        {"name": "ce loss 4096 tokens", "op": "ce", "pass": "loss", "T": 4096, "D": 4096, "V": 32000, "type": "bf16", "ignored": 0.0, "weights": False},
        # a fine-tuning batch with prompts masked out, an odd vocabulary, per-token weights
        {"name": "ce grad masked", "op": "ce", "pass": "grad", "T": 4001, "D": 2048, "V": 50257, "type": "bf16", "ignored": 0.4, "weights": True},
        # a pre-training micro-batch of a d = 4096 model with a large vocabulary
        {"name": "ce grad large", "op": "ce", "pass": "grad", "T": 8192, "D": 4096, "V": 128000, "type": "bf16", "ignored": 0.0, "weights": False},
        # an fp32 model (parity runs), nothing a multiple of anything
        {"name": "ce grad fp32", "op": "ce", "pass": "grad", "T": 517, "D": 1000, "V": 10007, "type": "f32", "ignored": 0.1, "weights": False},
        # the lookup of one decoding step
        {"name": "embed lookup 32 tokens", "op": "embed", "pass": "lookup", "T": 32, "D": 4096, "V": 32000, "type": "bf16", "out": "bf16"},
        # the lookup of a training micro-batch
        {"name": "embed lookup 32768 tokens", "op": "embed", "pass": "lookup", "T": 32768, "D": 4096, "V": 128000, "type": "bf16", "out": "bf16"},
        # the table's gradient in the step's layout (bf16), natural token frequencies
        {"name": "embed grad", "op": "embed", "pass": "grad", "T": 8192, "D": 2048, "V": 32000, "type": "bf16", "out": "bf16"},
        # an fp32 gradient of a large table
        {"name": "embed grad large", "op": "embed", "pass": "grad", "T": 32768, "D": 4096, "V": 128000, "type": "bf16", "out": "f32"},
        # the down projection's input of a d = 4096 layer, stored and read back
        {"name": "ckpt store and read", "op": "ckpt", "pass": "round trip", "T": 8192, "K": 11008, "type": "bf16"},
        # the weight gradient of that projection
        {"name": "ckpt weight grad", "op": "ckpt", "pass": "wgrad", "T": 8192, "N": 4096, "K": 11008, "E": 1, "type": "bf16", "out": "bf16"},
        # 64 experts' weight gradients of a routed batch, ragged, in fp32
        {"name": "ckpt expert grads", "op": "ckpt", "pass": "wgrad", "T": 16001, "N": 1408, "K": 2048, "E": 64, "type": "bf16", "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size of [lo, hi], spread over its logarithm: a multiple of 64 or any."""
    n = _log(rng, lo, hi)
    return max(lo, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["ce", "ce", "embed", "ckpt"])
    f32 = rng.random() < 0.2
    if op == "ce":
        while True:
            T, D, V = _size(rng, 1, 8192), _size(rng, 64, 4096), _size(rng, 1000, 131072)
            if T * D * V * (6 if f32 else 1) <= 8192 * 4096 * 128000 and (T * V >= 100000):
                break
        return {"op": "ce", "pass": rng.choice(["loss", "grad"]), "T": T, "D": D, "V": V, "type": "f32" if f32 else "bf16",
                "ignored": rng.choice([0.0, 0.1, 0.5, 0.9]), "weights": rng.random() < 0.3}
    if op == "embed":
        return {"op": "embed", "pass": rng.choice(["lookup", "grad"]), "T": _size(rng, 1, 32768), "D": _size(rng, 64, 8192), "V": _size(rng, 1000, 131072),
                "type": "f32" if f32 else "bf16", "out": rng.choice(["bf16", "f32"])}
    if rng.random() < 0.4:
        return {"op": "ckpt", "pass": "round trip", "T": _size(rng, 1, 16384), "K": _size(rng, 64, 16384), "type": "f32" if f32 else "bf16"}
    return {"op": "ckpt", "pass": "wgrad", "T": _size(rng, 1, 16384), "N": _size(rng, 64, 4096), "K": _size(rng, 64, 8192),
            "E": rng.choice([1, 1, 8]), "type": "f32" if f32 else "bf16", "out": "f32" if f32 else rng.choice(["bf16", "f32"])}


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


def _routed(case, seed):
    """Offsets of the experts' rows: uneven, some of them empty."""
    rng = np.random.default_rng([seed, 5])
    T, E = case["T"], case["E"]
    share = rng.exponential(1.0, E) * (rng.random(E) > 0.05)
    share[rng.integers(E)] += 0.1
    at = np.floor(np.cumsum(share) / share.sum() * T + 0.5).astype(np.int64)
    at[-1] = T
    return np.concatenate([[0], at]).astype(np.int32)


def _power(b):
    """2^(b − 133) of whole numbers b, exactly (b is at least 7 wherever the value is used)."""
    return (torch.clamp(b.to(torch.int32) - 6, 1, 254) << 23).view(torch.float32)


def _encode(x):
    """q (whole numbers in 8 bits) and biased exponents b of an fp32 matrix: x is about q·2^(b − 133), b shared by 32 columns of a row."""
    T, K = x.shape
    blocks = -(-K // BLOCK)
    x = torch.nn.functional.pad(x, (0, blocks * BLOCK - K)).view(T, blocks, BLOCK)
    most = x.abs().amax(2)
    b = torch.frexp(most)[1] + 126                                      # the biased exponent of the largest
    b = torch.clamp(b + (most * _power(266 - b) >= 127.5), max=254)     # rounding may need one more
    b = torch.where(most < 2.0 ** -120, 0, b)                           # no input here is as small as that
    q = torch.clamp(torch.round(x * _power(266 - b)[..., None]), -127, 127)
    q = torch.where((b > 0)[..., None], q, 0.0)
    return q.view(T, blocks * BLOCK)[:, :K].to(torch.int8).contiguous(), b.to(torch.uint8).contiguous()


def _decode(q, exps):
    return q.float() * _power(exps).repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    op, T = case["op"], case["T"]
    t = _dtype(case["type"])
    s = {"op": op, "pass": case["pass"]}
    if op == "ce":
        D, V = case["D"], case["V"]
        w = normal(V, D) * 0.02
        y = _tokens(T, V, gen)
        lean = torch.rand(T, 1, generator=gen, device="cuda") * 10 / (D * 4e-4)   # a model that knows its targets more or less
        s["h"] = (normal(T, D) * min(1.0, 64 / math.sqrt(D)) + lean * w[y]).to(t)
        s["w"] = w.to(t)
        s["targets"] = torch.where(torch.rand(T, generator=gen, device="cuda") < case["ignored"], IGNORE, y)
        if case["pass"] == "grad":
            valid = s["targets"] != IGNORE
            weight = torch.rand(T, generator=gen, device="cuda") if case["weights"] else torch.ones(T, device="cuda")
            s["grad_losses"] = weight / valid.sum().clamp(min=1)
            s["lse"] = torch.where(valid, torch.logsumexp(s["h"].float() @ s["w"].float().T, 1), 0.0)
    elif op == "embed":
        D, V = case["D"], case["V"]
        s.update(rows=V, scale=math.sqrt(D), out=_dtype(case["out"]), ids=_tokens(T, V, gen))
        if case["pass"] == "lookup":
            s["table"] = (normal(V, D) * 0.02).to(t)
        else:
            s["grad_out"] = (normal(T, D) * 1e-3).to(t)
    else:
        x = normal(T, case["K"]) * torch.exp(normal(1, case["K"]))       # channels of unequal size, as activations have
        x[:, ::2] = x[:, ::2].abs()
        x = x.to(t)
        if case["pass"] == "round trip":
            s.update(x=x, type=t)
        else:
            s["q"], s["exps"] = _encode(x.float())
            s["grad_out"] = (normal(T, case["N"]) * 1e-3).to(t)
            s["out"] = _dtype(case["out"])
            s["offsets"] = None
            if case["E"] > 1:
                at = _routed(case, seed)
                s["offsets"] = torch.from_numpy(at).cuda()
                s["most"] = int(np.diff(at).max())
    return s


def _run_own(s):
    import matrix_optimizer_muon_amd as mm
    if s["op"] == "ce":
        if s["pass"] == "loss":
            return mm.linear_cross_entropy(s["h"], s["w"], s["targets"], ignore_index=IGNORE)
        return mm.linear_cross_entropy_backward(s["h"], s["w"], s["targets"], s["lse"], s["grad_losses"], ignore_index=IGNORE)
    if s["op"] == "embed":
        if s["pass"] == "lookup":
            return mm.embedding(s["ids"], s["table"], scale=s["scale"])
        return mm.embedding_backward(s["ids"], s["grad_out"], s["rows"], scale=s["scale"], out_dtype=s["out"])
    if s["pass"] == "round trip":
        q, exps = mm.checkpoint_quantize(s["x"])
        return mm.checkpoint_dequantize(q, exps, dtype=s["type"])
    return mm.checkpoint_wgrad(s["grad_out"], s["q"], s["exps"], offsets=s["offsets"], out_dtype=s["out"])


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "ce":
        y = s["targets"]
        valid = y != IGNORE
        at = torch.where(valid, y, 0)[:, None]
        h, w = s["h"].float(), s["w"].float()
        z = h @ w.T
        if s["pass"] == "loss":
            most = z.amax(1)
            lse = most + torch.log(torch.exp(z - most[:, None]).sum(1))
            return torch.where(valid, lse - z.gather(1, at)[:, 0], 0.0), torch.where(valid, lse, 0.0)
        p = torch.exp(z - s["lse"][:, None])
        p.scatter_add_(1, at, torch.full_like(at, -1, dtype=p.dtype))
        p *= torch.where(valid, s["grad_losses"], 0.0)[:, None]
        return (p @ w).to(s["h"].dtype), (p.T @ h).to(s["w"].dtype)
    if s["op"] == "embed":
        if s["pass"] == "lookup":
            return (s["table"][s["ids"]].float() * s["scale"]).to(s["table"].dtype)
        g = s["grad_out"].float()
        return (torch.zeros(s["rows"], g.shape[1], device=g.device).index_add_(0, s["ids"], g) * s["scale"]).to(s["out"])
    if s["pass"] == "round trip":
        return _decode(*_encode(s["x"].float())).to(s["type"])
    x, g = _decode(s["q"], s["exps"]), s["grad_out"].float()
    if s["offsets"] is None:
        return (g.T @ x).to(s["out"])
    at = s["offsets"].long()
    k = at[:-1, None] + torch.arange(s["most"], device=x.device)[None]
    mine = (k < at[1:, None])[..., None]
    k = torch.clamp(k, max=x.shape[0] - 1)
    gt = torch.where(mine, g[k], 0.0).transpose(1, 2).contiguous()
    return torch.bmm(gt, torch.where(mine, x[k], 0.0)).to(s["out"])


def work(case):
    T, b = case["T"], _bytes(case["type"])
    if case["op"] == "ce":
        D, V = case["D"], case["V"]
        n = T * (1 - case["ignored"])                                    # rows that have a loss
        if case["pass"] == "loss":
            return {"bytes": (n + V) * D * b + T * 16, "flops": 2 * n * D * V}
        # the logits again (they are not kept), and two products with their gradient
        return {"bytes": (n + V + T + V) * D * b + T * 16, "flops": 6 * n * D * V}
    if case["op"] == "embed":
        D, V = case["D"], case["V"]
        if case["pass"] == "lookup":
            return {"bytes": min(T, V) * D * b + T * D * b + T * 8, "flops": T * D}
        return {"bytes": T * D * b + V * D * _bytes(case["out"]) + T * 8, "flops": T * D}
    K = case["K"]
    held = T * K + T * -(-K // BLOCK)                                    # a checkpoint's bytes
    if case["pass"] == "round trip":
        return {"bytes": 2 * T * K * b + 2 * held, "flops": 4 * T * K}
    N = case["N"]
    return {"bytes": T * N * b + held + case["E"] * N * K * _bytes(case["out"]), "flops": 2 * T * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "ce":
        keep = torch.nonzero(s["targets"] != IGNORE)[:, 0]
        y = s["targets"][keep]
        T = s["h"].shape[0]
        h, w = s["h"][keep].double(), s["w"].double()
        if s["pass"] == "loss":
            loss, lse = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(2))
            for i in range(0, len(keep), 1024):
                z = torch.mm(h[i:i + 1024], w.T)
                lse[keep[i:i + 1024]] = torch.logsumexp(z, 1)
                loss[keep[i:i + 1024]] = torch.nn.functional.cross_entropy(z, y[i:i + 1024], reduction="none")
            return loss, lse
        g = s["grad_losses"][keep].double()
        lse = s["lse"][keep].double()
        dh, dw = torch.zeros(T, h.shape[1], dtype=torch.float64, device="cuda"), torch.zeros_like(w)
        for i in range(0, len(keep), 1024):
            j = slice(i, i + 1024)
            d = (torch.mm(h[j], w.T) - lse[j, None]).exp_()
            d[torch.arange(d.shape[0], device="cuda"), y[j]] -= 1
            d.mul_(g[j, None])
            dh[keep[j]] = torch.mm(d, w)
            dw.addmm_(d.T, h[j])
        return dh, dw
    if s["op"] == "embed":
        if s["pass"] == "lookup":
            return s["table"].double().index_select(0, s["ids"]) * s["scale"]
        order = torch.argsort(s["ids"], stable=True)                     # sorted tokens, sums by differences of running sums
        ids, g = s["ids"][order], s["grad_out"].double()[order] * s["scale"]
        out = torch.zeros(s["rows"], g.shape[1], dtype=torch.float64, device="cuda")
        run_ = torch.cumsum(g, 0)
        last = torch.cat([ids[1:] != ids[:-1], torch.ones(1, dtype=torch.bool, device="cuda")])
        ends = run_[last]
        out[ids[last]] = ends - torch.cat([torch.zeros_like(ends[:1]), ends[:-1]])
        return out
    if s["pass"] == "round trip":
        x = s["x"].double()
        out = torch.zeros_like(x)
        for c in range(0, x.shape[1], BLOCK):                            # each block: the least power of two that keeps 7 bits and a sign
            part = x[:, c:c + BLOCK]
            most = part.abs().amax(1, keepdim=True)
            unit = torch.full_like(most, 2.0 ** -130)
            while bool((most >= 127.5 * unit).any()):
                unit = torch.where(most >= 127.5 * unit, unit * 2, unit)
            out[:, c:c + BLOCK] = torch.round(part / unit) * unit
        return out
    e = np.arange(s["q"].shape[1]) // BLOCK
    x = s["q"].double() * torch.pow(2.0, s["exps"].double() - 133)[:, torch.from_numpy(e).cuda()]
    g = s["grad_out"].double()
    if s["offsets"] is None:
        return torch.mm(g.T, x)
    at = s["offsets"].tolist()
    return torch.stack([torch.mm(g[a:b].T, x[a:b]) for a, b in zip(at, at[1:])])
