"""Infinities in the operands of the training products, the same in bf16 and fp32: an
infinity times a finite number other than 0 is the infinity (needs an MI355X)."""
import math

import pytest
import torch

from test_gpu_training import ce_inputs, ce_reference, ckpt_values, gen, mm, randn, within

pytestmark = pytest.mark.gpu

SIZES = [(16, 64, 500, torch.bfloat16), (16, 64, 500, torch.float32), (40, 70, 300, torch.float32),
         (100, 70, 900, torch.bfloat16), (100, 70, 900, torch.float32),
         (2001, 800, 6500, torch.bfloat16), (2001, 136, 6500, torch.float32)]


@pytest.mark.parametrize("T,D,V,dtype", SIZES)
def test_vocabulary_rows_of_minus_infinity(T, D, V, dtype):
    """Words masked out through a column of −inf: their logits are −inf, and the losses
    and the other words' gradients those of the vocabulary without them."""
    m = mm()
    h, w, y, gl = ce_inputs(T, D, V, dtype, 80 + T, ignored=0.0)
    h[:, D - 1] = torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, 1.37)      # a factor of one plane, and of more
    w[:, D - 1] = 0
    last = V - V // 3                                          # the words from here on are out
    w[last:, D - 1] = -math.inf
    y = y % last
    ref = ce_reference(h, w[:last], y, gl)
    losses, lse = m.linear_cross_entropy(h, w, y)
    within(losses, ref["loss"], ref["tol"], "loss")
    within(lse, ref["lse"], ref["tol"], "lse")
    ref = ce_reference(h, w[:last], y, gl, lse)
    _, dw = m.linear_cross_entropy_backward(h, w, y, lse, gl, need_h=False)
    assert not dw[last:].any()
    within(dw[:last], ref["dw"], ref["tol_w"], "dw")
    # a target among them: a loss of +inf, its lse as ever
    y[3] = last
    more, same = m.linear_cross_entropy(h, w, y)
    keep = torch.arange(T, device="cuda") != 3
    assert more[3] == math.inf and torch.equal(more[keep], losses[keep]) and torch.equal(same, lse)


@pytest.mark.parametrize("T,D,V,dtype", SIZES)
def test_infinite_hidden_states_stay_in_their_token(T, D, V, dtype):
    m = mm()
    h, w, y, _ = ce_inputs(T, D, V, dtype, 90 + T, ignored=0.0)
    w[:, 0] = w[:, 0].abs() + 0.25
    ref = m.linear_cross_entropy(h, w, y)
    h[3, 0], h[5, 0], h[7, 0] = -math.inf, math.inf, math.nan
    losses, lse = m.linear_cross_entropy(h, w, y)
    assert lse[3] == -math.inf and math.isnan(losses[3])       # every logit −inf
    for t in (5, 7):                                           # logits of +inf and NaN have no softmax
        assert math.isnan(lse[t]) and math.isnan(losses[t])
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[3, 5, 7]] = False
    assert torch.equal(losses[keep], ref[0][keep]) and torch.equal(lse[keep], ref[1][keep])


@pytest.mark.parametrize("T,N,K", [(100, 40, 72), (3001, 1500, 1700)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_infinite_output_gradients(T, N, K, dtype):
    """An infinite entry of grad_out makes its weight row ±inf by the signs of the kept
    row (NaN where that is 0) and touches no other."""
    m = mm()
    g = gen(T)
    x, grad = randn(g, T, K), randn(g, T, N).to(dtype)
    q, b = m.checkpoint_quantize(x)
    ref = m.checkpoint_wgrad(grad, q, b, out_dtype=torch.float32)
    grad[17, 5], grad[18, 6] = math.inf, -math.inf
    got = m.checkpoint_wgrad(grad, q, b, out_dtype=torch.float32)
    v = ckpt_values(q, b)
    for n, t, sign in ((5, 17, 1), (6, 18, -1)):
        want = torch.where(v[t] == 0, math.nan, sign * torch.sign(v[t]) * math.inf)
        assert torch.equal(torch.nan_to_num(got[n].double(), nan=7.0, posinf=1.0, neginf=-1.0),
                           torch.nan_to_num(want, nan=7.0, posinf=1.0, neginf=-1.0))
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[[5, 6]] = False
    assert torch.equal(got[keep], ref[keep])
