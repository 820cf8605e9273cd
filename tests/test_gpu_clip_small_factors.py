"""Clipping of gradients near fp32's end to a small norm: the factor lies below fp32's normal
numbers (needs an MI355X).  Bounds as in test_gpu_clip."""
import pytest
import torch
from test_gpu_clip import BF, F32, check, mm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bf16", "bf16-f32", "f32", "f32-bf16"])
@pytest.mark.parametrize("max_norm", [1e9, 1.0, 1e-2, 1e-5, 1e-10, 1e-20, 1e-37])
@pytest.mark.parametrize("size", [1e30, 3e36, 3e37])
def test_small_factors(types, max_norm, size):
    g = torch.Generator(device="cuda").manual_seed(9)
    grads = [(torch.randn(n, generator=g, device="cuda").clamp(-3, 3) * size / 3 / n ** 0.5 * 2).to(types[0]) for n in (1, 7, 5003, 40000)]
    grads[0].fill_(size)
    before = [x.clone() for x in grads]
    outs = [torch.empty_like(x, dtype=types[1]) for x in grads]
    norm = mm().clip_grad_norm(grads, max_norm, outs=outs, eps=0.0)
    assert torch.isfinite(norm)
    check(grads, outs, before, norm, max_norm, eps=0.0)
    if types[0] == types[1]:
        mm().clip_grad_norm(grads, max_norm, eps=0.0)
        check(grads, grads, before, norm, max_norm, eps=0.0)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_given_norm(dtype):
    """Of several owners: their common norm may be far above these gradients."""
    norm = torch.tensor(3e38, device="cuda")
    for max_norm in (1.0, 1e-3, 1e-6):
        x = torch.tensor([1e30, -3e37, 1e10, 0.0], device="cuda").to(dtype)
        ref = x.double() * (torch.tensor(max_norm).double() / norm.double().cpu()).item()
        mm().clip_grad_norm([x], max_norm, norm=norm, eps=0.0)
        u = 2.0 ** -8 if dtype == BF else 2.0 ** -24
        tol = (4 * 2.0 ** -24 * ref.abs()) * (1 + u) + u * ref.abs() + (2.0 ** -133 if dtype == BF else 2.0 ** -149)
        assert ((x.double() - ref).abs() <= tol).all()
