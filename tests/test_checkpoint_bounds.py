"""How far an 8-bit checkpoint may be from its values: half a step 2^(b − 134) (a step where
q saturates, b = 254), at most 1/127.5 of the block's largest, blocks below 2^-126 zero.
The format's arithmetic on the CPU; the kernels against the same bounds on the GPU."""
import math

import pytest
import torch


def blocks(seed, device):
    """One block of 32 per row: magnitudes over the whole range, and the borders where a
    largest value rounds up to the next exponent or saturates."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(4000, 32, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-124, 124, (4000, 1), generator=g).double())
    edge = []
    for e in (-126, -125, -60, 0, 3, 100, 126, 127):
        for m in (1.0, 1.5, 127.49 / 64, 127.5 / 64, 127.51 / 64, 2 - 2.0 ** -23):
            # the largest, values half a step off a whole q, and some below
            row = torch.rand(32, generator=g, dtype=torch.float64) * 2 - 1
            row[0], row[1], row[2] = m, m * 63.5 / 127, -m
            row[3:8] = (torch.arange(5) + 0.5) / 64
            edge.append(row * 2.0 ** e)
    x = torch.cat([x, torch.stack(edge)])
    return x.clamp(-torch.finfo(torch.float32).max, torch.finfo(torch.float32).max).float().to(device)


def check_bounds(x, q, b):
    from test_gpu_training import ckpt_values, p2
    v, xd = ckpt_values(q, b), x.double()
    most = xd.abs().amax(1, keepdim=True)
    step = p2(b.int() - 133)
    err = (v - xd).abs()
    zero = b == 0
    assert (most[zero] < 2.0 ** -126).all() and not v[zero.expand_as(v)].any()
    held = ~zero.expand_as(v)
    saturated = (b == 254) & (xd.abs() >= 127.5 * step)
    assert (err <= torch.where(saturated, step, step / 2))[held].all()
    assert (err * 127.5 <= most)[held].all()
    return err / most.clamp(min=1e-300), err / step, held, saturated


def test_the_formats_arithmetic():
    from test_gpu_training import ckpt_reference
    x = blocks(1, "cpu")
    q, b = ckpt_reference(x)
    assert q.min() >= -127 and q.max() == 127 and (b.int() <= 254).all()
    rel, steps, held, saturated = check_bounds(x, q, b)
    # both bounds are nearly reached, and neither holds with 2^-7 or half a step alone
    assert rel[held].max() > 2.0 ** -7 and steps[held & ~saturated].max() > 0.499
    assert saturated.any() and steps[saturated].max() > 0.9
    # q·2^(b − 133) is a bf16 value
    from test_gpu_training import ckpt_values
    v = ckpt_values(q, b)
    assert torch.equal(v.to(torch.bfloat16).double(), v)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_stored_values_are_within_the_bounds(dtype):
    import matrix_optimizer_muon_amd as mm
    from test_gpu_training import ckpt_reference
    x = blocks(2, "cuda")
    if dtype == torch.bfloat16:                     # cut off, so that nothing becomes infinite
        x = (x.view(torch.int32) & -65536).view(torch.float32)
    x = x.to(dtype)
    q, b = mm.checkpoint_quantize(x)
    rq, rb = ckpt_reference(x)
    assert torch.equal(q, rq) and torch.equal(b, rb)
    check_bounds(x, q, b)
    assert math.isfinite(mm.checkpoint_dequantize(q, b).float().abs().max())
