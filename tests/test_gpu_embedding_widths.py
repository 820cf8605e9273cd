"""The embedding table's gradient at the widths of real models: several slabs of 512
columns, 16 to 256 table rows per clearing workgroup, long runs of one id beside rare ones
and a padding id (needs an MI355X)."""
import pytest
import torch

from test_gpu_training import U, embed_reference, gen, mm, randn, within

pytestmark = pytest.mark.gpu


def ids_with_runs(T, V, pad, seed):
    """A third of the tokens hold one id, an eighth the padding id, a few hundred a
    second frequent one; some lie outside the table, the rest anywhere."""
    g = gen(seed)
    ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    u = torch.rand(T, generator=g, device="cuda")
    ids = torch.where(u < 0.33, V // 2, ids)
    ids = torch.where((u > 0.4) & (u < 0.52), pad, ids)
    return torch.where((u > 0.6) & (u < 0.65), V - 1, ids)


@pytest.mark.parametrize("gdt,odt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                     (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,V,D", [(100, 40, 520), (5000, 300, 520), (8192, 1000, 513), (3000, 100, 1023), (9000, 500, 2048),
                                   (9000, 2000, 4096), (33, 50, 4104), (70001, 700, 1030), (2000, 100, 16400)])
def test_wide_rows(T, V, D, gdt, odt):
    m = mm()
    pad = 7
    ids = ids_with_runs(T, V, pad, T + D)
    grad = randn(gen(D), T, D).to(gdt)
    for padding in (pad, None):
        want, tol = embed_reference(ids, grad, V, 1.3, padding, odt)
        got = m.embedding_backward(ids, grad, V, scale=1.3, padding_id=padding, out_dtype=odt)
        within(got, want, tol, f"padding {padding}")
        assert torch.equal(m.embedding_backward(ids, grad, V, scale=1.3, padding_id=padding, out_dtype=odt), got)
    # added to what is there: rows without tokens, and the padding's, as they were
    held = randn(gen(1), V, D).to(odt)
    out = held.clone()
    m.embedding_backward(ids, grad, V, scale=1.3, padding_id=pad, out=out, accumulate=True)
    want, _ = embed_reference(ids, grad, V, 1.3, pad, odt)
    _, tol = embed_reference(ids, grad, V, 1.3, pad, torch.float32)
    total = held.double() + want
    within(out, total, tol + (U[odt] + 2.0 ** -24) * (total.abs() + tol), "sum")
    assert torch.equal(out[pad], held[pad])


@pytest.mark.parametrize("off", [0, 3, 8])
def test_wide_strided_rows(off):
    """Rows of a larger buffer, on and off the 16-byte grid: the bits of dense ones; the
    gradient into a view between other values, which stay."""
    m = mm()
    T, V, D = 4000, 200, 1032
    ids = ids_with_runs(T, V, 7, 9)
    big = randn(gen(10), T, D + 16).to(torch.bfloat16)
    view = big[:, off:off + D]
    want = m.embedding_backward(ids, view.contiguous(), V, padding_id=7)
    assert torch.equal(m.embedding_backward(ids, view, V, padding_id=7), want)
    room = torch.full((V * D + 16,), 5.0, device="cuda", dtype=torch.bfloat16)
    out = room[off:off + V * D].view(V, D)
    assert torch.equal(m.embedding_backward(ids, view, V, padding_id=7, out=out), want)
    assert (room[:off] == 5).all() and (room[off + V * D:] == 5).all()
