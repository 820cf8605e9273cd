"""The global gradient norm and clipping against fp64 (needs an MI355X).

Tolerances: a square of an fp32 value is exact in 64 bits and the sum of N of them off by
N·2^-53 of itself at most, so the norm is its rounding to fp32 (2^-24; 2^-23 allows for a
neighbour across a tie).  The factor c is rounded to fp32 from an fp32 norm (2·2^-24), the
product to fp32 (2^-24) and to the output's type."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-6


def mm():
    import matrix_optimizer_muon_amd
    return matrix_optimizer_muon_amd


def grads_of(sizes, types, seed=1, scale=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def norm64(grads):
    return sum((g.double() ** 2).sum() for g in grads).sqrt()


def check(grads, outs, before, norm, max_norm, eps=EPS):
    """outs against c·before with the true norm."""
    want = norm64(before)
    assert abs(norm.double() - want) <= 2.0 ** -23 * want
    c = min(1.0, max_norm / (want.item() + eps)) if want > 0 or eps > 0 else 1.0
    for i, (b, o) in enumerate(zip(before, outs)):
        ref = b.double() * c
        tol = (4 * 2.0 ** -24 * ref.abs()) * (1 + U[o.dtype]) + U[o.dtype] * ref.abs() + (2.0 ** -133 if o.dtype == BF else 2.0 ** -149)
        assert ((o.double() - ref).abs() <= tol).all(), f"tensor {i}"


SETS = [[1], [7], [8], [2047], [2048], [2049], [5, 1, 100003, 64], [1 << 20, 3, (1 << 20) + 5], [1] * 70 + [4096] * 65, list(range(1, 700)),
        [0, 5, 0], [6_000_001, 12_345_678, 9]]


@pytest.mark.parametrize("types", [[BF], [F32], [BF, F32]], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_sizes(sizes, types):
    m = mm()
    grads = grads_of(sizes, types)
    before = [g.clone() for g in grads]
    want = norm64(before).item()
    norm = m.grad_norm(grads)
    assert norm.shape == () and norm.dtype == F32
    for max_norm in (want / 3, want * 2):
        for kinds in ([BF], [F32], [F32, BF]):
            outs = [torch.full(g.shape, 7.0, device="cuda", dtype=kinds[i % len(kinds)]) for i, g in enumerate(grads)]
            n = m.clip_grad_norm(grads, max_norm, outs=outs)
            assert torch.equal(n, norm)
            check(grads, outs, before, n, max_norm)
            for g, b in zip(grads, before):
                assert torch.equal(g, b)
    clip = m.ClipGradNorm(grads, want * 2)
    assert torch.equal(clip(), norm)
    for g, b in zip(grads, before):
        assert torch.equal(g, b)
    clip.max_norm = want / 3
    n = clip().clone()
    assert torch.equal(n, norm)
    check(grads, grads, before, n, want / 3)
    again = clip()                          # of the clipped gradients
    assert abs(again.item() - want / 3) <= 2.0 ** -7 * want / 3


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_magnitudes(dtype):
    """Squares beyond fp32 on either side, and a sum that fp32 could not hold."""
    m = mm()
    for value in (1e-30, 1e-38, 1e20, 1e37):
        g = [torch.full((1000,), value, device="cuda").to(dtype), torch.full((24,), -value, device="cuda").to(dtype)]
        before = [x.clone() for x in g]
        want = norm64(g)
        norm = m.clip_grad_norm(g, want.item() / 2, eps=0.0)
        check(g, g, before, norm, want.item() / 2, eps=0.0)
    big = torch.full((1 << 24,), 1.0, device="cuda", dtype=dtype)
    one = torch.full((1,), 2.0, device="cuda", dtype=dtype)
    assert m.grad_norm([big, one]).item() == torch.tensor((2.0 ** 24 + 4) ** 0.5).item()
    zero = torch.zeros(100, device="cuda", dtype=dtype)
    for eps in (0.0, 1e-6):
        assert m.clip_grad_norm([zero], 1.0, eps=eps).item() == 0 and not zero.any()
    g = grads_of([1000], [dtype])
    m.clip_grad_norm(g, 0.0)
    assert not g[0].any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_not_finite(value, dtype):
    m = mm()
    g = grads_of([5000, 77], [dtype])
    g[1][3] = value
    before = [x.clone() for x in g]
    outs = [torch.zeros_like(x, dtype=F32) for x in g]
    norm = m.clip_grad_norm(g, 1e-3, outs=outs)
    assert not torch.isfinite(norm) and torch.isnan(norm) == (value != value)
    for o, b in zip(outs, before):
        assert torch.equal(torch.nan_to_num(o, 9.0), torch.nan_to_num(b.float(), 9.0))
    m.clip_grad_norm(g, 1e-3)
    for x, b in zip(g, before):
        assert torch.equal(torch.nan_to_num(x, 9.0), torch.nan_to_num(b, 9.0))
    if dtype == F32:                        # finite gradients whose norm fp32 cannot hold
        huge = [torch.full((16,), 3e38, device="cuda")]
        assert m.clip_grad_norm(huge, 1.0).item() == float("inf") and (huge[0] == torch.tensor(3e38)).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_every_alignment_and_untouched_neighbours(dtype):
    m = mm()
    src, dst = torch.zeros(200000, device="cuda", dtype=dtype), torch.full((200000,), 5.0, device="cuda", dtype=dtype)
    grads, outs, at = [], [], 0
    fill = grads_of([200000], [dtype], seed=3)[0]
    for i, n in enumerate([1, 9, 2049, 4095, 30001, 17, 8192]):
        at += i + 1
        grads.append(src[at:at + n])
        outs.append(dst[at + i:at + i + n])
        grads[-1].copy_(fill[at:at + n])
        at += n + i
    before = [g.clone() for g in grads]
    norm = m.clip_grad_norm(grads, 0.1, outs=outs)
    check(grads, outs, before, norm, 0.1)
    total = sum(g.numel() for g in grads)
    assert (dst == 5.0).sum() >= 200000 - total
    touched = torch.zeros(200000, dtype=torch.bool, device="cuda")
    for o in outs:
        touched[o.storage_offset():o.storage_offset() + o.numel()] = True
    assert (dst[~touched] == 5.0).all()
    m.clip_grad_norm(grads, 0.1)
    check(grads, grads, before, norm, 0.1)
    mask = torch.ones(200000, dtype=torch.bool, device="cuda")
    for g in grads:
        mask[g.storage_offset():g.storage_offset() + g.numel()] = False
    assert not src[mask].any()


def test_a_norm_of_several_owners():
    m = mm()
    grads = grads_of([3000, 5000, 40000], [BF])
    whole = m.grad_norm(grads)
    parts = [m.grad_norm(grads[:1]), m.grad_norm(grads[1:])]
    joined = torch.stack(parts).double().square().sum().sqrt().float()
    assert abs(joined - whole) <= 2.0 ** -22 * whole
    a, b = ([torch.empty_like(g) for g in grads] for _ in range(2))
    assert m.clip_grad_norm(grads, 0.5, outs=a) is not None
    for lo, hi in ((0, 1), (1, 3)):
        assert m.clip_grad_norm(grads[lo:hi], 0.5, outs=b[lo:hi], norm=whole) is whole
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    assert m.grad_norm([]).item() == 0.0 and m.clip_grad_norm([], 1.0).item() == 0.0 and m.ClipGradNorm([], 1.0)().item() == 0.0
    assert m.grad_norm([grads[0][:0]]).item() == 0.0


def test_another_table_changes_nothing():
    """A run on a workspace that holds another plan's table writes neither norm nor outputs."""
    import ctypes

    from matrix_optimizer_muon_amd import _binding as B
    m = mm()
    a, b = grads_of([5000, 300], [BF]), grads_of([4000, 64], [F32], seed=2)
    clip, other = m.ClipGradNorm(a, 1e-3), m.ClipGradNorm(b, 1e-3)
    before, norm = [g.clone() for g in b], torch.full((), -1.0, device="cuda")
    ws = clip.workspace
    B.check(B.lib().dmuon_grad_clip_run(other._arr, other._n, 1e-3, 0.0, 1, norm.data_ptr(), ws.data_ptr(), ws.numel(),
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    B.check(B.lib().dmuon_grad_norm_run(other._arr, other._n, norm.data_ptr(), ws.data_ptr(), ws.numel(),
                                        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    torch.cuda.synchronize()
    assert norm.item() == -1.0
    for g, t in zip(b, before):
        assert torch.equal(g, t)


def test_same_bits_streams_and_graphs():
    m = mm()
    grads = grads_of([100, 70000, 1 << 20, 33], [BF, F32])
    outs = [torch.empty_like(g) for g in grads]
    clip = m.ClipGradNorm(grads, 0.5, outs=outs)
    norm = clip().clone()
    want = [o.clone() for o in outs]
    for _ in range(3):
        assert torch.equal(clip(), norm)
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    side = torch.cuda.Stream()
    for call in (lambda: clip(stream=side), lambda: m.clip_grad_norm(grads, 0.5, outs=outs, stream=side)):
        for o in outs:
            o.zero_()
        side.wait_stream(torch.cuda.current_stream())
        got = call()
        for _ in range(10):
            torch.empty(1 << 20, device="cuda").fill_(3.0)
        side.synchronize()
        assert torch.equal(got, norm)
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = clip()
        b = m.grad_norm(grads)
        single = [torch.empty_like(g) for g in grads]
        c = m.clip_grad_norm(grads, 0.5, outs=single)
    for k in (1.0, 3.0, 0.25, 1.0):
        fresh = grads_of([100, 70000, 1 << 20, 33], [BF, F32], seed=int(8 * k))
        for g, f in zip(grads, fresh):
            g.copy_(f * k)
        now = [g.clone() for g in grads]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(a, c)
        check(grads, outs, now, a, 0.5)
        for o, s in zip(outs, single):
            assert torch.equal(o, s)
        m.grad_norm(fresh)


def test_offsets_past_32_bits():
    m = mm()
    n = (1 << 31) + 12345
    g = torch.zeros(n, device="cuda", dtype=BF)
    g[0], g[-1], g[1 << 31] = 3.0, 4.0, 12.0
    assert m.grad_norm([g]).item() == 13.0
    m.clip_grad_norm([g], 6.5, eps=0.0)
    assert g[0] == 1.5 and g[-1] == 2.0 and g[1 << 31] == 6.0 and g.count_nonzero() == 3


def test_device_and_debug_sync(monkeypatch):
    m = mm()
    grads = grads_of([100, 5000], [F32])
    want = m.grad_norm(grads)
    monkeypatch.setenv("DMUON_DEBUG_SYNC", "1")
    assert torch.equal(m.grad_norm(grads), want)
    monkeypatch.delenv("DMUON_DEBUG_SYNC")
    monkeypatch.setenv("DMUON_TEST_FAIL_AT", "grad_clip")
    with pytest.raises(RuntimeError, match="forced failure"):
        m.clip_grad_norm(grads, 1.0)
    monkeypatch.delenv("DMUON_TEST_FAIL_AT")
    with pytest.raises(ValueError, match="contiguous"):
        m.grad_norm([torch.zeros(4, 6, device="cuda")[:, ::2]])
    with pytest.raises(ValueError, match="one value"):
        m.clip_grad_norm(grads, 1.0, norm=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        m.clip_grad_norm(grads, 1.0, outs=grads[::-1])
