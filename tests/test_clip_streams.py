"""ClipGradNorm called on another stream than its tensors': the allocator is told of every
tensor that the queued kernels use."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import matrix_optimizer_muon_amd as mm
from matrix_optimizer_muon_amd import _binding as B
from matrix_optimizer_muon_amd import clip as C


@pytest.mark.parametrize("in_place", [False, True])
def test_every_tensor_is_recorded(in_place, monkeypatch):
    """Without a GPU: the library, the streams and the allocator's hook are stand-ins."""
    recorded, running = [], []

    @contextlib.contextmanager
    def on(stream, *tensors):
        st = stream or "own"
        running.append(st)
        yield SimpleNamespace(handle=SimpleNamespace(value=st))
        running.pop()

    monkeypatch.setattr(C, "_on", on)
    monkeypatch.setattr(C, "_descs", lambda grads, outs: (None, len(grads), "cuda:0"))
    monkeypatch.setattr(C, "_workspace", lambda *a: "workspace")
    monkeypatch.setattr(C, "_new_norm", lambda *a: "norm")
    monkeypatch.setattr(C, "_ws_args", lambda ws: (0, 0))
    monkeypatch.setattr(C, "_ptr", lambda t: 0)
    monkeypatch.setattr(B, "lib", lambda: SimpleNamespace(dmuon_grad_prepare=lambda *a: 0, dmuon_grad_clip_run=lambda *a: 0))
    monkeypatch.setattr(B, "resolve_stream", lambda stream: running[-1])
    monkeypatch.setattr(B, "keep_until_done", lambda t, streams: recorded.extend((t, s) for s in streams))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(synchronize=lambda: None))
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])

    grads, outs = ["g0", "g1", "g2"], None if in_place else ["o0", "o1", "o2"]
    clip = C.ClipGradNorm(grads, 1.0, outs=outs)
    recorded.clear()
    clip(stream="side")
    assert {(t, "side") for t in ("norm", "workspace", *grads, *(outs or ()))} <= set(recorded)
    recorded.clear()
    clip(stream="side")                     # once per stream
    assert not {t for t, _ in recorded} & {*grads, *(outs or ())}
    capturing[0] = True                     # a capture records nothing, and does not count as the first call
    clip(stream="third")
    assert not recorded
    capturing[0] = False
    clip(stream="third")
    assert {(t, "third") for t in (*grads, *(outs or ()))} <= set(recorded)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_tensors_dropped_behind_a_call(in_place):
    """What is allocated while the call is queued does not lie in the dropped tensors."""
    side = torch.cuda.Stream()
    n = 3 << 20
    grads = [torch.ones(n, device="cuda") for _ in range(3)]
    outs = None if in_place else [torch.empty(n, device="cuda") for _ in range(3)]
    clip = mm.ClipGradNorm(grads, 1.0, outs=outs)
    torch.cuda.synchronize()
    used = {t.data_ptr() for t in (*grads, *(outs or ()))}
    a = torch.zeros(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(200):                # the call waits in the queue behind these
            a @ a
    norm = clip(stream=side)
    del clip, grads, outs
    fresh = [torch.zeros(n, device="cuda") for _ in range(8)]
    assert not used & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    assert norm.item() == torch.tensor((3.0 * n) ** 0.5).item()
    assert not any(t.any() for t in fresh)
