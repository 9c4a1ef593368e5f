"""Which stream's memory the layer operators' results come from, checked on the host: streams,
allocations and the library's call are stand-ins, nothing reaches a GPU."""
from contextlib import contextmanager

import pytest
import torch

from kimi_delta_attention_08_gb300 import layer

CUDA = torch.device("cuda", 0)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def seen(monkeypatch):
    """Every allocation as [handle of the stream that is current then, recorded streams]."""
    now, made = [100], []
    real = torch.empty

    @contextmanager
    def stream(s):
        now.append(s.cuda_stream)
        yield
        now.pop()

    class Result:
        def __init__(self, entry):
            self.entry = entry

        def data_ptr(self):
            return 256

        def numel(self):
            return 1 << 30

        def record_stream(self, s):
            self.entry[1].append(s.cuda_stream)

    def empty(*size, dtype=None, device=None, **kw):
        if device != CUDA:
            return real(*size, dtype=dtype, device=device, **kw)
        made.append([now[-1], []])
        return Result(made[-1])

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(now[-1]))
    monkeypatch.setattr(layer, "_call", lambda *a: None)
    monkeypatch.setattr(layer, "_size", lambda *a: 1 << 20)
    return made


class Tensor(torch.Tensor):
    """A contiguous tensor on the GPU without memory."""

    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=CUDA)

    @classmethod
    def __torch_dispatch__(cls, *args, **kw):
        return NotImplemented

    def data_ptr(self):
        return 256

    def record_stream(self, s):
        pass


def calls(stream, workspace):
    x, w, b = Tensor(2, 5, 8), Tensor(8, 4), Tensor(8)
    B, A, ini, st = Tensor(2, 5, 1, 16), Tensor(8, 16), Tensor(2, 3, 8), Tensor(2, 8, 16)
    kw = dict(stream=stream, workspace=workspace)
    return {"conv": lambda: layer.kda_conv_bwd(x, w, b, (x,), ini, **kw),
            "scan": lambda: layer.kda_scan_bwd(x, x, A, B, B, x, b, x, b, st, **kw),
            "prenorm": lambda: layer.kda_prenorm_bwd(x, None, x, b, res_scale=0.5, **kw),
            "postnorm": lambda: layer.kda_postnorm_bwd(x, x, b, x, res_scale=0.5, **kw)}


@pytest.mark.parametrize("op", ["conv", "scan", "prenorm", "postnorm"])
def test_results_come_from_the_stream_that_writes_them(seen, op):
    calls(None, None)[op]()
    assert len(seen) > 2 and all(e == [100, []] for e in seen)
    seen.clear()
    calls(Stream(7), None)[op]()
    assert len(seen) > 2 and all(h == 7 and 100 in r for h, r in seen), seen
    for handle in (7, 0):
        seen.clear()
        calls(handle, Tensor(1 << 20, dtype=torch.uint8))[op]()
        assert len(seen) > 1 and all(h == handle for h, _ in seen), seen
        assert all(r == [100] for _, r in seen)


def test_workspace_of_a_forward_call(seen):
    x, A, B = Tensor(2, 50, 8), Tensor(8, 16), Tensor(2, 50, 1, 16)
    layer.kda_scan_fwd(x, x, A, B, B, x, stream=Stream(7))
    assert seen == [[7, []]]


def test_gradients_of_the_recurrence(seen, monkeypatch):
    """kda_bwd with a stream: the same."""
    import kimi_delta_attention_08_gb300 as kda

    class Library:
        def kda_bwd(self, *args):
            return 0

        def kda_bwd_get_workspace_size(self, *args):
            return 0

    monkeypatch.setattr(kda._lib, "load", Library)
    bf = torch.bfloat16
    q, beta, A, bias = Tensor(1, 9, 2, 128, dtype=bf), Tensor(1, 9, 2, dtype=bf), Tensor(2), Tensor(2, 128)
    ws = Tensor(1 << 20, dtype=torch.uint8)
    for stream, handle, kept in ((None, 100, []), (Stream(7), 7, [100, 7]), (7, 7, [100]), (0, 0, [100])):
        seen.clear()
        kda.kda_bwd(q, q, q, q, beta, 1.0, A, bias, -5.0, q, workspace=ws, stream=stream)
        assert len(seen) == 8 and all(e == [handle, kept] for e in seen), (stream, seen)


def test_buffers_made_for_a_call_live_until_its_stream_is_done(seen, monkeypatch):
    """Saved states and workspaces may be dropped right after the call."""
    kept = []
    monkeypatch.setattr(Tensor, "record_stream", lambda self, s: kept.append((self, s.cuda_stream)))
    x, A, B, w, b = Tensor(2, 50, 8), Tensor(8, 16), Tensor(2, 50, 1, 16), Tensor(8, 4), Tensor(8)
    ws, st = (Tensor(1 << 20, dtype=torch.uint8) for _ in range(2))
    for run, buffers in (
            (lambda s: layer.kda_scan_fwd(x, x, A, B, B, x, workspace=ws, chunk_states=st, stream=s), {ws, st}),
            (lambda s: layer.kda_scan_bwd(x, x, A, B, B, x, workspace=ws, chunk_states=st, stream=s), {ws, st}),
            (lambda s: layer.kda_conv_fwd(x, w, b, x, workspace=ws, stream=s), {ws}),
            (lambda s: layer.kda_conv_bwd(x, w, b, x, workspace=ws, stream=s), {ws}),
            (lambda s: layer.kda_prenorm_bwd(x, None, x, b, workspace=ws, stream=s), {ws}),
            (lambda s: layer.kda_postnorm_bwd(x, x, b, None, ws, stream=s), {ws})):
        kept.clear()
        run(Stream(7))
        assert {id(t) for t, s in kept if s == 7} == {id(t) for t in buffers}
        kept.clear()
        run(None)
        assert not kept
