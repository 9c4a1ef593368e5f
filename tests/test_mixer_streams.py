"""The linear recurrence and the feed-forward product on another stream than the current one: where
their results' memory comes from, and that buffers made for a call outlive it.  On the host, with
the stand-ins of tests/test_layer_streams.py."""
import pytest
import torch

from kimi_delta_attention_08_gb300 import layer
from tests.test_layer_streams import Stream, Tensor, seen  # noqa: F401

BF = torch.bfloat16


def calls(ws, st, pre):
    x, A, fin = Tensor(2, 50, 8), Tensor(8), Tensor(2, 8)
    y, w, o = Tensor(2, 50, 8, dtype=BF), Tensor(16, 8, dtype=BF), Tensor(2, 50, 16, dtype=BF)
    return {"linrec_fwd": (lambda s: layer.kda_linrec_fwd(x, x, x, A, x, workspace=ws, chunk_states=st, stream=s), [ws, st]),
            "linrec_bwd": (lambda s: layer.kda_linrec_bwd(x, x, x, A, x, x, A, A, fin, workspace=ws, chunk_states=st,
                                                          stream=s), [ws, st]),
            "glu_fwd": (lambda s: layer.kda_glu_fwd(y, w, w, o, ws, pre=pre, stream=s), [ws, pre]),
            "glu_bwd": (lambda s: layer.kda_glu_bwd(y, w, w, o, ws, pre=pre, stream=s), [ws, pre])}


@pytest.mark.parametrize("op", ["linrec_fwd", "linrec_bwd", "glu_fwd", "glu_bwd"])
@pytest.mark.parametrize("ty", [BF, torch.int16])
def test_buffers_made_for_a_call_live_until_its_stream_is_done(seen, monkeypatch, op, ty):  # noqa: F811
    """Workspaces, saved states and kept pre-activations may be dropped right after the call."""
    kept = []
    monkeypatch.setattr(Tensor, "record_stream", lambda self, s: kept.append((self, s.cuda_stream)))
    ws, st, pre = (Tensor(1 << 20, dtype=torch.uint8), Tensor(1 << 20, dtype=torch.uint8), Tensor(2, 50, 32, dtype=ty))
    run, buffers = calls(ws, st, pre)[op]
    run(Stream(7))
    assert {id(t) for t, s in kept if s == 7} == {id(t) for t in buffers}
    kept.clear()
    run(None)
    assert not kept


@pytest.mark.parametrize("op", ["linrec_bwd", "glu_bwd"])
def test_results_come_from_the_stream_that_writes_them(seen, op):  # noqa: F811
    calls(None, None, None)[op][0](None)
    assert len(seen) > 2 and all(e == [100, []] for e in seen)
    seen.clear()
    calls(None, None, None)[op][0](Stream(7))
    assert len(seen) > 2 and all(h == 7 and 100 in r for h, r in seen), seen


def test_workspace_of_a_forward_call(seen):  # noqa: F811
    calls(None, None, None)["linrec_fwd"][0](Stream(7))
    assert seen == [[7, []]]
    seen.clear()
    calls(None, None, None)["glu_fwd"][0](Stream(7))
    assert not seen
