"""The gated feed-forward product on the host: refusals before anything reaches a GPU (fake,
never dereferenced pointers), sizes, and the plain form's gradients against differences."""
import ctypes

import pytest
import torch

from kimi_delta_attention_08_gb300 import _lib, build
from tests.glu_ref import glu

OK, NULLP, SHAPE, ARG, MISALIGNED, WS = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def problem(**kw):
    q = _lib.kda_glu_problem()
    v = dict(x=0x10000, w_gate=0x20000, w_up=0x30000, x_stride=64, rows=40, dim=64, hidden=128, fn=1, dtype=0)
    for k, x in {**v, **kw}.items():
        setattr(q, k, x)
    return q


def fwd(lib, q=None, **kw):
    a = dict(q=ctypes.byref(q if q is not None else problem()), out=0x70000, pre=None, ws=None, wb=0, stream=None)
    return lib.kda_glu_fwd(*[{**a, **kw}[k] for k in a])


def bwd(lib, q=None, **kw):
    a = dict(q=ctypes.byref(q if q is not None else problem()), dout=0x70000, pre=None, dx=0x71000,
             dwg=0x72000, dwu=0x73000, ws=0x100000, wb=1 << 40, stream=None)
    return lib.kda_glu_bwd(*[{**a, **kw}[k] for k in a])


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    for kw in (dict(x=None), dict(w_gate=None), dict(w_up=None)):
        assert call(lib, problem(**kw)) == NULLP, kw
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dim=60), dict(hidden=0), dict(hidden=129),
               dict(x_stride=56), dict(x_stride=68), dict(x_stride=1 << 31),
               dict(rows=(1 << 31) - 1, hidden=(1 << 31) - 8), dict(dim=(1 << 31) - 8, hidden=(1 << 31) - 8, x_stride=(1 << 31) - 8)):
        assert call(lib, problem(**kw)) == SHAPE, kw
    for kw in (dict(fn=0), dict(fn=4), dict(dtype=1)):
        assert call(lib, problem(**kw)) == ARG, kw
    for kw in (dict(x=0x10008), dict(w_gate=0x20008), dict(w_up=0x30002)):
        assert call(lib, problem(**kw)) == MISALIGNED, kw
    assert call(lib, pre=0x80008) == MISALIGNED
    assert call(lib, ws=0x100040, wb=1 << 30) == MISALIGNED
    assert call(lib, ws=0x100000, wb=255) == WS


def test_outputs_and_sizes(lib):
    assert fwd(lib, out=None) == NULLP and fwd(lib, out=0x70008) == MISALIGNED
    for k in ("dout", "dx", "dwg", "dwu", "ws"):
        assert bwd(lib, **{k: None}) == NULLP, k
    for k in ("dout", "dx", "dwg", "dwu"):
        assert bwd(lib, **{k: 0x70008}) == MISALIGNED, k
    n = ctypes.c_size_t(0)
    size = lambda *a: (lib.kda_glu_bwd_get_workspace_size(*a, ctypes.byref(n)), n.value)  # noqa: E731
    assert size(0, 64) == (OK, 256)
    st, b = size(100, 64)
    assert st == OK and b >= 256 + 2 * 100 * 64 * 2
    assert bwd(lib, wb=size(40, 128)[1] - 1) == WS
    for bad in ((-1, 64), (10, 0), (10, 60), (1 << 31, 64)):
        assert size(*bad)[0] == SHAPE
    assert lib.kda_glu_bwd_get_workspace_size(10, 64, None) == NULLP


def test_binding_refusals():
    import kimi_delta_attention_08_gb300 as kda
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    base = dict(x=t(2, 3, 8), w_gate=t(16, 8), w_up=t(16, 8), out=t(2, 3, 16))
    call = lambda **kw: kda.kda_glu_fwd(**{**base, **kw})  # noqa: E731
    for kw in (dict(x=t(2, 3, 8).float()), dict(w_gate=t(16, 8).float()), dict(w_up=None), dict(x=None),
               dict(out=t(2, 3, 16).float()), dict(pre=t(2, 3, 32).half()), dict(w_gate=3)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(x=t(3, 8)), dict(w_gate=t(16, 4)), dict(w_up=t(8, 8)), dict(w_gate=t(8, 16).T),
               dict(out=t(2, 3, 8)), dict(pre=t(2, 3, 16)), dict(activation="relu"),
               dict(workspace=torch.zeros(256)), dict()):  # the last: tensors that are not on a GPU
        with pytest.raises(ValueError):
            call(**kw)


@pytest.mark.parametrize("fn", ["silu", "gelu", "sigmoid"])
def test_plain_gradients_against_differences(fn):
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    v = dict(x=rnd(1, 3, 4), wg=rnd(5, 4), wu=rnd(5, 4))
    dout = rnd(1, 3, 5)
    got = glu(**v, fn=fn, dout=dout)
    loss = lambda **kw: float((glu(**{**v, **kw}, fn=fn)["out"][0] * dout).sum())  # noqa: E731
    for k, nm in (("dx", "x"), ("dw_gate", "wg"), ("dw_up", "wu")):
        t, num = v[nm], torch.zeros_like(v[nm])
        for j in range(t.numel()):
            e = torch.zeros_like(t)
            e.view(-1)[j] = 1e-6
            num.view(-1)[j] = (loss(**{nm: t + e}) - loss(**{nm: t - e})) / 2e-6
        # differences: 1e-12 of the third derivative, and 2^-53 of a loss of some tens over 2e-6
        assert (num - got[k][0]).abs().max() < 1e-7, k
