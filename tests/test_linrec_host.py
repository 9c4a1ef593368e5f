"""The gated linear recurrence on the host: refusals before anything reaches a GPU (fake,
never dereferenced pointers), sizes, and the plain form's gradients against differences."""
import ctypes

import pytest
import torch

from kimi_delta_attention_08_gb300 import _lib, build
from tests.linrec_ref import linrec

OK, NULLP, SHAPE, ARG, MISALIGNED, WS = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def problem(**kw):
    q = _lib.kda_linrec_problem()
    v = dict(x=0x10000, r=0x20000, i=0x30000, z=0x40000, x_stride=64, r_stride=64, i_stride=64,
             z_stride=64, A_log=0x50000, r_bias=0x51000, i_bias=0x52000, initial_state=None,
             cu_seqlens=None, batch=2, T=40, N=0, dim=64, dtype=0, state_dtype=0)
    for k, x in {**v, **kw}.items():
        setattr(q, k, x)
    return q


def fwd(lib, q=None, **kw):
    a = dict(q=ctypes.byref(q if q is not None else problem()), out=0x70000, fin=None, cs=None, cb=0,
             ws=0x100000, wb=1 << 40, stream=None)
    return lib.kda_linrec_fwd(*[{**a, **kw}[k] for k in a])


def bwd(lib, q=None, **kw):
    a = dict(q=ctypes.byref(q if q is not None else problem()), dout=0x70000, dfin=None, cs=None, cb=0,
             dx=0x71000, dr=0x72000, di=0x73000, dz=0x74000, dA=0x75000, drb=0x76000, dib=0x77000,
             dinit=None, ws=0x100000, wb=1 << 40, stream=None)
    return lib.kda_linrec_bwd(*[{**a, **kw}[k] for k in a])


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    for kw in (dict(x=None), dict(r=None), dict(i=None), dict(A_log=None)):
        assert call(lib, problem(**kw)) == NULLP, kw
    for kw in (dict(batch=0), dict(T=-1), dict(dim=0), dict(x_stride=63), dict(r_stride=63),
               dict(i_stride=63), dict(z_stride=63), dict(z_stride=1 << 31), dict(T=1 << 31),
               dict(batch=1 << 20, T=1 << 20), dict(cu_seqlens=0x80000),
               dict(cu_seqlens=0x80000, batch=1, N=0)):
        assert call(lib, problem(**kw)) == SHAPE, kw
    for kw in (dict(dtype=2), dict(dtype=-1), dict(state_dtype=2)):
        assert call(lib, problem(**kw)) == ARG, kw
    for kw in (dict(x=0x10001), dict(z=0x40001), dict(A_log=0x50002), dict(r_bias=0x51001),
               dict(initial_state=0x80002), dict(cu_seqlens=0x80004, batch=1, N=2)):
        assert call(lib, problem(**kw)) == MISALIGNED, kw
    assert call(lib, ws=0x100040) == MISALIGNED
    assert call(lib, wb=255) == WS
    assert call(lib, cs=0x80000, cb=16) == WS
    assert call(lib, cs=0x80008, cb=1 << 30) == MISALIGNED
    assert call(lib, ws=None) == NULLP


def test_outputs(lib):
    assert fwd(lib, out=None) == NULLP and fwd(lib, out=0x70001) == MISALIGNED
    assert fwd(lib, fin=0x70002) == MISALIGNED
    assert fwd(lib, problem(T=8), ws=None, wb=0) in (OK, 6, 7)       # no workspace needed
    assert fwd(lib, problem(T=8), ws=0x100000, wb=16) == WS
    assert fwd(lib, problem(T=8), ws=None, wb=0, cs=0x80000, cb=1 << 30) == NULLP
    for kw in (dict(dout=None), dict(dx=None), dict(dr=None), dict(di=None), dict(dz=None), dict(dA=None)):
        assert bwd(lib, **kw) == NULLP, kw
    for kw in (dict(dout=0x70001), dict(dx=0x71001), dict(dA=0x75002), dict(dinit=0x78002), dict(dfin=0x78001)):
        assert bwd(lib, **kw) == MISALIGNED, kw


def test_sizes(lib):
    n = ctypes.c_size_t(0)
    size = lambda fn, *a: (getattr(lib, fn)(*a, ctypes.byref(n)), n.value)  # noqa: E731
    assert size("kda_linrec_get_states_size", 130, 64) == (OK, 3 * 64 * 4)
    assert size("kda_linrec_get_states_size", 0, 64) == (OK, 64 * 4)
    for bad in ((-1, 64), (10, 0), (1 << 31, 64)):
        assert size("kda_linrec_get_states_size", *bad)[0] == SHAPE
    q = ctypes.byref(problem(T=1000))
    st, f = size("kda_linrec_get_workspace_size", q)
    assert st == OK and f >= 256 + 16 * 64 * 8
    st, with_states = size("kda_linrec_bwd_get_workspace_size", q, 1)
    st, without = size("kda_linrec_bwd_get_workspace_size", q, 0)
    assert without > with_states > f
    assert size("kda_linrec_get_workspace_size", ctypes.byref(problem(dim=0)))[0] == SHAPE
    assert size("kda_linrec_get_workspace_size", None)[0] == NULLP
    assert lib.kda_linrec_get_states_size(1, 1, None) == NULLP


def test_binding_refusals():
    import kimi_delta_attention_08_gb300 as kda
    x, A = torch.zeros(2, 3, 8, dtype=torch.bfloat16), torch.zeros(8)
    call = lambda **kw: kda.kda_linrec_fwd(**{**dict(x=x, r=x, i=x, A_log=A, out=x), **kw})  # noqa: E731
    for kw in (dict(x=x.half()), dict(r=x.float()), dict(A_log=A.double()), dict(out=x.float()),
               dict(initial_state=torch.zeros(2, 8, dtype=torch.float64)), dict(x=3), dict(r=None),
               dict(z=x.float()), dict(A_log=None)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(x=x[0]), dict(r=x[:, :2]), dict(A_log=torch.zeros(7)), dict(out=x[..., ::2]),
               dict(i=x.transpose(0, 1)), dict(initial_state=torch.zeros(3, 8)), dict(A_log=torch.zeros(8, 1)),
               dict(cu_seqlens=torch.zeros(3)), dict(r_bias=torch.zeros(8, 1)[:, 0].expand(3, 8)[0][:4]),
               dict(initial_state=torch.zeros(2, 8), final_state=torch.zeros(2, 7)), dict()):
        with pytest.raises(ValueError):  # the last: tensors that are not on a GPU
            call(**kw)
    with pytest.raises(ValueError, match="make_linrec_states"):
        call(chunk_states=torch.zeros(4))


@pytest.mark.parametrize("cu", [None, [0, 0, 3, 7]])
@pytest.mark.parametrize("z", [True, False])
def test_plain_gradients_against_differences(cu, z):
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    B, T, D, N = (2, 4, 3, 2) if cu is None else (1, 8, 3, 3)
    v = dict(x=rnd(B, T, D), r=rnd(B, T, D), i=rnd(B, T, D), A_log=rnd(D) - 1, z=rnd(B, T, D) if z else None,
             r_bias=rnd(D), i_bias=rnd(D), init=rnd(N, D))
    dout, dfin = rnd(B, T, D), rnd(N, D)

    def loss(**kw):
        o, f = linrec(**{**v, **kw}, cu=cu)
        return float((o * dout).sum() + (f * dfin).sum())
    got = linrec(**v, cu=cu, dout=dout, dfin=dfin)
    names = dict(dx="x", dr="r", di="i", dz="z", dA_log="A_log", dr_bias="r_bias", di_bias="i_bias",
                 dinitial_state="init")
    for k, grad in got.items():
        t = v[names[k]]
        num = torch.zeros_like(t)
        for j in range(t.numel()):
            e = torch.zeros_like(t)
            e.view(-1)[j] = 1e-6
            num.view(-1)[j] = (loss(**{names[k]: t + e}) - loss(**{names[k]: t - e})) / 2e-6
        # differences: 1e-12 of the curvature, and 2^-53 of a loss of some tens over 2e-6
        assert (num - grad).abs().max() < 1e-7, k
