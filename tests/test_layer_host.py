"""Host-side checks of the layer operators: every refusal comes back as a status before
anything reaches a GPU (fake, never dereferenced pointers), workspace sizes, and the
binding's own checks.  No kernel is launched here."""
import ctypes

import pytest
import torch

from kimi_delta_attention_08_gb300 import _lib, build

OK, NULLP, SHAPE, ARG, MISALIGNED, WS = 0, 1, 2, 3, 4, 5
NO_GPU = (6, 7)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def caller(fn, args):
    """fn with named default arguments, in order."""
    return lambda **kw: fn(*[{**args, **kw}[k] for k in args])


def conv_fwd(lib, outs=(0x40000,), counts=(64,)):
    n = len(outs)
    return caller(lib.kda_conv_fwd, dict(
        x=0x10000, xs=64, w=0x20000, b=0x30000, outs=(ctypes.c_void_p * n)(*outs),
        counts=(ctypes.c_int32 * n)(*counts), k=n, init=None, fin=None, cu=None, B=2, T=5, C=64, N=0,
        width=4, fn=1, dtype=0, ws=None, wb=0, stream=None))


def conv_bwd(lib, outs=(0x40000,), counts=(64,)):
    n = len(outs)
    return caller(lib.kda_conv_bwd, dict(
        x=0x10000, xs=64, w=0x20000, b=0x30000, outs=(ctypes.c_void_p * n)(*outs),
        counts=(ctypes.c_int32 * n)(*counts), k=n, ddt=0, init=None, dfin=None, cu=None, dx=0x50000,
        dw=0x60000, db=0x70000, di=None, B=2, T=5, C=64, N=0, width=4, fn=1, dtype=0, ws=0x100000,
        wb=1 << 30, stream=None))


@pytest.mark.parametrize("make", [conv_fwd, conv_bwd])
def test_conv_refusals(lib, make):
    call = make(lib)
    for kw in (dict(x=None), dict(w=None)):
        assert call(**kw) == NULLP, kw
    for kw in (dict(B=0), dict(T=-1), dict(C=0), dict(width=1), dict(width=5), dict(xs=63),
               dict(xs=1 << 31), dict(B=1, T=1 << 31), dict(B=1 << 20, T=1 << 20), dict(cu=0x80000, B=2, N=3),
               dict(cu=0x80000, B=1, N=0), dict(k=0), dict(k=5)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(fn=2), dict(fn=-1), dict(dtype=2)):
        assert call(**kw) == ARG, kw
    for kw in (dict(x=0x10001), dict(w=0x20002), dict(b=0x30001), dict(cu=0x80004, B=1, N=3)):
        assert call(**kw) == MISALIGNED, kw
    assert make(lib, (0x40000, 0x48000), (32, 31))() == SHAPE      # counts do not add up to C
    assert make(lib, (0x40000, 0x48000), (64, 0))() == SHAPE
    assert make(lib, (0x40000, None), (32, 32))() == NULLP
    assert make(lib, (0x40001,))() == MISALIGNED


def test_conv_workspaces(lib):
    assert conv_fwd(lib)(ws=0x100000, wb=255) == WS
    assert conv_fwd(lib)(ws=0x100040, wb=256) == MISALIGNED
    call = conv_bwd(lib)
    assert call(wb=16) == WS and call(ws=None) == NULLP and call(dw=None) == NULLP and call(dx=None) == NULLP
    n = ctypes.c_size_t(0)
    size = lambda *a: (lib.kda_conv_bwd_get_workspace_size(*a, ctypes.byref(n)), n.value)  # noqa: E731
    st, small = size(100, 64, 4)
    assert st == OK and small >= 256 + 5 * 64 * 4
    assert size(100000, 64, 4)[1] > small and size(0, 64, 4) == (OK, 256)
    for bad in ((-1, 64, 4), (10, 0, 4), (10, 64, 5), (1 << 31, 64, 4)):
        assert size(*bad)[0] == SHAPE
    assert lib.kda_conv_bwd_get_workspace_size(10, 64, 4, None) == NULLP


def scan_problem(**kw):
    q = _lib.kda_scan_problem()
    v = dict(x=0x10000, dt=0x20000, z=0x30000, B=0x40000, C=0x50000, x_stride=64, dt_stride=64,
             z_stride=64, B_stride=16, C_stride=16, A_log=0x60000, D=0x61000, dt_bias=0x62000,
             initial_state=None, cu_seqlens=None, batch=2, T=40, N=0, dim=64, state=16, groups=1,
             dtype=0, state_dtype=0)
    for k, x in {**v, **kw}.items():
        setattr(q, k, x)
    return q


def scan_fwd(lib, q=None, **kw):
    a = dict(q=ctypes.byref(q if q is not None else scan_problem()), out=0x70000, fin=None, cs=None, cb=0,
             ws=0x100000, wb=1 << 40, stream=None)
    return lib.kda_scan_fwd(*[{**a, **kw}[k] for k in a])


def scan_bwd(lib, q=None, **kw):
    a = dict(q=ctypes.byref(q if q is not None else scan_problem()), dout=0x70000, dfin=None, cs=None, cb=0,
             dx=0x71000, ddt=0x72000, dz=0x73000, dB=0x74000, dC=0x75000, dA=0x76000, dD=0x77000,
             db=0x78000, di=None, ws=0x100000, wb=1 << 40, stream=None)
    return lib.kda_scan_bwd(*[{**a, **kw}[k] for k in a])


@pytest.mark.parametrize("call", [scan_fwd, scan_bwd])
def test_scan_refusals(lib, call):
    for kw in (dict(x=None), dict(dt=None), dict(B=None), dict(C=None), dict(A_log=None)):
        assert call(lib, scan_problem(**kw)) == NULLP, kw
    for kw in (dict(batch=0), dict(T=-1), dict(dim=0), dict(state=12), dict(state=0), dict(state=128),
               dict(groups=0), dict(groups=3), dict(x_stride=63), dict(z_stride=63), dict(B_stride=15),
               dict(T=1 << 31), dict(batch=1 << 20, T=1 << 20), dict(cu_seqlens=0x80000),
               dict(cu_seqlens=0x80000, batch=1, N=0), dict(C_stride=1 << 32)):
        assert call(lib, scan_problem(**kw)) == SHAPE, kw
    for kw in (dict(dtype=2), dict(state_dtype=2)):
        assert call(lib, scan_problem(**kw)) == ARG, kw
    for kw in (dict(x=0x10001), dict(A_log=0x60002), dict(initial_state=0x80008), dict(D=0x61001),
               dict(cu_seqlens=0x80004, batch=1, N=2)):
        assert call(lib, scan_problem(**kw)) == MISALIGNED, kw
    assert call(lib, ws=0x100040) == MISALIGNED
    assert call(lib, cs=0x80000, cb=16) == WS
    assert call(lib, cs=0x80004, cb=1 << 30) == MISALIGNED


def test_scan_fwd_refusals(lib):
    assert scan_fwd(lib, out=None) == NULLP
    assert scan_fwd(lib, fin=0x80004) == MISALIGNED
    assert scan_fwd(lib, wb=16) == WS
    # few channels and many tokens: the scan is cut, which needs a workspace
    assert scan_fwd(lib, scan_problem(T=4096), ws=None, wb=0) == NULLP


def test_scan_bwd_refusals(lib):
    for k in ("dout", "dx", "ddt", "dB", "dC", "dA", "ws"):
        assert scan_bwd(lib, **{k: None}) == NULLP, k
    assert scan_bwd(lib, wb=256) == WS
    assert scan_bwd(lib, scan_problem(z=None)) == ARG          # dz without z
    assert scan_bwd(lib, scan_problem(D=None)) == ARG
    assert scan_bwd(lib, scan_problem(dt_bias=None)) == ARG


def test_scan_sizes(lib):
    n = ctypes.c_size_t(0)
    assert lib.kda_scan_get_states_size(100, 3, 64, 16, ctypes.byref(n)) == OK
    assert n.value == (100 // 32 + 3 + 1) * 64 * 16 * 4
    assert lib.kda_scan_get_states_size(-1, 3, 64, 16, ctypes.byref(n)) == SHAPE
    assert lib.kda_scan_get_states_size(100, 3, 64, 16, None) == NULLP
    q = scan_problem()
    fwd = lambda q: (lib.kda_scan_get_workspace_size(ctypes.byref(q), ctypes.byref(n)), n.value)  # noqa: E731
    bwd = lambda q, h: (lib.kda_scan_bwd_get_workspace_size(ctypes.byref(q), h, ctypes.byref(n)), n.value)  # noqa: E731
    assert fwd(scan_problem(batch=256, T=64, dim=4096, x_stride=4096)) == (OK, 256)  # not cut
    assert fwd(scan_problem(T=8192))[1] > 256
    assert bwd(q, 0)[1] > bwd(q, 1)[1] > 256
    assert fwd(scan_problem(state=5))[0] == SHAPE and bwd(scan_problem(dim=-1), 0)[0] == SHAPE
    assert lib.kda_scan_get_workspace_size(None, ctypes.byref(n)) == NULLP
    assert lib.kda_scan_get_workspace_size(ctypes.byref(q), None) == NULLP


def norms(lib):
    pre = dict(x=0x10000, res=0x20000, w=0x30000, s=None, sv=1.0, eps=1e-6, out=0x40000, ro=0x50000,
               rows=4, dim=64, dtype=0, sdt=0, stream=None)
    preb = dict(dout=0x10000, dh=0x20000, h=0x21000, w=0x30000, x=0x22000, s=None, sv=1.0, eps=1e-6,
                dx=0x40000, dr=0x50000, dw=0x60000, ds=None, rows=4, dim=64, dtype=0, sdt=0, ws=0x100000,
                wb=1 << 30, stream=None)
    post = dict(x=0x10000, w=0x30000, gate=0x20000, gs=64, heads=1, res=None, s=None, sv=1.0, eps=1e-6,
                fn=1, out=0x40000, rows=4, dim=64, dtype=0, stream=None)
    postb = dict(dout=0x10000, x=0x21000, w=0x30000, gate=0x20000, gs=64, heads=1, s=None, sv=1.0,
                 eps=1e-6, fn=1, dx=0x40000, dg=0x50000, dw=0x60000, ds=None, rows=4, dim=64, dtype=0,
                 ws=0x100000, wb=1 << 30, stream=None)
    return [caller(lib.kda_prenorm_fwd, pre), caller(lib.kda_prenorm_bwd, preb),
            caller(lib.kda_postnorm_fwd, post), caller(lib.kda_postnorm_bwd, postb)]


def test_norm_refusals(lib):
    pre, preb, post, postb = every = norms(lib)
    for call in every:
        for kw in (dict(rows=-1), dict(dim=0), dict(dim=8193)):
            assert call(**kw) == SHAPE, kw
        for kw in (dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(sv=float("inf"))):
            assert call(**kw) == ARG, kw
        assert call(w=None) == NULLP and call(w=0x30002) == MISALIGNED
    for call in (pre, post):
        assert call(x=None) == NULLP and call(out=None) == NULLP and call(x=0x10001) == MISALIGNED
    for call in (preb, postb):
        assert call(dout=None) == NULLP and call(dw=None) == NULLP and call(ws=None) == NULLP
        assert call(wb=16) == WS and call(ws=0x100040) == MISALIGNED
    for call in (post, postb):
        assert call(fn=0) == ARG
        for kw in (dict(heads=0), dict(heads=3), dict(gs=63), dict(gs=1 << 31)):
            assert call(**kw) == SHAPE, kw
    for call in (pre, preb):
        assert call(sdt=2) == ARG and call(dtype=1, sdt=0) == ARG   # fp32 rows, bf16 stream
    assert preb(h=None) == NULLP and preb(dx=None, dr=None) == NULLP and preb(ds=0x70000, x=None) == NULLP
    assert postb(gate=None) == NULLP                                # dgate without a gate
    n = ctypes.c_size_t(0)
    assert lib.kda_norm_bwd_get_workspace_size(10, 64, ctypes.byref(n)) == OK and n.value >= 256
    assert lib.kda_norm_bwd_get_workspace_size(10, 9000, ctypes.byref(n)) == SHAPE
    assert lib.kda_norm_bwd_get_workspace_size(10, 64, None) == NULLP


def test_accepted_calls_need_a_device(lib):
    """What passes the host checks stops at the device check on a host without a GPU."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert conv_fwd(lib)() in NO_GPU and conv_bwd(lib)() in NO_GPU
    assert scan_fwd(lib) in NO_GPU and scan_bwd(lib) in NO_GPU
    for call in norms(lib):
        assert call() in NO_GPU
    assert norms(lib)[0](x=None, out=None, rows=0) in NO_GPU        # no rows: no buffers needed


def test_binding_checks():
    """The binding refuses wrong dtypes, shapes and layouts, and tensors that are not on a GPU."""
    import kimi_delta_attention_08_gb300 as kda
    x, w, b = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(8)
    out = torch.zeros(2, 5, 8)
    with pytest.raises(TypeError):
        kda.kda_conv_fwd(x.half(), w, b, out)
    with pytest.raises(TypeError):
        kda.kda_conv_fwd(x, w.double(), b, out)
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w, b, out[:, :, :7].contiguous())
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w, b, [out] * 5)
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x.transpose(1, 2).contiguous().transpose(1, 2), w, b, out)
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w, b, out, torch.zeros(2, 4, 8))
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w, b, out, activation="relu")
    with pytest.raises(ValueError):
        kda.kda_conv_fwd(x, w, b, out)                       # not CUDA tensors
    with pytest.raises(ValueError):
        kda.kda_prenorm_fwd(x, x[:1], b, out)
    with pytest.raises(TypeError):
        kda.kda_prenorm_fwd(x, None, b.double(), out)
    with pytest.raises(ValueError):
        kda.kda_prenorm_bwd(x, None, x, b, res_scale=b)      # x is needed
    with pytest.raises(ValueError):
        kda.kda_postnorm_fwd(x, b, x, out, activation="tanh")
    A, B = torch.zeros(8, 16), torch.zeros(2, 5, 1, 16)
    with pytest.raises(ValueError):
        kda.kda_scan_fwd(x, x, A, B, B[:, :, :, :8], out)
    with pytest.raises(TypeError):
        kda.kda_scan_fwd(x, x, A, B, B, out, initial_state=torch.zeros(2, 8, 16, dtype=torch.float16))
    with pytest.raises(TypeError):
        kda.kda_scan_fwd(x, x, A, B, B, out, initial_state=torch.zeros(2, 8, 16),
                         final_state=torch.zeros(2, 8, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        kda.kda_scan_fwd(x, x, A, B, B, out)                 # not CUDA tensors
    with pytest.raises(AttributeError):
        kda.kda_nothing
