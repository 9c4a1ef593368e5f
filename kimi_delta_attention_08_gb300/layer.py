"""Binding of the operators around the KDA recurrence in a layer (include/kda_layer.h):
the short causal convolution, the selective state space scan, and the norms before
and after a block.

As in the rest of the binding, arguments are only checked and passed on: every
tensor has to have the documented dtype, device and layout.  Row arguments marked
"rows" may be a slice of a wider projection's output (contiguous channels, tokens
one fixed stride apart).  Work goes to torch's current stream of the tensors'
device, or to `stream`; what is allocated for it then comes from that stream's memory.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext

import torch

from . import _lib

KDA_OK = 0
ROW_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
CONV_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
GATE_ACTIVATIONS = {"silu": 1, "sigmoid": 2}
_f32 = torch.float32


def _raise(status, where):
    from . import KdaError
    raise KdaError(status, where)


def _tensor(t, name):
    """t, which has to be a tensor.  (Single tokens are bound by the host: what they check looks
    first and asks this only where that fails.)"""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    return t


def _tensors(**given):
    for name, t in given.items():
        _tensor(t, name)


def _row_dtype(t, name):
    try:
        code = ROW_DTYPES.get(t.dtype)
    except AttributeError:
        code = None
    if code is None:
        _tensor(t, name)
        raise TypeError(f"{name}: expected bfloat16 or float32, got {t.dtype} (no implicit conversion)")
    return code


def _need(t, name, dtype, dev, shape):
    """The pointer of a contiguous tensor of this dtype, device and shape."""
    try:
        if t.dtype == dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if _tensor(t, name).dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype} (no implicit conversion)")
    if t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be contiguous (no implicit copy)")


def _own(t, name):
    """The pointer of the tensor that the others are measured by."""
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous (no implicit copy)")
    return t.data_ptr()


def _opt(t, name, dtype, dev, shape):
    return None if t is None else _need(t, name, dtype, dev, shape)


def _rows(t, name, dtype, dev, shape):
    """(pointer, row stride) of [B, T, ...] rows with contiguous channels."""
    try:
        if len(shape) == 3 and t.dtype == dtype and t.device == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr(), shape[2]
    except AttributeError:
        pass
    if _tensor(t, name).dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype} (no implicit conversion)")
    if t.device != dev:
        raise ValueError(f"{name}: expected device {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    st, sh = t.stride(), t.shape
    width = 1
    for i in range(t.dim() - 1, 1, -1):
        if sh[i] != 1 and st[i] != width:
            raise ValueError(f"{name}: channels must be contiguous (no implicit copy)")
        width *= sh[i]
    if t.is_contiguous():
        return t.data_ptr(), width
    row = st[1] if sh[1] > 1 else st[0] if sh[0] > 1 else width
    if (sh[0] > 1 and st[0] != row * sh[1]) or row < width:
        raise ValueError(f"{name}: rows must lie one fixed stride apart (no implicit copy)")
    return t.data_ptr(), row


def _seqlens(cu, dev, B):
    """(pointer, N)"""
    if cu is None:
        return None, B
    if _tensor(cu, "cu_seqlens").dtype != torch.int64 or cu.dim() != 1 or cu.device != dev or not cu.is_contiguous():
        raise ValueError("cu_seqlens: expected a contiguous int64 vector on the tensors' device")
    return cu.data_ptr(), cu.numel() - 1


# The current stream's handle without a Stream object, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name, dev, stream, *args):
    """The library's `name` with these arguments and the stream, the tensors' device current."""
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    fn = getattr(_lib.load(), name)
    if stream is None:
        handle = _raw_stream(dev.index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _current_device() == dev.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != KDA_OK:
        _raise(status, name)


_CURRENT = nullcontext()


def _pool(stream, dev):
    """A context whose new tensors come from the memory of the stream that will write them.  A
    block of the current stream's memory may still be read by work that is queued there, which
    another stream does not wait for."""
    if stream is None:
        return _CURRENT
    if dev.type != "cuda":
        raise ValueError("expected CUDA tensors")
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def _results(stream, dev, grads):
    """Results in another stream's memory live until the current stream is done with them."""
    if stream is not None:
        here = torch.cuda.current_stream(dev)
        for t in grads.values():
            t.record_stream(here)
            _in_use(t, stream)
    return grads


def _in_use(t, stream):
    """A buffer that a caller made for a call lives until the call's stream is done with it."""
    if isinstance(stream, torch.cuda.Stream):
        t.record_stream(stream)


def _workspace(given, size, dev, stream):
    """(tensor, pointer, bytes): the caller's workspace, or one of size() bytes of the stream's
    memory (the caller of this function is within _pool)."""
    if given is None:
        if dev.type != "cuda":
            raise ValueError("expected CUDA tensors")
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise ValueError("workspace: required with a raw stream handle")
        given = torch.empty(size(), dtype=torch.uint8, device=dev)
    elif _tensor(given, "workspace").dtype != torch.uint8 or given.device != dev or not given.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the tensors' device")
    else:
        _in_use(given, stream)
    return given, given.data_ptr(), given.numel()


def _size(fn, *args):
    n = ctypes.c_size_t(0)
    st = getattr(_lib.load(), fn)(*args, ctypes.byref(n))
    if st != KDA_OK:
        _raise(st, fn)
    return n.value


def _scale_args(res_scale, dev, D):
    """(pointer of a per-channel scale or None, the number)"""
    if isinstance(res_scale, torch.Tensor):
        return _need(res_scale, "res_scale", _f32, dev, (D,)), 1.0
    return None, float(res_scale)


# ------------------------------------------------------------- convolution --
_POINTERS = [ctypes.c_void_p * k for k in range(5)]
_COUNTS = [ctypes.c_int32 * k for k in range(5)]


def _list(outs, name):
    """One to four tensors, given as one or as a sequence."""
    if isinstance(outs, torch.Tensor):
        return (outs,)
    try:
        if 1 <= len(outs) <= 4:
            return outs
    except TypeError:
        raise TypeError(f"{name}: expected a torch.Tensor or a sequence of them, got "
                        f"{type(outs).__name__}") from None
    raise ValueError(f"{name}: expected one to four tensors")


def _parts(outs, name, dtype, dev, B, T, C):
    """The pointers and channel counts of one [B, T, C] tensor or of a sequence of tensors
    [B, T, ...] that share the channels."""
    outs = _list(outs, name)
    k = len(outs)
    ptrs, counts = [], []
    for i, o in enumerate(outs):
        try:
            sh = o.shape
        except AttributeError:
            sh = _tensor(o, f"{name}[{i}]").shape
        if len(sh) < 3 or sh[0] != B or sh[1] != T:
            raise ValueError(f"{name}[{i}]: expected [{B}, {T}, ...], got {tuple(sh)}")
        if o.dtype == dtype and o.device == dev and o.is_contiguous():
            ptrs.append(o.data_ptr())
        else:
            _need(o, f"{name}[{i}]", dtype, dev, sh)
        n = sh[2]
        for m in sh[3:]:
            n *= m
        counts.append(n)
    if sum(counts) != C:
        raise ValueError(f"{name}: {sum(counts)} channels, x has {C}")
    return _POINTERS[k](*ptrs), _COUNTS[k](*counts), k


def _conv_common(x, weight, bias, activation):
    try:
        ok = x.dim() == 3 and weight.dim() == 2
    except AttributeError:
        _tensors(x=x, weight=weight)
        raise
    if not ok:
        raise ValueError("x must be [B, T, C] and weight [C, width]")
    B, T, C = x.shape
    dev = x.device
    if activation not in CONV_ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(CONV_ACTIVATIONS)}")
    W = weight.shape[1]
    return (B, T, C, W, dev, _row_dtype(x, "x"), CONV_ACTIVATIONS[activation],
            _need(weight, "weight", _f32, dev, (C, W)), _opt(bias, "bias", _f32, dev, (C,)))


def kda_conv_fwd(x, weight, bias, out, initial_state=None, final_state=None, cu_seqlens=None,
                 workspace=None, *, activation="silu", stream=None) -> None:
    """Enqueue the short causal depthwise convolution (include/kda_layer.h, kda_conv_fwd).

    x: rows [B, T, C] bf16 or fp32; weight fp32 [C, width], width 2 to 4; bias fp32 [C] or
    None; out: [B, T, C] in x's dtype, or up to four tensors [B, T, ...] that share the
    channels in order (q, k and v for kda_fwd), written.  initial_state / final_state:
    [N, width - 1, C] in x's dtype, the rows before the first and up to the last token; they
    may be one buffer.  cu_seqlens as in kda_fwd; its check is reported in `workspace`
    (uint8, 256 bytes or more) where one is given."""
    B, T, C, W, dev, dt, fn, w, b = _conv_common(x, weight, bias, activation)
    xp, xs = _rows(x, "x", x.dtype, dev, x.shape)
    ptrs, counts, k = _parts(out, "out", x.dtype, dev, B, T, C)
    cu, N = _seqlens(cu_seqlens, dev, B)
    st = (N, W - 1, C)
    ip = _opt(initial_state, "initial_state", x.dtype, dev, st)
    fp = _opt(final_state, "final_state", x.dtype, dev, st)
    wp, wb = (None, 0) if workspace is None else _workspace(workspace, None, dev, stream)[1:]
    _call("kda_conv_fwd", dev, stream, xp, xs, w, b, ptrs, counts, k, ip, fp, cu, B, T, C, N, W, fn,
          dt, wp, wb)


def make_conv_bwd_workspace(total_tokens, C, width, device=None):
    """Workspace for kda_conv_bwd."""
    return torch.empty(_size("kda_conv_bwd_get_workspace_size", int(total_tokens), int(C), int(width)),
                       dtype=torch.uint8, device=device if device is not None else "cuda")


def kda_conv_bwd(x, weight, bias, dout, initial_state=None, dfinal_state=None, cu_seqlens=None,
                 workspace=None, *, activation="silu", stream=None):
    """Enqueue the convolution's backward (include/kda_layer.h, kda_conv_bwd).  dout: as
    `out` of kda_conv_fwd, in x's dtype or fp32 (kda_bwd's dq, dk and dv as they are).
    Returns a dict: dx in x's dtype, dweight, dbias (with a bias) and dinitial_state (with
    an initial state) in fp32, and the workspace, whose status word tells of cu_seqlens."""
    B, T, C, W, dev, dt, fn, w, b = _conv_common(x, weight, bias, activation)
    xp, xs = _rows(x, "x", x.dtype, dev, x.shape)
    first = _list(dout, "dout")[0]
    ddt = _row_dtype(first, "dout")
    ptrs, counts, k = _parts(dout, "dout", first.dtype, dev, B, T, C)
    cu, N = _seqlens(cu_seqlens, dev, B)
    st = (N, W - 1, C)
    ip = _opt(initial_state, "initial_state", x.dtype, dev, st)
    dfp = _opt(dfinal_state, "dfinal_state", x.dtype, dev, st)
    with _pool(stream, dev):
        ws, wp, wb = _workspace(workspace, lambda: _size("kda_conv_bwd_get_workspace_size", B * T, C, W),
                                dev, stream)
        g = {"dx": torch.empty((B, T, C), dtype=x.dtype, device=dev),
             "dweight": torch.empty((C, W), dtype=_f32, device=dev)}
        if b is not None:
            g["dbias"] = torch.empty((C,), dtype=_f32, device=dev)
        if ip is not None:
            g["dinitial_state"] = torch.empty(st, dtype=_f32, device=dev)
    P = lambda nm: g[nm].data_ptr() if nm in g else None
    _call("kda_conv_bwd", dev, stream, xp, xs, w, b, ptrs, counts, k, ddt, ip, dfp, cu, P("dx"),
          P("dweight"), P("dbias"), P("dinitial_state"), B, T, C, N, W, fn, dt, wp, wb)
    g["workspace"] = ws
    return _results(stream, dev, g)


# --------------------------------------------------------------------- scan --
STATE_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


def _scan_problem(x, dt, A_log, B, C, D, z, dt_bias, initial_state, other_state, cu_seqlens, names):
    """The C problem of a call, and (B, T, N, D, state, groups, device)."""
    try:
        ok = x.dim() == 3 and A_log.dim() == 2 and B.dim() == 4
    except AttributeError:
        _tensors(x=x, A_log=A_log, B=B)
        raise
    if not ok:
        raise ValueError("x must be [B, T, D], A_log [D, state] and B [B, T, groups, state]")
    dev, ty = x.device, x.dtype
    q = _lib.kda_scan_problem()
    q.batch, q.T, q.dim = x.shape
    q.groups, q.state = B.shape[2:]
    q.dtype = _row_dtype(x, "x")
    d, n = q.dim, q.state
    q.x, q.x_stride = _rows(x, "x", ty, dev, x.shape)
    q.dt, q.dt_stride = _rows(dt, "dt", ty, dev, x.shape)
    if z is not None:
        q.z, q.z_stride = _rows(z, "z", ty, dev, x.shape)
    bc = torch.Size((x.shape[0], x.shape[1], q.groups, n))
    q.B, q.B_stride = _rows(B, "B", ty, dev, bc)
    q.C, q.C_stride = _rows(C, "C", ty, dev, bc)
    q.A_log = _need(A_log, "A_log", _f32, dev, (d, n))
    q.D = _opt(D, "D", _f32, dev, (d,))
    q.dt_bias = _opt(dt_bias, "dt_bias", _f32, dev, (d,))
    q.cu_seqlens, q.N = _seqlens(cu_seqlens, dev, x.shape[0])
    one = initial_state if initial_state is not None else other_state
    if one is not None:
        if _tensor(one, names[0]).dtype not in STATE_DTYPES:
            raise TypeError(f"{names[0]}: states must be float32 or bfloat16, got {one.dtype}")
        q.state_dtype = STATE_DTYPES[one.dtype]
    sty = None if one is None else one.dtype
    q.initial_state = _opt(initial_state, names[0], sty, dev, (q.N, d, n))
    return q, _opt(other_state, names[1], sty, dev, (q.N, d, n)), sty


def make_scan_states(total_tokens, N, dim, state, device=None):
    """Buffer for the states that kda_scan_fwd(..., chunk_states=buf) saves and
    kda_scan_bwd(..., chunk_states=buf) starts from."""
    return torch.empty(_size("kda_scan_get_states_size", int(total_tokens), int(N), int(dim), int(state)),
                       dtype=torch.uint8, device=device if device is not None else "cuda")


def make_scan_workspace(batch, T, dim, state, groups=1, N=None, *, backward=False,
                        have_states=False, device=None):
    """Workspace for kda_scan_fwd, or with `backward` for kda_scan_bwd (have_states: it is
    given chunk_states).  N: the number of packed sequences when cu_seqlens is used."""
    q = _lib.kda_scan_problem()
    q.batch, q.T, q.dim, q.state, q.groups, q.N = batch, T, dim, state, groups, N or batch
    if N is not None:
        q.cu_seqlens = 8  # only whether there is one counts here
    if backward:
        n = _size("kda_scan_bwd_get_workspace_size", ctypes.byref(q), int(have_states))
    else:
        n = _size("kda_scan_get_workspace_size", ctypes.byref(q))
    return torch.empty(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def _states_arg(buf, dev, stream):
    if buf is None:
        return None, 0
    if _tensor(buf, "chunk_states").dtype != torch.uint8 or buf.device != dev or not buf.is_contiguous():
        raise ValueError("chunk_states: expected make_scan_states's buffer on the tensors' device")
    _in_use(buf, stream)
    return buf.data_ptr(), buf.numel()


def kda_scan_fwd(x, dt, A_log, B, C, out, D=None, z=None, dt_bias=None, initial_state=None,
                 final_state=None, cu_seqlens=None, workspace=None, *, chunk_states=None,
                 stream=None) -> None:
    """Enqueue the selective state space scan (include/kda_layer.h, kda_scan_fwd):
    delta = softplus(dt + dt_bias), h = exp(-delta exp(A_log)) h + delta x B,
    out = (C . h + D x) silu(z).

    x, dt, z: rows [B, T, D] bf16 or fp32; B, C: rows [B, T, groups, state] in x's dtype, state
    8, 16, 32 or 64; out [B, T, D] in x's dtype, written; A_log fp32 [D, state]; D, dt_bias
    fp32 [D]; D, z and dt_bias may be None.  initial_state / final_state: [N, D, state],
    both fp32 or both bf16; they may be one buffer.  cu_seqlens as in kda_fwd, its check
    reported in `workspace` (make_scan_workspace; allocated here when None).
    chunk_states: make_scan_states's buffer, written for kda_scan_bwd."""
    q, fp, _ = _scan_problem(x, dt, A_log, B, C, D, z, dt_bias, initial_state, final_state,
                             cu_seqlens, ("initial_state", "final_state"))
    dev = x.device
    op = _need(out, "out", x.dtype, dev, x.shape)
    cp, cb = _states_arg(chunk_states, dev, stream)
    wp = wb = 0
    if workspace is not None or q.T > 8 or q.cu_seqlens or cp:
        with _pool(stream, dev):
            _, wp, wb = _workspace(workspace, lambda: _size("kda_scan_get_workspace_size", ctypes.byref(q)),
                                   dev, stream)
    _call("kda_scan_fwd", dev, stream, ctypes.byref(q), op, fp, cp, cb, wp, wb)


def kda_scan_bwd(x, dt, A_log, B, C, dout, D=None, z=None, dt_bias=None, initial_state=None,
                 dfinal_state=None, cu_seqlens=None, workspace=None, *, chunk_states=None,
                 stream=None):
    """Enqueue the scan's backward (include/kda_layer.h, kda_scan_bwd) for the forward call
    with the same inputs.  chunk_states: what that call saved; without it the states are
    computed again.  Returns a dict: dx, ddt, dB, dC (and dz) in x's dtype, dA_log (and dD,
    ddt_bias, dinitial_state, each where its input is given) in fp32, and the workspace."""
    q, dfp, _ = _scan_problem(x, dt, A_log, B, C, D, z, dt_bias, initial_state, dfinal_state,
                              cu_seqlens, ("initial_state", "dfinal_state"))
    dev, ty = x.device, x.dtype
    dop = _need(dout, "dout", ty, dev, x.shape)
    cp, cb = _states_arg(chunk_states, dev, stream)
    E = lambda shape, t=_f32: torch.empty(shape, dtype=t, device=dev)
    with _pool(stream, dev):
        ws, wp, wb = _workspace(workspace, lambda: _size("kda_scan_bwd_get_workspace_size",
                                                         ctypes.byref(q), int(cp is not None)), dev, stream)
        g = {"dx": E(x.shape, ty), "ddt": E(x.shape, ty), "dB": E(B.shape, ty), "dC": E(B.shape, ty),
             "dA_log": E(A_log.shape)}
        if z is not None:
            g["dz"] = E(x.shape, ty)
        if D is not None:
            g["dD"] = E((q.dim,))
        if dt_bias is not None:
            g["ddt_bias"] = E((q.dim,))
        if initial_state is not None:
            g["dinitial_state"] = E(initial_state.shape)
    P = lambda nm: g[nm].data_ptr() if nm in g else None
    _call("kda_scan_bwd", dev, stream, ctypes.byref(q), dop, dfp, cp, cb, P("dx"), P("ddt"), P("dz"),
          P("dB"), P("dC"), P("dA_log"), P("dD"), P("ddt_bias"), P("dinitial_state"), wp, wb)
    g["workspace"] = ws
    return _results(stream, dev, g)


# -------------------------------------------------------------------- norms --
def kda_prenorm_fwd(x, residual, weight, out, residual_out=None, *, res_scale=1.0, eps=1e-6,
                    stream=None) -> None:
    """Enqueue the norm before a block (include/kda_layer.h, kda_prenorm_fwd):
    residual_out = residual + res_scale * x, out = unit(residual_out) * weight.

    x, out: [..., D] bf16 or fp32; residual (or None) and residual_out (or None; it may be
    residual): the same shape in x's dtype or fp32; weight fp32 [D]; res_scale: a number or
    an fp32 tensor [D]."""
    dt = _row_dtype(x, "x")
    dev, D, shape = x.device, x.shape[-1], x.shape
    xp = _own(x, "x")
    stream_t = residual if residual is not None else residual_out
    sdt = dt if stream_t is None else _row_dtype(stream_t, "residual")
    sty = x.dtype if stream_t is None else stream_t.dtype
    sp, sv = _scale_args(res_scale, dev, D)
    _call("kda_prenorm_fwd", dev, stream, xp, _opt(residual, "residual", sty, dev, shape),
          _need(weight, "weight", _f32, dev, (D,)), sp, sv, eps,
          _need(out, "out", x.dtype, dev, shape),
          _opt(residual_out, "residual_out", sty, dev, shape), x.numel() // D if D else 0, D, dt, sdt)


def make_norm_bwd_workspace(rows, dim, device=None):
    """Workspace for kda_prenorm_bwd and kda_postnorm_bwd over `rows` rows of `dim` values."""
    return torch.empty(_size("kda_norm_bwd_get_workspace_size", int(rows), int(dim)),
                       dtype=torch.uint8, device=device if device is not None else "cuda")


def kda_prenorm_bwd(dout, dresidual_out, h, weight, x=None, workspace=None, *, res_scale=1.0,
                    eps=1e-6, stream=None):
    """Enqueue the backward of kda_prenorm_fwd.  h: the forward's residual_out;
    dresidual_out: its gradient from elsewhere (h's dtype) or None.  Returns a dict: dx
    (dout's dtype), dresidual (h's dtype), dweight, and with a per-channel res_scale, for
    which x is needed, dres_scale; dx is dresidual itself where they are equal (res_scale 1
    and one dtype)."""
    dt, sdt = _row_dtype(dout, "dout"), _row_dtype(h, "h")
    dev, D, shape = dout.device, dout.shape[-1], dout.shape
    sp, sv = _scale_args(res_scale, dev, D)
    if sp is not None and x is None:
        raise ValueError("x: needed for the gradient of a per-channel res_scale")
    rows = dout.numel() // D if D else 0
    same = sp is None and sv == 1.0 and dt == sdt
    with _pool(stream, dev):
        ws, wp, wb = _workspace(workspace, lambda: _size("kda_norm_bwd_get_workspace_size", rows, D), dev,
                                stream)
        g = {"dresidual": torch.empty(shape, dtype=h.dtype, device=dev),
             "dweight": torch.empty((D,), dtype=_f32, device=dev)}
        g["dx"] = g["dresidual"] if same else torch.empty(shape, dtype=dout.dtype, device=dev)
        if sp is not None:
            g["dres_scale"] = torch.empty((D,), dtype=_f32, device=dev)
    _call("kda_prenorm_bwd", dev, stream, _own(dout, "dout"),
          _opt(dresidual_out, "dresidual_out", h.dtype, dev, shape),
          _need(h, "h", h.dtype, dev, shape), _need(weight, "weight", _f32, dev, (D,)),
          None if sp is None else _need(x, "x", dout.dtype, dev, shape), sp, sv, eps,
          None if same else g["dx"].data_ptr(), g["dresidual"].data_ptr(), g["dweight"].data_ptr(),
          None if sp is None else g["dres_scale"].data_ptr(), rows, D, dt, sdt, wp, wb)
    g["workspace"] = ws
    return _results(stream, dev, g)


def _gate_args(gate, x, dev):
    """(pointer, token stride, heads) of a gate [..., D] or [B, T, H, D] rows."""
    if gate is None:
        return None, 0, 1
    if _tensor(gate, "gate").dim() == 4 and not gate.is_contiguous():
        p, st = _rows(gate, "gate", x.dtype, dev, x.shape)
        return p, st, x.shape[2]
    return _need(gate, "gate", x.dtype, dev, x.shape), x.shape[-1], 1


def kda_postnorm_fwd(x, weight, gate, out, residual=None, *, res_scale=1.0, activation="sigmoid",
                     eps=1e-6, stream=None) -> None:
    """Enqueue the norm after a block (include/kda_layer.h, kda_postnorm_fwd):
    out = residual + res_scale * unit(x) * weight * activation(gate).

    x, out, residual (or None): [..., D] bf16 or fp32, out may be x; gate: None, x's shape,
    or for x [B, T, H, D] rows whose H * D channels are contiguous; weight fp32 [D]."""
    dt = _row_dtype(x, "x")
    dev, D, shape = x.device, x.shape[-1], x.shape
    if activation not in GATE_ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(GATE_ACTIVATIONS)}")
    gp, gs, heads = _gate_args(gate, x, dev)
    sp, sv = _scale_args(res_scale, dev, D)
    _call("kda_postnorm_fwd", dev, stream, _own(x, "x"),
          _need(weight, "weight", _f32, dev, (D,)), gp, gs, heads,
          _opt(residual, "residual", x.dtype, dev, shape), sp, sv, eps,
          GATE_ACTIVATIONS[activation], _need(out, "out", x.dtype, dev, shape),
          x.numel() // D if D else 0, D, dt)


def kda_postnorm_bwd(dout, x, weight, gate=None, workspace=None, *, res_scale=1.0,
                     activation="sigmoid", eps=1e-6, stream=None):
    """Enqueue the backward of kda_postnorm_fwd; the gradient of its residual is dout.
    Returns a dict: dx, dgate (with a gate) in x's dtype, dweight, and dres_scale (with a
    per-channel res_scale) in fp32."""
    dt = _row_dtype(x, "x")
    dev, D, shape = x.device, x.shape[-1], x.shape
    if activation not in GATE_ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(GATE_ACTIVATIONS)}")
    dop = _need(dout, "dout", x.dtype, dev, shape)
    gp, gs, heads = _gate_args(gate, x, dev)
    sp, sv = _scale_args(res_scale, dev, D)
    rows = x.numel() // D if D else 0
    with _pool(stream, dev):
        ws, wp, wb = _workspace(workspace, lambda: _size("kda_norm_bwd_get_workspace_size", rows, D), dev,
                                stream)
        g = {"dx": torch.empty(shape, dtype=x.dtype, device=dev),
             "dweight": torch.empty((D,), dtype=_f32, device=dev)}
        if gate is not None:
            g["dgate"] = torch.empty(shape, dtype=x.dtype, device=dev)
        if sp is not None:
            g["dres_scale"] = torch.empty((D,), dtype=_f32, device=dev)
    _call("kda_postnorm_bwd", dev, stream, dop, _own(x, "x"),
          _need(weight, "weight", _f32, dev, (D,)), gp, gs, heads, sp, sv, eps,
          GATE_ACTIVATIONS[activation], g["dx"].data_ptr(),
          None if gate is None else g["dgate"].data_ptr(), g["dweight"].data_ptr(),
          None if sp is None else g["dres_scale"].data_ptr(), rows, D, dt, wp, wb)
    g["workspace"] = ws
    return _results(stream, dev, g)
