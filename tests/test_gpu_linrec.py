"""The gated linear recurrence against its 64-bit form, token by token: types, batched and
packed sequences (empty, one token, around the tiles of 64 and 128 rows and groups of 16
tiles), states in place, saved states, slices of wider rows, single tokens.

Bounds, in steps of 2^-24 of the magnitudes of tests/linrec_ref.py.  A gate's sigmoid is off
by the hardware exponential's and reciprocal's 2^-22 each (8 steps) and, for bf16 rows, by
1.5 steps for each unit of its argument, which the magnitudes hold; with the rate's 6 and
the products' roundings L is off by 16 steps of itself, a = exp(-L) by 16 L + 5.  A term that
has decayed by e^-X through t tokens carries 5 t + 16 X of them, and X e^-X < 1; joining
runs and tiles adds 3 per token at most.  sqrt(1 - a^2) adds 20 and the input's products 16.
So a state is within 8 steps per token and 64.  The backward meets such states with
gradients that carry as much, and adds over tokens: 16 per token and 256."""
import time

import pytest
import torch

from tests import layer_ref as R
from tests.linrec_ref import linrec

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
SEQS = {"one": (5, 1, None), "few": (3, 7, None), "batch": (2, 70, None), "odd": (3, 333, None),
        "packed": (1, 211, [0, 0, 1, 33, 64, 64, 128, 129, 211]), "tail": (1, 70, [0, 31, 50]),
        "tiles": (1, 650, [0, 127, 128, 130, 512, 512, 650]), "ends": (1, 400, [0, 64, 320, 320])}
# past a group of 16 tiles of 128 (forward) and of 64 rows (backward), aligned and not
LONG = {"group": (1, 2048 + 64, None), "groups": (2, 4500, None),
        "mixed": (1, 6500, [0, 100, 2300, 2300, 4396, 4397, 6450])}


def make(seq, dim, ty, seed=0, wide=0, sty=F):
    B, T, cu = seq
    g = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    r = lambda *s, t=ty, k=1.0: (torch.randn(*s, generator=g) * k).to(t).cuda()  # noqa: E731
    rows = lambda: r(B, T, dim + wide)[..., wide:]  # noqa: E731
    a0 = 0.9 + 0.099 * torch.rand(dim, generator=g)
    a = dict(x=rows(), r=rows(), i=rows(), A_log=torch.log(-8 * torch.log(a0)).cuda())
    b = dict(z=rows(), r_bias=r(dim, t=F), i_bias=r(dim, t=F), initial_state=r(N, dim, t=sty))
    return a, b, r(B, T, dim), r(N, dim, t=sty), None if cu is None else torch.tensor(cu, device="cuda")


def longest(seq):
    B, T, cu = seq
    return T if cu is None else max(q - p for p, q in zip(cu[:-1], cu[1:]))


def ref_args(a, b, cu):
    return (a["x"], a["r"], a["i"], a["A_log"], b["z"], b["r_bias"], b["i_bias"], b["initial_state"], cu)


def check_fwd(kda, seq, dim, ty, drop=(), wide=0, sty=F, saved=False, workspace=True):
    a, b, _, _, cud = make(seq, dim, ty, dim, wide, sty)
    B, T, cu = seq
    N = B if cu is None else len(cu) - 1
    for k in drop:
        b[k] = None
    out = torch.full((B, T, dim), float("nan"), dtype=ty, device="cuda")
    fin = torch.full((N, dim), float("nan"), dtype=sty, device="cuda")
    ws = kda.make_linrec_workspace(B, T, dim, N if cu else None) if workspace else None
    if ws is not None:
        ws.fill_(0x5A)  # a workspace may hold anything
    st = kda.make_linrec_states(B * T, dim) if saved else None
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud, workspace=ws, chunk_states=st)
    if ws is not None:
        assert kda.kda_get_device_status(ws) == 0
    ref, rfin = linrec(*ref_args(a, b, cu))
    mag, mfin = linrec(*ref_args(a, b, cu), mag=True)
    steps = 8 * longest(seq) + 64
    end = T if cu is None else cu[-1]
    R.close(out[:, :end], ref[:, :end], mag[:, :end], steps, "out")
    assert out[:, end:].isnan().all(), "rows of no sequence were written"
    R.close(fin, rfin, mfin, steps, "final_state")
    return a, b, cud, out, fin


@pytest.mark.parametrize("seq", list(SEQS))
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("dim", [1, 33, 64, 130])
def test_forward(kda_lib, seq, ty, dim):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, SEQS[seq], dim, ty)


@pytest.mark.parametrize("seq", list(LONG))
@pytest.mark.parametrize("ty,dim", [(BF, 66), (BF, 5), (F, 40)])
def test_forward_over_many_tiles(kda_lib, seq, ty, dim):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, LONG[seq], dim, ty, saved=True)


@pytest.mark.parametrize("drop", [("z",), ("r_bias",), ("i_bias",), ("initial_state",),
                                  ("z", "r_bias", "i_bias", "initial_state")])
@pytest.mark.parametrize("seq", ["few", "packed"])
def test_forward_parts_left_out(kda_lib, drop, seq):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, SEQS[seq], 64, BF, drop=drop)


@pytest.mark.parametrize("wide", [64, 3])
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("seq", ["one", "batch", "packed"])
def test_forward_slices(kda_lib, wide, ty, seq):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, SEQS[seq], 64, ty, wide=wide)


@pytest.mark.parametrize("seq", ["one", "few", "batch", "packed"])
@pytest.mark.parametrize("dim", [64, 7])
def test_bf16_states(kda_lib, seq, dim):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, SEQS[seq], dim, BF, sty=BF)


@pytest.mark.parametrize("seq", ["one", "few", "batch", "packed", "tiles"])
def test_state_in_place(kda_lib, seq):
    import kimi_delta_attention_08_gb300 as kda
    a, b, cud, out, fin = check_fwd(kda, SEQS[seq], 48, BF)
    st, o = b["initial_state"].clone(), torch.full_like(out, float("nan"))
    kda.kda_linrec_fwd(**a, out=o, **{**b, "initial_state": st}, final_state=st, cu_seqlens=cud)
    assert torch.equal(st, fin)
    assert torch.equal(o.nan_to_num(nan=7.0), out.nan_to_num(nan=7.0))


@pytest.mark.parametrize("sty", [F, BF])
@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("T", [1, 9])
def test_states_anywhere(kda_lib, T, off, sty):
    """States that begin at any element of a buffer, next to values that stay."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, _, _, _ = make((3, T, None), 64, BF, 4, sty=sty)
    buf = [torch.full((3 * 64 + 16,), 7.0, dtype=sty, device="cuda") for _ in range(2)]
    init, fin = (v[off:off + 192].view(3, 64) for v in buf)
    init.copy_(b["initial_state"])
    out, want, wfin = (torch.empty_like(a["x"]), torch.empty_like(a["x"]), torch.empty_like(b["initial_state"]))
    kda.kda_linrec_fwd(**a, out=want, **b, final_state=wfin)
    kda.kda_linrec_fwd(**a, out=out, **{**b, "initial_state": init}, final_state=fin)
    assert torch.equal(out, want) and torch.equal(fin, wfin)
    assert (buf[1][:off] == 7).all() and (buf[1][off + 192:] == 7).all()


def test_tokens_one_at_a_time(kda_lib):
    """Carried states: a prompt, then single tokens, against the whole sequence at once."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, _, _, _ = make((2, 140, None), 66, F, 3)
    ref, rfin = linrec(*ref_args(a, b, None))
    mag, mfin = linrec(*ref_args(a, b, None), mag=True)
    st = b["initial_state"].clone()
    cuts = [0, 129, 130, 131, 133, 140]
    for p, q in zip(cuts, cuts[1:]):
        part = lambda v: v[:, p:q].contiguous()  # noqa: E731
        o = torch.empty(2, q - p, 66, device="cuda")
        kda.kda_linrec_fwd(part(a["x"]), part(a["r"]), part(a["i"]), a["A_log"], o, part(b["z"]),
                           b["r_bias"], b["i_bias"], st, st)
        R.close(o, ref[:, p:q], mag[:, p:q], 8 * q + 64, f"tokens {p} to {q}")
    R.close(st, rfin, mfin, 8 * 140 + 64, "state")


GRADS = {"dx": "x", "dr": "r", "di": "i", "dz": "z", "dr_bias": "r_bias", "di_bias": "i_bias",
         "dinitial_state": "initial_state"}


def check_bwd(kda, seq, dim, ty, drop=(), wide=0, sty=F, saved=False, dfinal=True):
    a, b, dout, dfin, cud = make(seq, dim, ty, dim + 1, wide, sty)
    B, T, cu = seq
    N = B if cu is None else len(cu) - 1
    for k in drop:
        b[k] = None
    dfin = dfin if dfinal else None
    end = T if cu is None else cu[-1]
    if end < T:  # what lies behind the last sequence counts for nothing
        for v in (a["x"], a["r"], a["i"], dout) + (() if b["z"] is None else (b["z"],)):
            v[:, end:] = float("nan")
    st = None
    if saved:
        st = kda.make_linrec_states(B * T, dim)
        kda.kda_linrec_fwd(**a, out=torch.empty_like(dout), **b, cu_seqlens=cud, chunk_states=st)
    ws = kda.make_linrec_workspace(B, T, dim, N if cu else None, backward=True, have_states=saved)
    ws.fill_(0x5A)
    got = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud, workspace=ws,
                             chunk_states=st)
    assert kda.kda_get_device_status(ws) == 0
    ref = linrec(*ref_args(a, b, cu), dout=dout, dfin=dfin)
    mag = linrec(*ref_args(a, b, cu), dout=dout, dfin=dfin, mag=True)
    L = longest(seq)
    for k, v in ref.items():
        if k in GRADS and GRADS[k] in drop:
            assert k not in got
            continue
        summed = v.dim() == 1
        if v.dim() == 3 and end < T:
            assert (got[k][:, end:] == 0).all(), f"{k}: rows of no sequence"
            R.close(got[k][:, :end], v[:, :end], mag[k][:, :end], 16 * L + 256, k)
        else:
            if end < T and summed:  # the plain form's own rows there are NaN
                continue
            R.close(got[k], v, mag[k], 16 * L + 256 + (B * T if summed else 0), k)
    return got


@pytest.mark.parametrize("seq", list(SEQS))
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("dim", [1, 33, 64, 130])
def test_backward(kda_lib, seq, ty, dim):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, SEQS[seq], dim, ty, saved=dim == 64)


@pytest.mark.parametrize("seq", list(LONG))
@pytest.mark.parametrize("ty,dim", [(BF, 66), (BF, 5), (F, 40)])
@pytest.mark.parametrize("saved", [False, True])
def test_backward_over_many_tiles(kda_lib, seq, ty, dim, saved):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, LONG[seq], dim, ty, saved=saved)


@pytest.mark.parametrize("drop", [("z",), ("r_bias",), ("i_bias",), ("initial_state",),
                                  ("z", "r_bias", "i_bias", "initial_state")])
@pytest.mark.parametrize("seq", ["few", "packed"])
def test_backward_parts_left_out(kda_lib, drop, seq):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, SEQS[seq], 64, BF, drop=drop, dfinal="z" not in drop)


@pytest.mark.parametrize("wide", [64, 3])
@pytest.mark.parametrize("ty", [BF, F])
def test_backward_slices(kda_lib, wide, ty):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, SEQS["tiles"], 64, ty, wide=wide)


def test_backward_bf16_states(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, SEQS["packed"], 64, BF, sty=BF)


@pytest.mark.parametrize("T,cu", [(0, None), (0, [0, 0, 0]), (5, [0, 0, 0])])
def test_no_tokens(kda_lib, T, cu):
    import kimi_delta_attention_08_gb300 as kda
    B, D = (2, 40) if cu is None else (1, 40)
    a, b, dout, dfin, cud = make((B, T, cu), D, BF, 1)
    out, fin = torch.empty_like(dout), torch.full_like(dfin, 9.0)
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud)
    assert torch.equal(fin, b["initial_state"])
    g = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud)
    assert torch.equal(g["dinitial_state"], dfin)
    for k in ("dA_log", "dr_bias", "di_bias", "dx", "dr", "di", "dz"):
        assert (g[k] == 0).all(), k


@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("T", [3, 200])
def test_extreme_gates(kda_lib, ty, T):
    """Gates far out on both sides, decay rates of zero and infinity, tiny steps: 1 - a^2 and
    the slopes keep their digits, and what is finite in 64 bits stays finite.  The magnitudes
    count the arguments."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(5)
    vals = torch.tensor([-60.0, -30.0, -17.0, -9.0, -3.0, 0.0, 3.0, 9.0, 17.0, 30.0, 60.0])
    pick = lambda *s: vals[torch.randint(len(vals), s, generator=g)].to(ty).cuda()  # noqa: E731
    D = 64
    a = dict(x=torch.randn(2, T, D, generator=g).to(ty).cuda(), r=pick(2, T, D), i=pick(2, T, D),
             A_log=torch.linspace(-30, 4, D).cuda())
    b = dict(z=pick(2, T, D), r_bias=None, i_bias=None, initial_state=torch.randn(2, D, generator=g).cuda())
    out, fin = torch.empty_like(a["x"]), torch.empty(2, D, device="cuda")
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin)
    ref, rfin = linrec(*ref_args(a, b, None))
    mag, mfin = linrec(*ref_args(a, b, None), mag=True)
    R.close(out, ref, mag, 8 * T + 64, "out")
    R.close(fin, rfin, mfin, 8 * T + 64, "final_state")
    dout = torch.randn(2, T, D, generator=g).to(ty).cuda()
    got = kda.kda_linrec_bwd(**a, dout=dout, **b)
    ref = linrec(*ref_args(a, b, None), dout=dout)
    mag = linrec(*ref_args(a, b, None), dout=dout, mag=True)
    for k in ref:
        if k in got:
            R.close(got[k], ref[k], mag[k], 16 * T + 256 + (2 * T if ref[k].dim() == 1 else 0), k)


def test_rates_of_zero_and_infinity(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    D, T = 8, 150
    x = torch.ones(1, T, D, device="cuda")
    A = torch.full((D,), -float("inf"), device="cuda")
    A[4:] = float("inf")
    init, out, fin = torch.full((1, D), 3.0, device="cuda"), torch.empty_like(x), torch.empty(1, D, device="cuda")
    kda.kda_linrec_fwd(x, x, x, A, out, initial_state=init, final_state=fin)
    assert (out[..., :4] == 3).all() and (fin[:, :4] == 3).all()      # nothing decays, nothing enters
    s = torch.sigmoid(torch.ones((), dtype=torch.float64)).item()
    assert (out[..., 4:].double() - s).abs().max() < 1e-6             # nothing is kept
    g = kda.kda_linrec_bwd(x, x, x, A, x, initial_state=init)
    for k in ("dx", "dr", "di", "dA_log", "dinitial_state"):
        assert g[k].isfinite().all(), k


@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("T", [3, 200])
def test_infinite_gates(kda_lib, ty, T):
    """Gates of plus and minus infinity are 1 and 0 exactly; an input gate that is NaN makes NaN from
    its row on."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(6)
    inf = float("inf")
    pick = lambda *s: torch.tensor([-inf, inf])[torch.randint(2, s, generator=g)].to(ty).cuda()  # noqa: E731
    D = 64
    x, r, i = torch.randn(1, T, D, generator=g).to(ty).cuda(), pick(1, T, D), pick(1, T, D)
    A = torch.linspace(-3, 2, D).cuda()
    out = torch.empty_like(x)
    kda.kda_linrec_fwd(x, r, i, A, out)
    L = torch.exp(A.double().cpu()) * (r.double().cpu() > 0)
    a, b = torch.exp(-L), torch.sqrt(1 - torch.exp(-2 * L)) * (i.double().cpu() > 0) * x.double().cpu()
    h, want, mag, m = torch.zeros(D, dtype=torch.float64), [], [], torch.zeros(D, dtype=torch.float64)
    for t in range(T):
        h, m = a[0, t] * h + b[0, t], a[0, t] * m + b[0, t].abs()
        want.append(h), mag.append(m)
    # 2^-21 of a factor at most: as many steps for each token as in the other tests
    R.close(out, torch.stack(want)[None], torch.stack(mag)[None], 8 * T + 64, "out")
    i[0, T // 2] = float("nan")
    kda.kda_linrec_fwd(x, r, i, A, out)
    assert out[0, T // 2:].isnan().all() and out[0, :T // 2].isfinite().all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_sequence_and_channel(kda_lib, bad):
    import kimi_delta_attention_08_gb300 as kda
    cu, D = [0, 90, 91, 300, 430], 64
    a, b, dout, dfin, cud = make((1, 430, cu), D, BF, 2)
    run = lambda: (torch.empty_like(dout), torch.empty_like(dfin))  # noqa: E731
    want, wfin = run()
    kda.kda_linrec_fwd(**a, out=want, **b, final_state=wfin, cu_seqlens=cud)
    wg = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud)
    a["x"][0, 150, 7] = bad
    out, fin = run()
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud)
    g = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud)
    assert not out[0, 150:300, 7].isfinite().any() and not fin[2, 7].isfinite()
    keep = torch.ones(430, D, dtype=torch.bool, device="cuda")
    keep[91:300, 7] = False
    for got, ref in [(out, want)] + [(g[k], wg[k]) for k in ("dx", "dr", "di", "dz")]:
        assert torch.equal(got[0][keep], ref[0][keep])
    only = torch.arange(D, device="cuda") != 7
    assert torch.equal(fin[:, only], wfin[:, only]) and torch.equal(g["dA_log"][only], wg["dA_log"][only])


def many(kind):
    """More sequences than are searched one by one: single tokens; short and empty ones; runs of empty
    ones longer than what a warp looks at, between some long ones; rows behind the last."""
    g = torch.Generator().manual_seed(8)
    if kind == "tokens":
        n = [1] * 300
    elif kind == "short":
        n = torch.randint(0, 6, (400,), generator=g).tolist()
    else:
        n = ([0] * 40 + [3] + [0] * 70 + [130, 1, 0, 2]) * 4
    cu = [0]
    for v in n:
        cu.append(cu[-1] + v)
    return 1, cu[-1] + (9 if kind == "empty" else 0), cu


@pytest.mark.parametrize("ty,dim", [(BF, 64), (BF, 37), (F, 40)])
@pytest.mark.parametrize("kind", ["tokens", "short", "empty"])
def test_many_sequences(kda_lib, kind, ty, dim):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, many(kind), dim, ty)
    check_bwd(kda, many(kind), dim, ty)


def test_many_bad_sequences_are_reported(kda_lib):
    """Bounds out of order, beyond the rows or below zero, among many: a status, nothing out of range."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(9)
    for cu in ([0] + torch.randint(-50, 400, (200,), generator=g).tolist(), [0] * 100 + [500] * 100, list(range(150, -1, -1))):
        a, b, dout, _, cud = make((1, 200, cu), 64, BF, 2)
        ws = kda.make_linrec_workspace(1, 200, 64, len(cu) - 1)
        fin = torch.empty(len(cu) - 1, 64, device="cuda")
        kda.kda_linrec_fwd(**a, out=torch.empty_like(dout), **b, final_state=fin, cu_seqlens=cud, workspace=ws)
        assert kda.kda_get_device_status(ws) == 9
        g2 = kda.kda_linrec_bwd(**a, dout=dout, **b, cu_seqlens=cud)
        assert kda.kda_get_device_status(g2["workspace"]) == 9


def test_bad_sequences_are_reported(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    for cu in ([0, 50, 40, 200], [3, 50, 200], [0, 50, 300], [0, -5, 200]):
        a, b, dout, _, cud = make((1, 200, cu), 64, BF, 2)
        ws = kda.make_linrec_workspace(1, 200, 64, len(cu) - 1)
        fin = torch.empty(len(cu) - 1, 64, device="cuda")
        kda.kda_linrec_fwd(**a, out=torch.empty_like(dout), **b, final_state=fin, cu_seqlens=cud, workspace=ws)
        assert kda.kda_get_device_status(ws) == 9, cu
        g = kda.kda_linrec_bwd(**a, dout=dout, **b, cu_seqlens=cud)
        assert kda.kda_get_device_status(g["workspace"]) == 9, cu


def test_a_wait_that_runs_out_is_reported(kda_lib):
    """The first tile's result is never handed on: the tiles behind it give up."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, dout, _, _ = make((1, 700, None), 64, BF, 2)
    out = torch.empty_like(dout)
    ws = kda.make_linrec_workspace(1, 700, 64)
    t0 = time.time()
    kda.kda_linrec_fwd(**a, out=out, **b, workspace=ws, debug_stall=True)
    assert kda.kda_get_device_status(ws) == 8
    g = kda.kda_linrec_bwd(**a, dout=dout, **b, debug_stall=True)
    assert kda.kda_get_device_status(g["workspace"]) == 8
    assert time.time() - t0 < 10
    check_bwd(kda, (1, 700, None), 64, BF)


def test_runs_are_the_same_bits(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    a, b, dout, dfin, cud = make((1, 9000, [0, 8000, 8001, 9000]), 1024, BF, 2)
    first = None
    for _ in range(5):
        out, fin = torch.empty_like(dout), torch.empty_like(dfin)
        kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud)
        g = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud)
        now = [out, fin] + [g[k] for k in sorted(g) if k != "workspace"]
        first = first or now
        assert all(torch.equal(p, q) for p, q in zip(first, now))


def test_captured_with_a_shared_workspace(kda_lib):
    """Two captured graphs that share a workspace, replayed in turn on new inputs."""
    import kimi_delta_attention_08_gb300 as kda
    D, T = 128, 700
    ws = kda.make_linrec_workspace(2, T, D, backward=True)
    sets = []
    for seed in (1, 2):
        a, b, dout, dfin, _ = make((2, T, None), D, BF, seed)
        out, fin = torch.empty_like(dout), torch.empty_like(dfin)

        def step(a=a, b=b, dout=dout, dfin=dfin, out=out, fin=fin):
            kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, workspace=ws)
            return kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, workspace=ws)
        step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            g = step()
        sets.append((a, b, dout, dfin, out, fin, g, gr, step))
    for _ in range(2):
        for s in sets:
            s[0]["x"].copy_(torch.randn_like(s[0]["x"]))
        for s in sets:
            s[7].replay()
        torch.cuda.synchronize()
        for a, b, dout, dfin, out, fin, g, gr, step in sets:
            kept = [out.clone(), fin.clone()] + [g[k].clone() for k in sorted(g) if k != "workspace"]
            g2 = step()
            for p, q in zip(kept, [out, fin] + [g2[k] for k in sorted(g2) if k != "workspace"]):
                assert torch.equal(p, q)


def test_offsets_beyond_32_bits(kda_lib):
    """Rows whose offsets pass 2^31 elements and 2^32 bytes."""
    import kimi_delta_attention_08_gb300 as kda
    T, D, wide = 3000, 64, 1 << 20
    base = torch.zeros(T * wide, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    x = base.view(1, T, wide)[..., 64:64 + D]
    vals = torch.randn(1, T, D, generator=g).to(BF).cuda()
    x.copy_(vals)
    A, out, ref = torch.zeros(D, device="cuda"), torch.empty_like(vals), torch.empty_like(vals)
    kda.kda_linrec_fwd(x, x, x, A, out)
    kda.kda_linrec_fwd(vals, vals, vals, A, ref)
    assert torch.equal(out, ref)
