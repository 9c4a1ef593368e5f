"""The gated linear recurrence over batches of sequences that are whole tiles (128 rows forward,
64 backward), which are walked a tile of each in turn, over groups of 16 tiles at every
alignment of the rows, and with rows behind the last sequence; no writes beyond the results.
Every result by its values (bounds of tests/test_gpu_linrec.py) and by the norm of its error."""
import ctypes

import pytest
import torch

from tests import layer_ref as R
from tests.linrec_norm import near
from tests.linrec_ref import linrec
from tests.test_gpu_linrec import longest, make, ref_args

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
# whole tiles of both passes, of the backward only, a group's tiles in two sequences, one past a group
BATCHES = {"two": (2, 128, None), "three": (3, 256, None), "half": (2, 64, None), "halves": (3, 192, None),
           "across": (4, 1024, None), "beyond": (2, 2176, None)}
# one sequence beyond a group, and packed ones around groups, with rows behind the last
LONG = {"one": (1, 4500, None), "mixed": (1, 6500, [0, 100, 2300, 2300, 4396, 4397, 6450])}
# by TMA (bf16, fp32), lanes of two channels, of one (bf16, fp32)
KINDS = [(BF, 72), (F, 40), (BF, 66), (BF, 5), (F, 33)]


def check(kda, seq, dim, ty, saved):
    a, b, dout, dfin, cud = make(seq, dim, ty, dim + 2)
    B, T, cu = seq
    end = T if cu is None else cu[-1]
    behind = lambda v: (a["x"], a["r"], a["i"], b["z"], dout) if end < T else ()  # noqa: E731
    for v in behind(0):
        v[:, end:] = float("nan")
    N = B if cu is None else len(cu) - 1
    out = torch.full((B, T, dim), float("nan"), dtype=ty, device="cuda")
    fin = torch.full((N, dim), float("nan"), device="cuda")
    st = kda.make_linrec_states(B * T, dim) if saved else None
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud, chunk_states=st)
    got = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud, chunk_states=st)
    assert kda.kda_get_device_status(got["workspace"]) == 0
    assert out[:, end:].isnan().all()
    for v in behind(0):  # those rows count for nothing: as zeros they do so in the plain form too
        v[:, end:] = 0
    args, L = ref_args(a, b, cu), longest(seq)
    (ref, rfin), (mag, mfin) = linrec(*args), linrec(*args, mag=True)
    for nm, v, w, m in (("out", out[:, :end], ref[:, :end], mag[:, :end]), ("state", fin, rfin, mfin)):
        R.close(v, w, m, 8 * L + 64, nm)
        near(v, w, nm)
    ref, mag = linrec(*args, dout=dout, dfin=dfin), linrec(*args, dout=dout, dfin=dfin, mag=True)
    for k, v in ref.items():
        w, m, g = v, mag[k], got[k]
        if v.dim() == 3:
            assert (g[:, end:] == 0).all(), f"{k}: rows of no sequence"
            g, w, m = g[:, :end], w[:, :end], m[:, :end]
        R.close(g, w, m, 16 * L + 256 + (B * T if v.dim() == 1 else 0), k)
        near(g, w, k)


@pytest.mark.parametrize("seq", list(BATCHES))
@pytest.mark.parametrize("ty,dim", KINDS)
def test_batches_of_whole_tiles(kda_lib, seq, ty, dim):
    import kimi_delta_attention_08_gb300 as kda
    check(kda, BATCHES[seq], dim, ty, saved=seq in ("three", "across"))


@pytest.mark.parametrize("seq", list(LONG))
@pytest.mark.parametrize("ty,dim", KINDS)
@pytest.mark.parametrize("saved", [False, True])
def test_groups_of_tiles(kda_lib, seq, ty, dim, saved):
    import kimi_delta_attention_08_gb300 as kda
    check(kda, LONG[seq], dim, ty, saved)


@pytest.mark.parametrize("cu,T", [([0, 31, 50], 70), ([0, 64, 320, 320], 400), ([0, 0, 127, 128], 200)])
@pytest.mark.parametrize("ty,dim", [(BF, 64), (BF, 33), (F, 40)])
def test_rows_behind_the_last_sequence_reach_no_sum(kda_lib, cu, T, ty, dim):
    import kimi_delta_attention_08_gb300 as kda
    check(kda, (1, T, cu), dim, ty, saved=False)


def test_batches_are_their_sequences(kda_lib):
    """Sequences of a batch by themselves: the same values.  (Not the same bits: a group of tiles ends
    elsewhere, so that sums are joined in another order.)"""
    import kimi_delta_attention_08_gb300 as kda
    a, b, dout, dfin, _ = make((3, 1152, None), 128, BF, 5)
    out, fin = torch.empty_like(dout), torch.empty_like(dfin)
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin)
    g = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin)
    for n in range(3):
        one = lambda v: v[n:n + 1].contiguous()  # noqa: E731
        rows = {k: one(v) if v.dim() == 3 else v for k, v in {**a, **b}.items() if k != "initial_state"}
        o, f = one(out) * 0, one(fin) * 0
        kda.kda_linrec_fwd(**rows, out=o, initial_state=one(b["initial_state"]), final_state=f)
        h = kda.kda_linrec_bwd(**rows, dout=one(dout), initial_state=one(b["initial_state"]), dfinal_state=one(dfin))
        near(o, R.d(one(out)), "out")
        near(f, R.d(one(fin)), "state")
        for k in ("dx", "dr", "di", "dz", "dinitial_state"):
            near(h[k], R.d(one(g[k])), k)


def guarded(shape, dtype):
    """A tensor of this shape in the middle of a buffer of sevens, and a check that those stay."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 8192,), 7.0, dtype=dtype, device="cuda")

    def stays():
        return bool((buf[:4096] == 7).all() and (buf[4096 + n:] == 7).all())
    return buf[4096:4096 + n].view(shape), stays


@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("dim", [64, 66, 33])
@pytest.mark.parametrize("seq", [(3, 5, None), (2, 130, None), (1, 211, [0, 0, 1, 33, 64, 129, 200])])
def test_nothing_beyond_the_results_is_written(kda_lib, seq, dim, ty):
    import kimi_delta_attention_08_gb300 as kda
    from kimi_delta_attention_08_gb300 import layer
    a, b, dout, dfin, cud = make(seq, dim, ty, 6)
    B, T, cu = seq
    (out, ok0), (fin, ok1) = guarded((B, T, dim), ty), guarded(tuple(dfin.shape), F)
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud)
    assert ok0() and ok1()
    q, dfp = layer._linrec_problem(a["x"], a["r"], a["i"], a["A_log"], b["z"], b["r_bias"], b["i_bias"],
                                   b["initial_state"], dfin, cud, ("initial_state", "dfinal_state"), False)
    ws = kda.make_linrec_workspace(B, T, dim, None if cu is None else len(cu) - 1, backward=True)
    grads = [guarded((B, T, dim), ty) for _ in range(4)] + [guarded((dim,), F) for _ in range(3)] + [
        guarded(tuple(dfin.shape), F)]
    layer._call("kda_linrec_bwd", dout.device, None, ctypes.byref(q), dout.data_ptr(), dfp, None, 0,
                *[v.data_ptr() for v, _ in grads], ws.data_ptr(), ws.numel())
    want = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud)
    names = ("dx", "dr", "di", "dz", "dA_log", "dr_bias", "di_bias", "dinitial_state")
    for nm, (v, ok) in zip(names, grads):
        assert ok() and torch.equal(v, want[nm]), nm
