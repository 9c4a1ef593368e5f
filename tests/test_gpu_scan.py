"""The selective state space scan against its 64-bit form, token by token: state sizes,
types, groups, batched and packed sequences (empty, one token, around the 32-token block),
sequences cut into segments, states in place, saved states, slices of wider rows.

Bounds, in steps of 2^-24 of the magnitudes of tests/layer_ref.py.  A step's decay
2^(delta A2) is off by the exponential's 2^-22 and by its argument's roundings and
delta's, 13 |arg| at most; a term that has decayed by e^-X through t steps carries
4 t + 13 X of them, and X e^-X < 1, so a state is within 6 steps per token and 32 in all.
The backward meets such states with gradients that carry as much, and adds over tokens:
16 per token."""
import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
SEQS = {"one": (5, 1, None), "few": (3, 7, None), "batch": (2, 70, None),
        "packed": (1, 211, [0, 0, 1, 33, 65, 65, 129, 211]), "tail": (1, 70, [0, 31, 50])}


def make(seq, dim, n, G, ty, seed=0, wide=0, sty=F):
    B, T, cu = SEQS[seq] if isinstance(seq, str) else seq
    g = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    r = lambda *s, t=ty, k=1.0: (torch.randn(*s, generator=g) * k).to(t).cuda()  # noqa: E731

    def rows(*s):
        if not wide:
            return r(*s)
        flat = 1
        for k in s[2:]:
            flat *= k
        return r(s[0], s[1], flat + wide)[..., wide:].unflatten(2, s[2:])
    a = dict(x=rows(B, T, dim), dt=rows(B, T, dim),
             A_log=(torch.log(torch.arange(1, n + 1.0)) + 0.1 * torch.randn(dim, n, generator=g)).cuda(),
             B=rows(B, T, G, n), C=rows(B, T, G, n))
    b = dict(D=r(dim, t=F), z=rows(B, T, dim), dt_bias=r(dim, t=F) - 3, initial_state=r(N, dim, n, t=sty))
    c = dict(dout=r(B, T, dim), dfin=r(N, dim, n, t=sty))
    return a, b, c, cu, None if cu is None else torch.tensor(cu, device="cuda"), (B, T, N)


def longest(seq):
    B, T, cu = SEQS[seq] if isinstance(seq, str) else seq
    return T if cu is None else max(q - p for p, q in zip(cu[:-1], cu[1:]))


def ref_args(a, b, cu):
    return (a["x"], a["dt"], a["A_log"], a["B"], a["C"], b["D"], b["z"], b["dt_bias"],
            b["initial_state"], cu)


def check_fwd(kda, seq, dim, n, G, ty, drop=(), wide=0, sty=F, saved=False):
    a, b, _, cu, cud, (B, T, N) = make(seq, dim, n, G, ty, dim + n, wide, sty)
    for k in drop:
        b[k] = None
    out = torch.full((B, T, dim), float("nan"), dtype=ty, device="cuda")
    fin = torch.full((N, dim, n), float("nan"), dtype=sty, device="cuda")
    ws = kda.make_scan_workspace(B, T, dim, n, G, N if cu else None)
    st = kda.make_scan_states(B * T, N, dim, n) if saved else None
    kda.kda_scan_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud, workspace=ws, chunk_states=st)
    assert kda.kda_get_device_status(ws) == 0
    ref, rfin = R.scan(*ref_args(a, b, cu))
    mag, mfin = R.scan(*ref_args(a, b, cu), mag=True)
    steps = 6 * longest(seq) + 64
    end = T if cu is None else cu[-1]
    R.close(out[:, :end], ref[:, :end], mag[:, :end], steps, "out")
    assert out[:, end:].isnan().all(), "rows of no sequence were written"
    R.close(fin, rfin, mfin, steps, "final_state")
    return a, b, cud, out, fin


@pytest.mark.parametrize("seq", list(SEQS))
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("dim,n,G", [(64, 16, 1), (33, 16, 1), (48, 8, 2), (128, 32, 4), (40, 64, 1), (7, 8, 7)])
def test_forward(kda_lib, seq, ty, dim, n, G):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, seq, dim, n, G, ty)


@pytest.mark.parametrize("drop", [("D",), ("z",), ("dt_bias",), ("initial_state",),
                                  ("D", "z", "dt_bias", "initial_state")])
@pytest.mark.parametrize("seq", ["few", "packed"])
def test_forward_parts_left_out(kda_lib, drop, seq):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, seq, 64, 16, 1, BF, drop=drop)


@pytest.mark.parametrize("wide", [64, 3])
@pytest.mark.parametrize("seq", ["one", "batch"])
def test_forward_slices(kda_lib, wide, seq):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, seq, 64, 16, 2, BF, wide=wide)


@pytest.mark.parametrize("seq", ["one", "few", "batch", "packed"])
def test_bf16_states(kda_lib, seq):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, seq, 64, 16, 1, BF, sty=BF)


# long enough that the few channels are cut into segments of 256 tokens and more
SPLIT = {"batched": (2, 600, None), "packed": (1, 1400, [0, 257, 257, 258, 1300, 1400]),
         "exact": (1, 1024, [0, 512, 1024])}


@pytest.mark.parametrize("seq", list(SPLIT))
@pytest.mark.parametrize("n,G", [(16, 1), (64, 2)])
def test_forward_cut_into_segments(kda_lib, seq, n, G):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, SPLIT[seq], 16, n, G, F, saved=True)


@pytest.mark.parametrize("seq", ["one", "few", "batch", "packed", SPLIT["packed"]])
def test_state_in_place(kda_lib, seq):
    import kimi_delta_attention_08_gb300 as kda
    a, b, cud, out, fin = check_fwd(kda, seq, 48, 16, 1, BF)
    st, o = b["initial_state"].clone(), torch.full_like(out, float("nan"))
    kda.kda_scan_fwd(**a, out=o, **{**b, "initial_state": st}, final_state=st, cu_seqlens=cud)
    assert torch.equal(st, fin) and torch.equal(o.view(torch.int16), out.view(torch.int16))


def test_steps_equal_a_prompt(kda_lib):
    """Token by token with the state carried in place, against one call over the prompt:
    the same recurrence, in another order of the dot product's additions."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, _, _, _, (B, T, N) = make("batch", 96, 16, 1, F, 5)
    out, fin = torch.empty_like(a["x"]), torch.empty_like(b["initial_state"])
    kda.kda_scan_fwd(**a, out=out, **b, final_state=fin)
    st, got = b["initial_state"].clone(), torch.empty_like(out)
    cut = lambda v, t: v[:, t:t + 1]  # noqa: E731
    for t in range(T):
        o = torch.empty(B, 1, 96, device="cuda")
        step = {k: (cut(v, t) if k != "A_log" else v) for k, v in a.items()}
        kda.kda_scan_fwd(**step, out=o, **{**b, "z": cut(b["z"], t), "initial_state": st}, final_state=st)
        got[:, t:t + 1] = o
    mag, mfin = R.scan(*ref_args(a, b, None), mag=True)
    R.close(st, R.d(fin), mfin, 16, "state")
    R.close(got, R.d(out), mag, 16, "out")


GRADS = ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias", "dinitial_state")


def check_bwd(kda, seq, dim, n, G, ty, drop=(), wide=0, saved=False, sty=F):
    a, b, c, cu, cud, (B, T, N) = make(seq, dim, n, G, ty, dim + n + 1, wide, sty)
    for k in drop:
        if k in c:
            c[k] = None
        else:
            b[k] = None
    st = None
    if saved:
        st = kda.make_scan_states(B * T, N, dim, n)
        out = torch.empty(B, T, dim, dtype=ty, device="cuda")
        kda.kda_scan_fwd(**a, out=out, **b, cu_seqlens=cud, chunk_states=st)
    g = kda.kda_scan_bwd(**a, dout=c["dout"], **b, dfinal_state=c["dfin"], cu_seqlens=cud, chunk_states=st)
    assert kda.kda_get_device_status(g["workspace"]) == 0
    ref = R.scan(*ref_args(a, b, cu), dout=c["dout"], dfin=c["dfin"])
    mag = R.scan(*ref_args(a, b, cu), dout=c["dout"], dfin=c["dfin"], mag=True)
    left = {"dD": "D", "dz": "z", "ddt_bias": "dt_bias", "dinitial_state": "initial_state"}
    names = [k for k in GRADS if b.get(left.get(k, ""), 0) is not None]
    assert set(names) == set(g) - {"workspace"}
    for nm in names:
        steps = 16 * longest(seq) + 256 + (B * T if nm in ("dA_log", "dD", "ddt_bias") else 0)
        R.close(g[nm], ref[nm], mag[nm], steps, nm)
    return g


@pytest.mark.parametrize("seq", list(SEQS))
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("dim,n,G", [(64, 16, 1), (33, 16, 1), (48, 8, 2), (128, 32, 4), (40, 64, 1),
                                     (200, 16, 1), (7, 8, 7)])
def test_backward(kda_lib, seq, ty, dim, n, G):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, seq, dim, n, G, ty)


@pytest.mark.parametrize("drop", [("D",), ("z",), ("dt_bias",), ("initial_state",), ("dfin",),
                                  ("D", "z", "dt_bias", "initial_state", "dfin")])
def test_backward_parts_left_out(kda_lib, drop):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, "packed", 64, 16, 1, BF, drop=drop)


@pytest.mark.parametrize("wide", [64, 3])
def test_backward_slices(kda_lib, wide):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, "batch", 64, 16, 2, BF, wide=wide)


@pytest.mark.parametrize("seq", list(SPLIT))
@pytest.mark.parametrize("n,G", [(16, 1), (64, 2)])
def test_backward_cut_into_segments(kda_lib, seq, n, G):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, SPLIT[seq], 16, n, G, F)


@pytest.mark.parametrize("seq", ["packed", SPLIT["packed"]])
def test_backward_with_saved_states(kda_lib, seq):
    """The forward's saved states give the bits of the recomputed ones, and every run the
    same bits."""
    import kimi_delta_attention_08_gb300 as kda
    g = [check_bwd(kda, seq, 72, 16, 1, BF, saved=s) for s in (True, False, True)]
    for nm in GRADS:
        assert torch.equal(g[0][nm], g[1][nm]) and torch.equal(g[0][nm], g[2][nm]), nm


def test_many_sequences(kda_lib):
    """More sequences than one search step tells apart, from empty to longer than a segment."""
    import itertools
    import kimi_delta_attention_08_gb300 as kda
    cu = list(itertools.accumulate([(7 * i * i + 3 * i) % 41 if i % 50 else 300 for i in range(120)], initial=0))
    check_fwd(kda, (1, cu[-1] + 5, cu), 24, 16, 1, F, saved=True)
    check_bwd(kda, (1, cu[-1] + 5, cu), 24, 16, 1, F)


def test_bf16_state_gradients(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, "packed", 64, 16, 1, BF, sty=BF)


def test_extreme_steps(kda_lib):
    """Steps from none at all (dt far below zero: the state stays) to large ones (the state
    is forgotten): finite everywhere and within the bounds."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, c, cu, _, (B, T, N) = make("batch", 64, 16, 1, F, 3)
    a["dt"][:, :20] = -200.0
    a["dt"][:, 20:40] = 80.0
    out, fin = torch.empty_like(a["x"]), torch.empty_like(b["initial_state"])
    kda.kda_scan_fwd(**a, out=out, **b, final_state=fin)
    ref, rfin = R.scan(*ref_args(a, b, None))
    mag, mfin = R.scan(*ref_args(a, b, None), mag=True)
    R.close(out, ref, mag, 6 * T + 64, "out")
    R.close(fin, rfin, mfin, 6 * T + 64, "final_state")
    g = kda.kda_scan_bwd(**a, dout=c["dout"], **b, dfinal_state=c["dfin"])
    ref = R.scan(*ref_args(a, b, None), dout=c["dout"], dfin=c["dfin"])
    mag = R.scan(*ref_args(a, b, None), dout=c["dout"], dfin=c["dfin"], mag=True)
    for nm in GRADS:
        R.close(g[nm], ref[nm], mag[nm], 17 * T + 256, nm)


@pytest.mark.parametrize("seq", ["one", "batch", SPLIT["packed"]])
def test_steps_of_zero_keep_the_state(kda_lib, seq):
    """softplus(-200) is 0 in fp32: every decay is exactly 1 and nothing is added."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, _, cu, cud, (B, T, N) = make(seq, 64, 16, 1, BF)
    a["dt"].fill_(-200.0)
    out = torch.empty(B, T, 64, dtype=BF, device="cuda")
    fin = torch.full((N, 64, 16), float("nan"), device="cuda")
    ws = kda.make_scan_workspace(B, T, 64, 16, 1, N if cu else None)
    kda.kda_scan_fwd(**a, out=out, **b, final_state=fin, cu_seqlens=cud, workspace=ws)
    assert torch.equal(fin, b["initial_state"])


@pytest.mark.parametrize("seq", ["one", "batch"])
@pytest.mark.parametrize("v", [-float("inf"), 100.0, 300.0])
def test_rates_of_zero_and_infinity(kda_lib, seq, v):
    """exp(A_log) of 0 keeps a state for ever, one of infinity forgets it at each step."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, _, cu, _, (B, T, N) = make(seq, 64, 16, 1, F)
    a["A_log"][:, ::2] = v
    out = torch.empty(B, T, 64, device="cuda")
    fin = torch.empty(N, 64, 16, device="cuda")
    kda.kda_scan_fwd(**a, out=out, **b, final_state=fin)
    ref, rfin = R.scan(*ref_args(a, b, cu))
    mag, mfin = R.scan(*ref_args(a, b, cu), mag=True)
    R.close(out, ref, mag, 6 * T + 64, "out")
    R.close(fin, rfin, mfin, 6 * T + 64, "final_state")


def test_no_tokens(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    a, b, c, _, _, _ = make((2, 0, None), 64, 16, 1, BF)
    fin = torch.full_like(b["initial_state"], float("nan"))
    kda.kda_scan_fwd(**a, out=torch.empty_like(a["x"]), **b, final_state=fin)
    assert torch.equal(fin, b["initial_state"])
    g = kda.kda_scan_bwd(**a, dout=c["dout"], **b, dfinal_state=c["dfin"])
    assert torch.equal(g["dinitial_state"], c["dfin"])
    assert not g["dA_log"].any() and not g["dD"].any() and not g["ddt_bias"].any()


def test_bad_seqlens_are_reported(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    a, b, c, _, _, _ = make((1, 400, None), 16, 16, 1, F)
    b["initial_state"] = None
    for cu in ([0, 300, 200, 400], [1, 400], [0, 401], [-5, 100, 400]):
        cud = torch.tensor(cu, device="cuda")
        ws = kda.make_scan_workspace(1, 400, 16, 16, 1, len(cu) - 1)
        kda.kda_scan_fwd(**a, out=torch.zeros_like(a["x"]), **b, cu_seqlens=cud, workspace=ws)
        assert kda.kda_get_device_status(ws) == 9, cu
        g = kda.kda_scan_bwd(**a, dout=c["dout"], **b, cu_seqlens=cud)
        assert kda.kda_get_device_status(g["workspace"]) == 9, cu
