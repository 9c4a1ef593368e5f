"""The short causal convolution against its 64-bit form: widths, types, packed and
batched sequences (empty, one token, shorter than the window), states in place, slices of
wider rows, split outputs, channel counts off the vector width.

Bounds: a pre-activation is a sum of width + 1 terms (5 roundings of 2^-24 at most); the
activation adds the exponential (2^-22), a reciprocal and three products: under 16 steps
of 2^-24 of the magnitudes of tests/layer_ref.py.  A weight's gradient is a sum over
tokens, added a run at a time (8 to 32 tokens at these sizes), then by 4 and by row blocks,
every 32nd together: 80 steps and one per 256 tokens."""
import zlib

import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
SEQS = {"one": (3, 1, None), "short": (2, 3, None), "batch": (2, 67, None), "long": (1, 300, None),
        "packed": (1, 211, [0, 0, 1, 3, 70, 70, 135, 211]), "tail": (1, 90, [0, 31, 64])}


def seed_of(*what):
    return zlib.crc32(repr(what).encode()) % 1000


def make(seq, C, W, ty, seed, wide=0, init=True):
    B, T, cu = SEQS[seq]
    g = torch.Generator().manual_seed(seed)
    N = B if cu is None else len(cu) - 1
    r = lambda *s, t=ty: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    x = r(B, T, C + wide)[..., wide // 2:wide // 2 + C]
    a = {"x": x, "w": r(C, W, t=F), "b": r(C, t=F), "init": r(N, W - 1, C) if init else None,
         "dout": r(B, T, C), "dfin": r(N, W - 1, C)}
    return a, B, T, N, cu, None if cu is None else torch.tensor(cu, device="cuda")


def nan(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def check_fwd(kda, seq, C, W, ty, act="silu", wide=0, init=True, split=None, bias=True):
    a, B, T, N, cu, cud = make(seq, C, W, ty, seed_of(seq, C, W), wide, init)
    b = a["b"] if bias else None
    outs = [nan(B, T, n, dtype=ty) for n in split or [C]]
    fin = nan(N, W - 1, C, dtype=ty)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    kda.kda_conv_fwd(a["x"], a["w"], b, outs if split else outs[0], a["init"], fin, cud, ws,
                     activation=act)
    assert kda.kda_get_device_status(ws) == 0
    ref, rfin = R.conv(a["x"], a["w"], b, a["init"], cu, act)
    mag, _ = R.conv(a["x"], a["w"], b, a["init"], cu, act, mag=True)
    end = T if cu is None else cu[-1]
    out = torch.cat(outs, 2)
    R.close(out[:, :end], ref[:, :end], mag[:, :end], 16, "out")
    assert out[:, end:].isnan().all(), "rows of no sequence were written"
    assert torch.equal(R.d(fin), rfin), "final state"
    return a, out, fin


@pytest.mark.parametrize("seq", list(SEQS))
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("C,W", [(64, 4), (257, 3), (1000, 2), (5, 4)])
def test_forward(kda_lib, seq, ty, C, W):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, seq, C, W, ty)


@pytest.mark.parametrize("act", ["silu", None])
@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_forward_options(kda_lib, act, init, bias):
    import kimi_delta_attention_08_gb300 as kda
    check_fwd(kda, "packed", 96, 4, BF, act=act, init=init, bias=bias)


@pytest.mark.parametrize("wide", [64, 3])
@pytest.mark.parametrize("split", [[128, 64, 64], [100, 100, 55, 1]])
def test_forward_slices_and_split(kda_lib, wide, split):
    import kimi_delta_attention_08_gb300 as kda
    for seq in ("one", "packed"):
        check_fwd(kda, seq, 256, 4, BF, wide=wide, split=split)


@pytest.mark.parametrize("seq", ["one", "short", "batch", "packed"])
@pytest.mark.parametrize("C", [64, 37])
def test_state_in_place(kda_lib, seq, C):
    """final_state may be the initial_state buffer: the same bits as with two buffers."""
    import kimi_delta_attention_08_gb300 as kda
    a, out, fin = check_fwd(kda, seq, C, 4, BF)
    _, B, T, N, cu, cud = make(seq, C, 4, BF, 0)
    st, o = a["init"].clone(), torch.full_like(out, float("nan"))
    kda.kda_conv_fwd(a["x"], a["w"], a["b"], o, st, st, cud)
    assert torch.equal(st, fin) and torch.equal(o.view(torch.int16), out.view(torch.int16))


def test_steps_equal_a_prompt(kda_lib):
    """Token by token with the state carried in place: the prompt's bits."""
    import kimi_delta_attention_08_gb300 as kda
    a, B, T, N, cu, _ = make("batch", 320, 4, BF, 7)
    out, fin = nan(B, T, 320, dtype=BF), nan(N, 3, 320, dtype=BF)
    kda.kda_conv_fwd(a["x"], a["w"], a["b"], out, a["init"], fin)
    st, got = a["init"].clone(), torch.empty_like(out)
    for t in range(T):
        o = nan(B, 1, 320, dtype=BF)
        kda.kda_conv_fwd(a["x"][:, t:t + 1].contiguous(), a["w"], a["b"], o, st, st)
        got[:, t:t + 1] = o
    assert torch.equal(got, out) and torch.equal(st, fin)


def check_bwd(kda, seq, C, W, ty, act="silu", wide=0, init=True, split=None, dout_ty=None, dfin=True):
    a, B, T, N, cu, cud = make(seq, C, W, ty, seed_of(seq, C, W) + 1, wide, init)
    dout = a["dout"].to(dout_ty or ty)
    df = a["dfin"] if dfin else None
    parts = [p.contiguous() for p in dout.split(split, 2)] if split else dout
    g = kda.kda_conv_bwd(a["x"], a["w"], a["b"], parts, a["init"], df, cud, activation=act)
    assert kda.kda_get_device_status(g["workspace"]) == 0
    args = (a["x"], a["w"], a["b"], a["init"], cu, act, dout, df)
    ref, mag = R.conv(*args), R.conv(*args, mag=True)
    names = ["dx", "dweight", "dbias"] + (["dinitial_state"] if init else [])
    assert set(names) == set(g) - {"workspace"}
    for nm in names:
        R.close(g[nm], ref[nm], mag[nm], 16 if nm in ("dx", "dinitial_state") else 96 + B * T / 256, nm)
    return g


@pytest.mark.parametrize("seq", list(SEQS))
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("C,W", [(64, 4), (257, 3), (1000, 2), (5, 4)])
def test_backward(kda_lib, seq, ty, C, W):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, seq, C, W, ty)


@pytest.mark.parametrize("kw", [dict(act=None), dict(init=False), dict(dfin=False), dict(dout_ty=F),
                                dict(split=[64, 128, 64]), dict(split=[64, 128, 64], dout_ty=F),
                                dict(split=[1, 255]), dict(wide=64), dict(wide=3)])
def test_backward_options(kda_lib, kw):
    import kimi_delta_attention_08_gb300 as kda
    check_bwd(kda, "packed", 256, 4, BF, **kw)


@pytest.mark.parametrize("n", [150, 1500])
@pytest.mark.parametrize("C", [64, 33])
def test_many_sequences(kda_lib, n, C):
    """More sequences than one search step tells apart, from empty to longer than a run."""
    import itertools
    import kimi_delta_attention_08_gb300 as kda
    cu = list(itertools.accumulate([(7 * i * i + 3 * i) % 41 if i % 50 else 140 for i in range(n)], initial=0))
    SEQS["many"] = (1, cu[-1] + 3, cu)
    try:
        check_fwd(kda, "many", C, 4, BF)
        check_bwd(kda, "many", C, 4, BF)
    finally:
        del SEQS["many"]


def test_backward_repeats_its_bits(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    a = check_bwd(kda, "long", 264, 4, BF)
    b = check_bwd(kda, "long", 264, 4, BF)
    for nm in a:
        if nm != "workspace":
            assert torch.equal(a[nm], b[nm])


def test_no_tokens(kda_lib):
    """Empty input: the final state is the initial one, gradients are those of the state."""
    import kimi_delta_attention_08_gb300 as kda
    w, b = torch.randn(16, 4, device="cuda"), torch.randn(16, device="cuda")
    x = torch.empty(2, 0, 16, dtype=BF, device="cuda")
    init, fin = torch.randn(2, 3, 16, device="cuda").to(BF), nan(2, 3, 16, dtype=BF)
    kda.kda_conv_fwd(x, w, b, torch.empty_like(x), init, fin)
    assert torch.equal(init, fin)
    g = kda.kda_conv_bwd(x, w, b, torch.empty_like(x), init, init)
    assert torch.equal(g["dinitial_state"], init.float()) and not g["dweight"].any() and not g["dbias"].any()


def test_bad_seqlens_are_reported(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    w = torch.randn(16, 4, device="cuda")
    x = torch.randn(1, 40, 16, device="cuda")
    for cu in ([0, 30, 20, 40], [1, 40], [0, 41], [-5, 10, 40]):
        c = torch.tensor(cu, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        out, fin = torch.zeros_like(x), torch.zeros(len(cu) - 1, 3, 16, device="cuda")
        kda.kda_conv_fwd(x, w, None, out, None, fin, c, ws)
        assert kda.kda_get_device_status(ws) == 9, cu
        g = kda.kda_conv_bwd(x, w, None, x, None, fin, c)
        assert kda.kda_get_device_status(g["workspace"]) == 9, cu
    c = torch.tensor([0, 10, 40], device="cuda")
    kda.kda_conv_fwd(x, w, None, out, None, None, c, ws)
    assert kda.kda_get_device_status(ws) == 0  # the word is written anew by each call
