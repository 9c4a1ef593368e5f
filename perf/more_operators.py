"""The gated linear recurrence and the gated feed-forward product, as they are measured.
`run` is one pass of an operator, in its plain torch form or (with `own`) as the
library's calls; `exact` is its definition in 64 bits.

The sizes are those of this repository's workloads (prefill B=8 T=4096 with 32 heads of
128, the irregular packed lengths with 16 heads, the long packed sequence with 8, decode
steps of 256 sequences), with a feed-forward width of three times the model's.
"""
import math

import torch

own = False

PACKED = "1023,1025,1,17,4096,65537,2048,333"
LONG = "65536,1024,1024,1024,1024,1024"


def listed():
    return [
        # the recurrence in one decode step of 256 sequences: latency
        {"name": "linrec_step", "op": "linrec", "B": 256, "T": 1, "lengths": "", "D": 4096,
         "type": "bf16", "z": False, "bwd": False, "saved": False},
        # batched prompts
        {"name": "linrec_prompt", "op": "linrec", "B": 8, "T": 4096, "lengths": "", "D": 4096,
         "type": "bf16", "z": False, "bwd": False, "saved": False},
        # a packed prompt batch of very different lengths, gated output
        {"name": "linrec_packed", "op": "linrec", "B": 1, "T": 0, "lengths": PACKED, "D": 2048,
         "type": "bf16", "z": True, "bwd": False, "saved": False},
        # one long prompt with few channels next to short ones
        {"name": "linrec_long", "op": "linrec", "B": 1, "T": 0, "lengths": LONG, "D": 1024,
         "type": "bf16", "z": False, "bwd": False, "saved": False},
        # a training step: the forward that keeps its chunk states, then the backward
        {"name": "linrec_train", "op": "linrec", "B": 4, "T": 4096, "lengths": "", "D": 4096,
         "type": "bf16", "z": True, "bwd": True, "saved": True},
        # a packed training batch in fp32 at an odd width, states recomputed
        {"name": "linrec_odd", "op": "linrec", "B": 1, "T": 0, "lengths": "4099,1,0,733,8191,2050",
         "D": 1001, "type": "fp32", "z": False, "bwd": True, "saved": False},
        # the feed-forward product for one token: the weights are read once
        {"name": "glu_token", "op": "glu", "rows": 1, "D": 4096, "F": 12288, "act": "silu",
         "bwd": False, "saved": False},
        # the same for a small decode batch
        {"name": "glu_step", "op": "glu", "rows": 32, "D": 4096, "F": 12288, "act": "silu",
         "bwd": False, "saved": False},
        # one decode step of 256 sequences
        {"name": "glu_batch", "op": "glu", "rows": 256, "D": 4096, "F": 12288, "act": "silu",
         "bwd": False, "saved": False},
        # prompts at the prefill size
        {"name": "glu_prompt", "op": "glu", "rows": 32768, "D": 4096, "F": 12288, "act": "silu",
         "bwd": False, "saved": False},
        # a training step: the forward that keeps its pre-activations, then the backward
        {"name": "glu_train", "op": "glu", "rows": 16384, "D": 4096, "F": 12288, "act": "silu",
         "bwd": True, "saved": True},
        # the backward at ragged sizes, pre-activations recomputed
        {"name": "glu_odd", "op": "glu", "rows": 4097, "D": 1000, "F": 2728, "act": "gelu",
         "bwd": True, "saved": False},
    ]


def _lengths(rng, total):
    """Packed lengths from empty to long that sum to at most `total`."""
    out, left = [], total
    for _ in range(rng.randint(2, 24)):
        n = min(left, int(math.exp(rng.uniform(0.0, math.log(total)))) - 1)
        out.append(n)
        left -= n
    out[-1] += 1
    return ",".join(map(str, out))


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    bwd = rng.random() < 0.5
    if rng.random() < 0.5:
        D = _spread(rng, 33, 4096)
        if rng.random() < 0.6:
            D = -(-D // 64) * 64
        c = {"op": "linrec", "D": D, "type": rng.choice(["bf16", "bf16", "fp32"]),
             "z": rng.random() < 0.5}
        kind = rng.choice(["step", "batch", "packed"])
        c["bwd"] = bwd and kind != "step"
        c["saved"] = c["bwd"] and rng.random() < 0.5
        if kind == "step":
            c.update(B=_spread(rng, 1, 256), T=rng.choice([1, 1, 2, 5]), lengths="")
        elif kind == "batch":
            c.update(B=rng.randint(1, 6), T=_spread(rng, 17, 4096), lengths="")
        else:
            c.update(B=1, T=0, lengths=_lengths(rng, _spread(rng, 64, 32768)))
        return c
    rows = _spread(rng, 1, 16384)
    D, F = _spread(rng, 8, 512) * 8, _spread(rng, 8, 1536) * 8
    return {"op": "glu", "rows": rows, "D": D, "F": F,
            "act": rng.choice(["silu", "silu", "gelu", "sigmoid"]), "bwd": bwd,
            "saved": bwd and rng.random() < 0.5}


# ------------------------------------------------------------------- inputs --
class _Rand:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=self.gen, device="cuda") * scale).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=self.gen, device="cuda") * (hi - lo) + lo


def _shape(case):
    """(B, T, N, cu_seqlens or None) of a case's token axis."""
    if not case["lengths"]:
        return case["B"], case["T"], case["B"], None
    n = [int(x) for x in case["lengths"].split(",")]
    cu = torch.tensor([0] + n, dtype=torch.int64).cumsum(0).cuda()
    return 1, sum(n), len(n), cu


def prepare(case, seed):
    s = {"case": case, "op": case["op"], "bwd": case["bwd"], "saved": case["saved"]}
    s.update((_prepare_linrec if case["op"] == "linrec" else _prepare_glu)(case, _Rand(seed)))
    return s


def _prepare_linrec(c, r):
    B, T, N, cu = _shape(c)
    D, ty = c["D"], torch.bfloat16 if c["type"] == "bf16" else torch.float32
    # both gates are the two halves of one projection's output
    gates = r.normal(B, T, 2 * D, dtype=ty)
    # decays between 0.9 and 0.999 a token at an open gate, to the eighth power
    a0 = r.uniform(D, lo=0.9, hi=0.999)
    s = {"x": r.normal(B, T, D, dtype=ty), "r": gates[..., :D], "i": gates[..., D:],
         "z": r.normal(B, T, D, dtype=ty) if c["z"] else None,
         "A_log": torch.log(-8 * torch.log(a0)), "r_bias": r.normal(D, scale=0.1),
         "i_bias": r.normal(D, scale=0.1), "init": r.normal(N, D), "cu": cu,
         "out": torch.empty(B, T, D, dtype=ty, device="cuda")}
    if c["bwd"]:
        s["dout"], s["dfin"] = r.normal(B, T, D, dtype=ty), r.normal(N, D)
    else:
        s["fin"] = torch.empty(N, D, device="cuda")
    return s


def _prepare_glu(c, r):
    M, D, F, ty = c["rows"], c["D"], c["F"], torch.bfloat16
    s = {"x": r.normal(1, M, D, dtype=ty), "w_gate": r.normal(F, D, scale=D ** -0.5, dtype=ty),
         "w_up": r.normal(F, D, scale=D ** -0.5, dtype=ty), "act": c["act"],
         "out": torch.empty(1, M, F, dtype=ty, device="cuda")}
    if c["bwd"]:
        s["dout"] = r.normal(1, M, F, dtype=ty)
    return s


# ---------------------------------------------------------------------- run --
def run(s):
    return (_own if own else _plain)[s["op"], s["bwd"]](s)


def _kda():
    import kimi_delta_attention_08_gb300 as kda
    return kda


def _own_linrec(s):
    _kda().kda_linrec_fwd(s["x"], s["r"], s["i"], s["A_log"], s["out"], s["z"], s["r_bias"],
                          s["i_bias"], s["init"], s["fin"], s["cu"])
    return s["out"], s["fin"]


def _own_linrec_bwd(s):
    kda, x = _kda(), s["x"]
    states, out = None, {}
    if s["saved"]:
        states = kda.make_linrec_states(x.shape[0] * x.shape[1], x.shape[2], x.device)
        kda.kda_linrec_fwd(x, s["r"], s["i"], s["A_log"], s["out"], s["z"], s["r_bias"],
                           s["i_bias"], s["init"], None, s["cu"], chunk_states=states)
        out["out"] = s["out"]
    g = kda.kda_linrec_bwd(x, s["r"], s["i"], s["A_log"], s["dout"], s["z"], s["r_bias"],
                           s["i_bias"], s["init"], s["dfin"], s["cu"], chunk_states=states)
    names = _LINREC_GRADS + (() if s["z"] is None else ("dz",))
    return {**out, **{k: g[k] for k in names}}


def _own_glu(s):
    _kda().kda_glu_fwd(s["x"], s["w_gate"], s["w_up"], s["out"], activation=s["act"])
    return s["out"]


def _own_glu_bwd(s):
    kda, x = _kda(), s["x"]
    pre, out = None, {}
    if s["saved"]:
        pre = torch.empty(*x.shape[:2], 2 * s["out"].shape[2], dtype=x.dtype, device=x.device)
        kda.kda_glu_fwd(x, s["w_gate"], s["w_up"], s["out"], pre=pre, activation=s["act"])
        out["out"] = s["out"]
    g = kda.kda_glu_bwd(x, s["w_gate"], s["w_up"], s["dout"], pre=pre, activation=s["act"])
    return {**out, **{k: g[k] for k in ("dx", "dw_gate", "dw_up")}}


_LINREC_GRADS = ("dx", "dr", "di", "dA_log", "dr_bias", "di_bias", "dinitial_state")


# ------------------------------------------------------ the plain torch forms --
def _bounds_of(s):
    """The packed rows' first row and end of each sequence."""
    B, T = s["x"].shape[:2]
    cu = s["cu"]
    if cu is None:
        cu = torch.arange(B + 1, device=s["x"].device) * T
    return cu[:-1], cu[1:]


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t over the first axis, by doubling; a and b are used up."""
    s = 1
    while s < a.shape[0]:
        b[s:] += a[s:] * b[:-s].clone()
        a[s:] *= a[:-s].clone()
        s *= 2
    return b


def _linrec_terms(s):
    sh = s["x"].shape
    flat = lambda v: v.reshape(sh[0] * sh[1], sh[2]).float()  # noqa: E731
    x, R, I = flat(s["x"]), torch.sigmoid(flat(s["r"]) + s["r_bias"]), \
        torch.sigmoid(flat(s["i"]) + s["i_bias"])
    L = torch.exp(s["A_log"]) * R
    return x, R, I, L, torch.exp(-L), torch.sqrt(-torch.expm1(-2 * L))


def _linrec_states(s, a, b):
    """Every h_t, from the initial states."""
    bos, eos = _bounds_of(s)
    live = eos > bos
    first = bos[live]
    q = a.clone()
    b[first] += a[first] * s["init"][live]
    q[first] = 0
    return _linear_scan(q, b), live, first, eos[live] - 1


def _gated(s, h):
    if s["z"] is not None:
        z = s["z"].reshape(h.shape).float()
        h = h * z * torch.sigmoid(z)
    return h.to(s["x"].dtype).view(s["x"].shape)


def _plain_linrec(s):
    x, _, I, _, a, m = _linrec_terms(s)
    h, live, _, last = _linrec_states(s, a, m * I * x)
    fin = s["init"].clone()
    fin[live] = h[last]
    return _gated(s, h), fin


def _plain_linrec_bwd(s):
    x, R, I, L, a, m = _linrec_terms(s)
    h, live, first, last = _linrec_states(s, a, m * I * x)
    ty, sh = s["x"].dtype, s["x"].shape
    out = {"out": _gated(s, h)} if s["saved"] else {}
    dy = s["dout"].reshape(x.shape).float()
    if s["z"] is not None:
        z = s["z"].reshape(x.shape).float()
        g = torch.sigmoid(z)
        out["dz"] = (dy * h * g * (1 + z * (1 - g))).to(ty).view(sh)
        dy = dy * z * g
    b = dy.clone()
    b[last] += s["dfin"][live]
    q = torch.zeros_like(a)
    q[:-1] = a[1:]
    q[last] = 0
    g = _linear_scan(q.flip(0), b.flip(0)).flip(0)
    dinit = s["dfin"].clone()
    dinit[live] = a[first] * g[first]
    before = torch.roll(h, 1, 0)
    before[first] = s["init"][live]
    e = g * L * (a * a / m * I * x - a * before)
    dr, dw = e * (1 - R), g * m
    di = dw * x * I * (1 - I)
    total = lambda v: v.sum(0, dtype=torch.float64).float()  # noqa: E731
    return {**out, "dx": (dw * I).to(ty).view(sh), "dr": dr.to(ty).view(sh),
            "di": di.to(ty).view(sh), "dA_log": total(e), "dr_bias": total(dr),
            "di_bias": total(di), "dinitial_state": dinit}


GELU = math.sqrt(8 / math.pi)  # gelu(g) = g sigmoid(GELU (g + 0.044715 g^3)), the tanh form


def _activation(g, act):
    """f(g) and its slope."""
    if act == "gelu":
        q = torch.sigmoid(GELU * (g + 0.044715 * g * g * g))
        return g * q, q + g * q * (1 - q) * GELU * (1 + 3 * 0.044715 * g * g)
    q = torch.sigmoid(g)
    return (q, q * (1 - q)) if act == "sigmoid" else (g * q, q * (1 + g * (1 - q)))


def _plain_glu(s):
    x = s["x"][0].float()
    g, u = x @ s["w_gate"].float().T, x @ s["w_up"].float().T
    return (_activation(g, s["act"])[0] * u).to(s["x"].dtype)[None]


def _plain_glu_bwd(s):
    x, wg, wu, dout = s["x"][0].float(), s["w_gate"].float(), s["w_up"].float(), s["dout"][0].float()
    ty = s["x"].dtype
    g, u = x @ wg.T, x @ wu.T
    f, df = _activation(g, s["act"])
    out = {"out": (f * u).to(ty)[None]} if s["saved"] else {}
    dg, du = dout * u * df, dout * f
    return {**out, "dx": (dg @ wg + du @ wu).to(ty)[None], "dw_gate": (dg.T @ x).to(ty),
            "dw_up": (du.T @ x).to(ty)}


_plain = {("linrec", False): _plain_linrec, ("linrec", True): _plain_linrec_bwd,
          ("glu", False): _plain_glu, ("glu", True): _plain_glu_bwd}
_own = {("linrec", False): _own_linrec, ("linrec", True): _own_linrec_bwd,
        ("glu", False): _own_glu, ("glu", True): _own_glu_bwd}


# --------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] == "glu":
        M, D, F = c["rows"], c["D"], c["F"]
        if not c["bwd"]:
            return {"bytes": 2 * (M * D + 2 * D * F + M * F), "flops": 4 * M * D * F}
        # dx and the weights' gradients, and the pre-activations once in either form
        return {"bytes": 2 * (2 * M * D + 4 * D * F + M * F * (2 if c["saved"] else 1)),
                "flops": 12 * M * D * F}
    n = [int(x) for x in c["lengths"].split(",")] if c["lengths"] else [c["T"]] * c["B"]
    M, N, D = sum(n), len(n), c["D"]
    e, z = 2 if c["type"] == "bf16" else 4, int(c["z"])
    fwd = (4 + z) * M * D * e + 8 * N * D + 12 * D
    if not c["bwd"]:
        return {"bytes": fwd, "flops": M * D * (20 + 5 * z)}
    bwd = (7 + 2 * z) * M * D * e + 12 * N * D + 24 * D
    return {"bytes": bwd + (fwd - 4 * N * D if c["saved"] else 0),
            "flops": M * D * (60 + 12 * z) if not c["saved"] else M * D * (80 + 17 * z)}


# -------------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linrec(s) if s["op"] == "linrec" else _exact_glu(s)


def _exact_linrec(s):
    """Token by token in 64 bits; all sequences of a batch at once, packed ones in turn."""
    f = lambda k: s[k].double()  # noqa: E731
    x, (B, T, D) = f("x"), s["x"].shape
    R = 1 / (1 + torch.exp(-(f("r") + f("r_bias"))))
    I = 1 / (1 + torch.exp(-(f("i") + f("i_bias"))))
    L = torch.exp(f("A_log")) * R
    a = torch.exp(-L)
    m = torch.sqrt(-torch.expm1(-2 * L))
    b = m * I * x
    h, before = torch.empty_like(x), torch.empty_like(x)
    if s["cu"] is None:
        spans = [(slice(None), slice(None), 0, T)] if T else []
    else:
        c = s["cu"].tolist()
        spans = [(slice(n, n + 1), slice(0, 1), p, q) for n, (p, q) in enumerate(zip(c, c[1:])) if q > p]
    fin = f("init")
    for n, bt, p, q in spans:
        st = f("init")[n]
        for t in range(p, q):
            before[bt, t] = st
            st = torch.addcmul(b[bt, t], a[bt, t], st)
            h[bt, t] = st
        fin[n] = st
    z, silu = None, 1.0
    if s["z"] is not None:
        z = f("z")
        sg = 1 / (1 + torch.exp(-z))
        silu = z * sg
    if not s["bwd"]:
        return h * silu, fin
    dout = f("dout")
    dy = dout * silu
    g, dinit = torch.empty_like(x), f("dfin")
    for n, bt, p, q in spans:
        carry = f("dfin")[n]
        for t in range(q - 1, p - 1, -1):
            gt = dy[bt, t] + carry
            g[bt, t] = gt
            carry = a[bt, t] * gt
        dinit[n] = carry
    # through the decay: d h_t / d L_t = -a h_{t-1} + (d m / d L) I x, with d m / d L = a^2 / m
    e = g * (torch.where(L > 0, a * a / m, 0) * I * x - a * before) * L
    r = {"dx": g * m * I, "dr": e * (1 - R), "di": g * m * x * I * (1 - I), "dA_log": e.sum((0, 1)),
         "dinitial_state": dinit}
    r["dr_bias"], r["di_bias"] = r["dr"].sum((0, 1)), r["di"].sum((0, 1))
    if z is not None:
        r["dz"] = dout * h * (sg + z * sg * (1 - sg))
    if s["saved"]:
        r["out"] = h * silu
    order = ("out", "dz") + _LINREC_GRADS
    return {k: r[k] for k in order if k in r}


def _exact_glu(s):
    """Gradients by differentiating the definition."""
    M, D, F = s["case"]["rows"], s["case"]["D"], s["case"]["F"]
    if M * D * F * (12 if s["bwd"] else 4) > 1.5e13:
        return None
    x, wg, wu = (s[k].double().requires_grad_(s["bwd"]) for k in ("x", "w_gate", "w_up"))
    with torch.enable_grad():
        g = torch.einsum("bmd,fd->bmf", x, wg)
        if s["act"] == "gelu":
            f = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
        else:
            f = 1 / (1 + torch.exp(-g)) * (g if s["act"] == "silu" else 1)
        out = f * torch.einsum("bmd,fd->bmf", x, wu)
        if not s["bwd"]:
            return out
        dx, dwg, dwu = torch.autograd.grad(out, (x, wg, wu), s["dout"].double())
    r = {"out": out.detach()} if s["saved"] else {}
    return {**r, "dx": dx, "dw_gate": dwg, "dw_up": dwu}
