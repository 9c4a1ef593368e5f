"""The operators around the KDA recurrence in a layer, as they are measured: the
short causal convolution, the selective state space scan, and the norms before
and after a block.  `run` is one pass of an operator, in its plain torch form or
(with `own`) as the library's calls; `exact` is its definition in 64 bits.

The sizes are those of this repository's workloads (prefill B=8 T=4096 with 32
heads of 128, the irregular packed lengths, the long packed sequence) and of
decode steps of 256 sequences.
"""
import math

import torch

own = False

PACKED = "1023,1025,1,17,4096,65537,2048,333"
LONG = "65536,1024,1024,1024,1024,1024"
EPS = 1e-6


def listed():
    return [
        # one decode step of 256 sequences over the q, k, v channels of 32 heads
        {"name": "conv_step", "op": "conv", "B": 256, "T": 1, "lengths": "", "C": 12288, "W": 4,
         "type": "bf16", "split": True, "bwd": False},
        # a packed prompt batch of very different lengths, q, k, v of 16 heads, states kept
        {"name": "conv_packed", "op": "conv", "B": 1, "T": 0, "lengths": PACKED, "C": 6144, "W": 4,
         "type": "bf16", "split": True, "bwd": False},
        # the convolution's backward in training at the prefill size
        {"name": "conv_train", "op": "conv", "B": 8, "T": 4096, "lengths": "", "C": 12288, "W": 4,
         "type": "bf16", "split": False, "bwd": True},
        # one decode step of 256 sequences
        {"name": "scan_step", "op": "scan", "B": 256, "T": 1, "lengths": "", "D": 4096, "N": 16,
         "G": 1, "type": "bf16", "bwd": False, "saved": False},
        # batched prompts
        {"name": "scan_prompt", "op": "scan", "B": 8, "T": 4096, "lengths": "", "D": 4096, "N": 16,
         "G": 1, "type": "bf16", "bwd": False, "saved": False},
        # one long prompt with few channels next to short ones
        {"name": "scan_long", "op": "scan", "B": 1, "T": 0, "lengths": LONG, "D": 1024, "N": 16,
         "G": 1, "type": "bf16", "bwd": False, "saved": False},
        # a training step of the scan: the forward that keeps its chunk states, then the backward
        {"name": "scan_train", "op": "scan", "B": 4, "T": 4096, "lengths": "", "D": 4096, "N": 16,
         "G": 1, "type": "bf16", "bwd": True, "saved": True},
        # the norm before a block in a small decode batch: latency
        {"name": "prenorm_step", "op": "prenorm", "rows": 32, "D": 4096, "type": "bf16",
         "stream": "bf16", "scale": "number", "bwd": False},
        # the same over a training batch, with the residual stream in fp32
        {"name": "prenorm_prompt", "op": "prenorm", "rows": 32768, "D": 4096, "type": "bf16",
         "stream": "fp32", "scale": "number", "bwd": False},
        # its backward, with a learned scale for each channel
        {"name": "prenorm_train", "op": "prenorm", "rows": 32768, "D": 4096, "type": "bf16",
         "stream": "bf16", "scale": "channel", "bwd": True},
        # the gated norm of each head on the recurrence's output at the prefill size
        {"name": "postnorm_heads", "op": "postnorm", "rows": 8 * 4096 * 32, "D": 128,
         "type": "bf16", "gate": "sigmoid", "residual": False, "scale": "number", "bwd": False},
        # the norm after a block of an odd width, in fp32, with gate and scaled residual: backward
        {"name": "postnorm_train", "op": "postnorm", "rows": 74097, "D": 1001, "type": "fp32",
         "gate": "silu", "residual": True, "scale": "channel", "bwd": True},
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
    op = rng.choice(["conv", "conv", "scan", "scan", "prenorm", "postnorm"])
    ty = rng.choice(["bf16", "bf16", "fp32"])
    bwd = rng.random() < 0.5
    if op in ("conv", "scan"):
        width = _spread(rng, 33, 4096)
        if rng.random() < 0.5:
            width = -(-width // 64) * 64
        kind = rng.choice(["step", "batch", "packed"])
        c = {"op": op, "type": ty, "bwd": bwd and kind != "step"}
        if kind == "step":
            c.update(B=_spread(rng, 1, 256), T=rng.choice([1, 1, 2, 5]), lengths="")
        elif kind == "batch":
            c.update(B=rng.randint(1, 6), T=_spread(rng, 17, 4096), lengths="")
        else:
            c.update(B=1, T=0, lengths=_lengths(rng, _spread(rng, 64, 16384)))
        if op == "conv":
            c.update(C=width, W=rng.randint(2, 4), split=rng.random() < 0.5)
        else:
            c.update(D=min(width, 2048), N=rng.choice([8, 16, 16, 32, 64]), G=1,
                     saved=c["bwd"] and rng.random() < 0.5)
            if c["D"] % 64 == 0:
                c["G"] = rng.choice([1, 1, 2, 4])
            rows = c["B"] * c["T"] or sum(int(n) for n in c["lengths"].split(","))
            c["D"] = max(64, min(c["D"], int(6e8 / (rows * c["N"])) // 64 * 64)) \
                if rows * c["D"] * c["N"] > 6e8 else c["D"]
        return c
    wide = rng.random() < 0.5
    D = _spread(rng, 1000, 8192) if wide else rng.choice([64, 96, 128, 128, 192, 257])
    if wide and rng.random() < 0.5:
        D = D // 8 * 8
    c = {"op": op, "rows": _spread(rng, 1, 64 * 1024 * 1024 // D), "D": D, "type": ty,
         "scale": rng.choice(["number", "channel"]), "bwd": bwd}
    if op == "prenorm":
        c["stream"] = rng.choice([ty, "fp32"])
    else:
        c["gate"] = rng.choice(["none", "sigmoid", "silu"])
        c["residual"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------- inputs --
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


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
    s = {"case": case, "op": case["op"], "bwd": case["bwd"]}
    s.update({"conv": _prepare_conv, "scan": _prepare_scan, "prenorm": _prepare_prenorm,
              "postnorm": _prepare_postnorm}[case["op"]](case, _Rand(seed)))
    return s


def _prepare_conv(c, r):
    B, T, N, cu = _shape(c)
    C, W, ty = c["C"], c["W"], _dtype(c["type"])
    # the channels are a part of a wider projection's output
    x = r.normal(B, T, C + 64, dtype=ty)[..., :C]
    s = {"x": x, "w": r.normal(C, W, scale=W ** -0.5), "b": r.normal(C, scale=0.1),
         "init": r.normal(N, W - 1, C, dtype=ty), "cu": cu}
    if c["bwd"]:
        s["dout"] = r.normal(B, T, C, dtype=ty)
        s["dfin"] = r.normal(N, W - 1, C, dtype=ty)
    else:
        third = C // 3
        sizes = [third, third, C - 2 * third] if c["split"] else [C]
        s["out"] = [torch.empty(B, T, n, dtype=ty, device="cuda") for n in sizes]
        s["fin"] = torch.empty(N, W - 1, C, dtype=ty, device="cuda")
    return s


def _prepare_scan(c, r):
    B, T, N, cu = _shape(c)
    D, n, G, ty = c["D"], c["N"], c["G"], _dtype(c["type"])
    # steps between 1e-3 and 1e-1 at dt = 0, decay rates 1 .. n, as such layers start out
    step = torch.exp(r.uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s = {"x": r.normal(B, T, D, dtype=ty), "dt": r.normal(B, T, D, dtype=ty),
         "z": r.normal(B, T, 2 * D, dtype=ty)[..., D:],  # half of a projection's output
         "A_log": torch.log(torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
                            ).expand(D, n).contiguous() + r.normal(D, n, scale=0.1),
         "B": r.normal(B, T, G, n, dtype=ty), "C": r.normal(B, T, G, n, dtype=ty),
         "D": 1.0 + r.normal(D, scale=0.1), "dt_bias": torch.log(torch.expm1(step)),
         "init": r.normal(N, D, n, scale=0.1), "cu": cu, "saved": c["saved"],
         "out": torch.empty(B, T, D, dtype=ty, device="cuda")}
    if c["bwd"]:
        s["dout"] = r.normal(B, T, D, dtype=ty)
        s["dfin"] = r.normal(N, D, n, scale=0.1)
    else:
        s["fin"] = torch.empty(N, D, n, device="cuda")
    return s


def _scale(c, r, D):
    return 0.5 + r.normal(D, scale=0.1) if c["scale"] == "channel" else 0.5


def _prepare_prenorm(c, r):
    R, D, ty, st = c["rows"], c["D"], _dtype(c["type"]), _dtype(c["stream"])
    s = {"x": r.normal(R, D, dtype=ty), "w": 1.0 + r.normal(D, scale=0.1), "s": _scale(c, r, D)}
    if c["bwd"]:
        s["h"] = r.normal(R, D, scale=2.0, dtype=st)  # the residual stream after the forward
        s["dout"], s["dh"] = r.normal(R, D, dtype=ty), r.normal(R, D, dtype=st)
    else:
        s["res"] = r.normal(R, D, scale=2.0, dtype=st)
        s["out"], s["res_out"] = torch.empty_like(s["x"]), torch.empty_like(s["res"])
    return s


def _prepare_postnorm(c, r):
    R, D, ty = c["rows"], c["D"], _dtype(c["type"])
    s = {"x": r.normal(R, D, dtype=ty), "w": 1.0 + r.normal(D, scale=0.1), "s": _scale(c, r, D),
         "gate": None if c["gate"] == "none" else r.normal(R, D, dtype=ty),
         "act": "sigmoid" if c["gate"] == "none" else c["gate"]}
    if c["bwd"]:
        s["dout"] = r.normal(R, D, dtype=ty)
    else:
        s["res"] = r.normal(R, D, dtype=ty) if c["residual"] else None
        s["out"] = torch.empty_like(s["x"])
    return s


# ---------------------------------------------------------------------- run --
def run(s):
    return (_own if own else _plain)[s["op"], s["bwd"]](s)


def _kda():
    import kimi_delta_attention_08_gb300 as kda
    return kda


def _own_conv(s):
    _kda().kda_conv_fwd(s["x"], s["w"], s["b"], s["out"], s["init"], s["fin"], s["cu"])
    return s["out"], s["fin"]


def _own_conv_bwd(s):
    g = _kda().kda_conv_bwd(s["x"], s["w"], s["b"], s["dout"], s["init"], s["dfin"], s["cu"])
    return {k: g[k] for k in ("dx", "dweight", "dbias", "dinitial_state")}


def _own_scan(s):
    _kda().kda_scan_fwd(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["out"], s["D"], s["z"],
                        s["dt_bias"], s["init"], s["fin"], s["cu"])
    return s["out"], s["fin"]


def _own_scan_bwd(s):
    kda, x = _kda(), s["x"]
    states = None
    if s["saved"]:
        states = kda.make_scan_states(x.shape[0] * x.shape[1], s["init"].shape[0], x.shape[2],
                                      s["A_log"].shape[1], x.device)
    kda.kda_scan_fwd(x, s["dt"], s["A_log"], s["B"], s["C"], s["out"], s["D"], s["z"],
                     s["dt_bias"], s["init"], None, s["cu"], chunk_states=states)
    g = kda.kda_scan_bwd(x, s["dt"], s["A_log"], s["B"], s["C"], s["dout"], s["D"], s["z"],
                         s["dt_bias"], s["init"], s["dfin"], s["cu"], chunk_states=states)
    return {"out": s["out"], **{k: g[k] for k in _SCAN_GRADS}}


def _own_prenorm(s):
    _kda().kda_prenorm_fwd(s["x"], s["res"], s["w"], s["out"], s["res_out"], res_scale=s["s"],
                           eps=EPS)
    return s["out"], s["res_out"]


def _own_prenorm_bwd(s):
    g = _kda().kda_prenorm_bwd(s["dout"], s["dh"], s["h"], s["w"], s["x"], res_scale=s["s"],
                               eps=EPS)
    return {k: g[k] for k in ("dx", "dresidual", "dweight", "dres_scale") if k in g}


def _own_postnorm(s):
    _kda().kda_postnorm_fwd(s["x"], s["w"], s["gate"], s["out"], s["res"], res_scale=s["s"],
                            activation=s["act"], eps=EPS)
    return s["out"]


def _own_postnorm_bwd(s):
    g = _kda().kda_postnorm_bwd(s["dout"], s["x"], s["w"], s["gate"], res_scale=s["s"],
                                activation=s["act"], eps=EPS)
    return {k: g[k] for k in ("dx", "dgate", "dweight", "dres_scale") if k in g}


_SCAN_GRADS = ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias", "dinitial_state")


# ------------------------------------------------------ the plain torch forms --
def _rows(x, cu):
    """Packed rows [M, ...] of a batch, and each row's sequence, first row and end."""
    B, T = x.shape[:2]
    x = x.reshape(B * T, *x.shape[2:])
    if cu is None:
        cu = torch.arange(B + 1, device=x.device) * T
    seq = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=x.device), cu.diff())
    return x, seq, cu[:-1], cu[1:]


def _silu(p):
    return p * torch.sigmoid(p)


def _dsilu(p):
    g = torch.sigmoid(p)
    return g * (1 + p * (1 - g))


def _shifted(x, init, seq, bos, back):
    """Row t - back of each row's sequence, from the initial state before its start."""
    t = torch.arange(x.shape[0], device=x.device)
    pos = t - bos[seq] - back
    old = init.float()[seq, (pos + init.shape[1]).clamp(0, init.shape[1] - 1)]
    return torch.where((pos >= 0)[:, None], x.float()[(t - back).clamp(min=0)], old)


def _conv_sum(s, x, seq, bos):
    W = s["w"].shape[1]
    return sum((_shifted(x, s["init"], seq, bos, W - 1 - j) * s["w"][:, j] for j in range(W - 1)),
               x.float() * s["w"][:, W - 1]) + s["b"]


def _plain_conv(s):
    x, seq, bos, eos = _rows(s["x"], s["cu"])
    W, ty = s["w"].shape[1], s["x"].dtype
    y = _silu(_conv_sum(s, x, seq, bos)).to(ty).view(s["x"].shape)
    pos = (eos - bos)[:, None] + torch.arange(1 - W, 0, device=x.device)  # rows of the state
    n = torch.arange(bos.numel(), device=x.device)[:, None]
    old = s["init"][n, (pos + W - 1).clamp(0, W - 2)]
    new = x[(bos[:, None] + pos).clamp(0, max(x.shape[0] - 1, 0))]
    fin = torch.where((pos >= 0)[..., None], new, old)
    return [p.contiguous() for p in y.split([o.shape[2] for o in s["out"]], 2)], fin


def _plain_conv_bwd(s):
    x, seq, bos, eos = _rows(s["x"], s["cu"])
    dout = s["dout"].reshape(x.shape).float()
    w, W, ty, N = s["w"], s["w"].shape[1], s["x"].dtype, bos.numel()
    dp = dout * _dsilu(_conv_sum(s, x, seq, bos))
    t = torch.arange(x.shape[0], device=x.device)
    dx = dp * w[:, W - 1]
    dinit = torch.zeros_like(s["init"], dtype=torch.float32)
    dw = []
    for j in range(W):
        back = W - 1 - j
        # a sum over all tokens: its terms in 64 bits, since they cancel
        dw.append((dp * _shifted(x, s["init"], seq, bos, back)).sum(0, dtype=torch.float64))
        if back:
            ok = t + back < eos[seq]
            dx = dx + torch.where(ok[:, None], dp[(t + back).clamp(max=x.shape[0] - 1)], 0) * w[:, j]
            first = torch.arange(back, device=x.device)  # rows that reach into the state
            at = bos[:, None] + first
            use = (at < eos[:, None])[..., None]
            dinit[:, j:j + back] += torch.where(use, dp[at.clamp(max=x.shape[0] - 1)], 0) * w[:, j]
    pos = (eos - bos)[:, None] + torch.arange(1 - W, 0, device=x.device)
    n = torch.arange(N, device=x.device)[:, None].expand_as(pos)
    old = pos < 0
    dinit.index_put_((n[old], pos[old] + W - 1), s["dfin"].float()[old], accumulate=True)
    dx.index_put_(((bos[:, None] + pos)[~old],), s["dfin"].float()[~old], accumulate=True)
    return {"dx": dx.to(ty).view(s["x"].shape), "dweight": torch.stack(dw, 1).float(),
            "dbias": dp.sum(0, dtype=torch.float64).float(), "dinitial_state": dinit}


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t over the first axis, by doubling; a and b are used up."""
    s = 1
    while s < a.shape[0]:
        b[s:] += a[s:] * b[:-s].clone()
        a[s:] *= a[:-s].clone()
        s *= 2
    return b


def _scan_terms(s):
    """Packed x, delta, a, the sequences' rows, and B and C for each channel's group."""
    x, seq, bos, eos = _rows(s["x"], s["cu"])
    D = x.shape[1]
    v = s["dt"].reshape(x.shape).float() + s["dt_bias"]
    delta = torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))
    a = torch.exp(delta[..., None] * -torch.exp(s["A_log"]))
    per = D // s["B"].shape[2]
    Bm, Cm = (s[k].reshape(x.shape[0], *s[k].shape[2:]).float() for k in ("B", "C"))
    return x.float(), v, delta, a, bos, eos, per, Bm, Cm


def _spread_groups(m, per):
    return m[:, :, None].expand(-1, -1, per, -1).reshape(m.shape[0], -1, m.shape[-1])


def _scan_states(s, x, delta, a, bos, eos, per, Bm):
    """Every h_t [M, D, N], and the first decays with the initial states folded in."""
    live = eos > bos
    b = (delta * x)[..., None] * (Bm if Bm.shape[1] == 1 else _spread_groups(Bm, per))
    first = bos[live]
    b[first] += a[first] * s["init"][live]
    q = a.clone()
    q[first] = 0
    return _linear_scan(q, b), live


def _plain_scan_forward(s):
    x, v, delta, a, bos, eos, per, Bm, Cm = _scan_terms(s)
    h, live = _scan_states(s, x, delta, a, bos, eos, per, Bm)
    if Cm.shape[1] == 1:
        y = torch.matmul(h, Cm.transpose(1, 2))[..., 0]
    else:
        y = (h * _spread_groups(Cm, per)).sum(-1)
    y = y + s["D"] * x
    out = (y * _silu(s["z"].reshape(x.shape).float())).to(s["x"].dtype).view(s["x"].shape)
    return out, h, y, (x, v, delta, a, bos, eos, per, Bm, Cm, live)


def _plain_scan(s):
    out, h, _, (_, _, _, _, _, eos, _, _, _, live) = _plain_scan_forward(s)
    fin = s["init"].clone()
    fin[live] = h[eos[live] - 1]
    return out, fin


def _plain_scan_bwd(s):
    out, h, y, (x, v, delta, a, bos, eos, per, Bm, Cm, live) = _plain_scan_forward(s)
    M, D, n = h.shape
    G, ty = Bm.shape[1], s["x"].dtype
    z, dout = s["z"].reshape(x.shape).float(), s["dout"].reshape(x.shape).float()
    dz, dy = dout * y * _dsilu(z), dout * _silu(z)
    dC = (dy[..., None] * h).view(M, G, per, n).sum(2)
    first, last = bos[live], eos[live] - 1
    # g_t = dy_t C_t + a_{t+1} g_{t+1} within each sequence, from its last token back
    b = dy[..., None] * (Cm if G == 1 else _spread_groups(Cm, per))
    b[last] += s["dfin"][live]
    q = torch.zeros_like(a)
    q[:-1] = a[1:]
    q[last] = 0
    g = _linear_scan(q.flip(0), b.flip(0)).flip(0)
    del q, b
    dinit = s["dfin"].clone()
    dinit[live] = a[first] * g[first]
    dxd = (g * (Bm if G == 1 else _spread_groups(Bm, per))).sum(-1)
    dB = ((delta * x)[..., None] * g).view(M, G, per, n).sum(2)
    # t <- g a h_{t-1}, in place of h
    h = torch.roll(h, 1, 0)
    h[first] = s["init"][live]
    h *= a
    h *= g
    del g, a
    A = -torch.exp(s["A_log"])
    ddelta = dxd * x + (h * A).sum(-1)
    dA = torch.einsum("td,tdn->dn", delta, h) * A
    dv = ddelta * torch.sigmoid(v)
    sh = s["x"].shape
    return {"out": out, "dx": (dxd * delta + dy * s["D"]).to(ty).view(sh), "ddt": dv.to(ty).view(sh),
            "dA_log": dA, "dB": dB.to(ty).view(s["B"].shape), "dC": dC.to(ty).view(s["C"].shape),
            "dD": (dy * x).sum(0, dtype=torch.float64).float(), "dz": dz.to(ty).view(sh),
            "ddt_bias": dv.sum(0, dtype=torch.float64).float(), "dinitial_state": dinit}


def _unit(h):
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    return h * r, r


def _plain_prenorm(s):
    h = s["res"].float() + s["s"] * s["x"].float()
    return (_unit(h)[0] * s["w"]).to(s["x"].dtype), h.to(s["res"].dtype)


def _plain_prenorm_bwd(s):
    u, r = _unit(s["h"].float())
    dy = s["dout"].float()
    du = dy * s["w"]
    dh = s["dh"].float() + r * (du - u * (du * u).mean(-1, keepdim=True))
    out = {"dx": (dh * s["s"]).to(s["x"].dtype), "dresidual": dh.to(s["h"].dtype),
           "dweight": (dy * u).sum(0, dtype=torch.float64).float()}
    if isinstance(s["s"], torch.Tensor):
        out["dres_scale"] = (dh * s["x"].float()).sum(0, dtype=torch.float64).float()
    return out


def _gates(s):
    """act(gate) and its derivative in fp32."""
    if s["gate"] is None:
        return 1.0, None
    p = s["gate"].float()
    if s["act"] == "silu":
        return _silu(p), _dsilu(p)
    g = torch.sigmoid(p)
    return g, g * (1 - g)


def _plain_postnorm(s):
    y = _unit(s["x"].float())[0] * s["w"] * _gates(s)[0] * s["s"]
    if s["res"] is not None:
        y = s["res"].float() + y
    return y.to(s["x"].dtype)


def _plain_postnorm_bwd(s):
    u, r = _unit(s["x"].float())
    act, dact = _gates(s)
    dout = s["dout"].float()
    dy = dout * s["s"]
    dn = dy * act
    du = dn * s["w"]
    ty = s["x"].dtype
    out = {"dx": (r * (du - u * (du * u).mean(-1, keepdim=True))).to(ty),
           "dweight": (dn * u).sum(0, dtype=torch.float64).float()}
    if dact is not None:
        out["dgate"] = (dy * u * s["w"] * dact).to(ty)
    if isinstance(s["s"], torch.Tensor):
        out["dres_scale"] = (dout * (u * s["w"] * act)).sum(0, dtype=torch.float64).float()
    return out


_plain = {("conv", False): _plain_conv, ("conv", True): _plain_conv_bwd,
          ("scan", False): _plain_scan, ("scan", True): _plain_scan_bwd,
          ("prenorm", False): _plain_prenorm, ("prenorm", True): _plain_prenorm_bwd,
          ("postnorm", False): _plain_postnorm, ("postnorm", True): _plain_postnorm_bwd}
_own = {("conv", False): _own_conv, ("conv", True): _own_conv_bwd,
        ("scan", False): _own_scan, ("scan", True): _own_scan_bwd,
        ("prenorm", False): _own_prenorm, ("prenorm", True): _own_prenorm_bwd,
        ("postnorm", False): _own_postnorm, ("postnorm", True): _own_postnorm_bwd}


# --------------------------------------------------------------------- work --
def work(case):
    c = case
    e = 2 if c["type"] == "bf16" else 4
    if c["op"] in ("conv", "scan"):
        n = [int(x) for x in c["lengths"].split(",")] if c["lengths"] else [c["T"]] * c["B"]
        M, N = sum(n), len(n)
    if c["op"] == "conv":
        C, W = c["C"], c["W"]
        state = N * (W - 1) * C
        if c["bwd"]:
            return {"bytes": 3 * M * C * e + state * (2 * e + 4) + 8 * C * (W + 1),
                    "flops": M * C * (6 * W + 8)}
        return {"bytes": 2 * M * C * e + 2 * state * e + 4 * C * (W + 1),
                "flops": M * C * (2 * W + 4)}
    if c["op"] == "scan":
        D, k, G = c["D"], c["N"], c["G"]
        par = 4 * D * (k + 2)
        if c["bwd"]:  # the forward, then the backward
            return {"bytes": 4 * M * D * e + 2 * M * G * k * e + N * D * k * 4 + par
                    + 7 * M * D * e + 4 * M * G * k * e + 3 * N * D * k * 4 + 2 * par,
                    "flops": M * D * k * (7 + 21)}
        return {"bytes": 4 * M * D * e + 2 * M * G * k * e + 2 * N * D * k * 4 + par,
                "flops": M * D * k * 7}
    M = c["rows"] * c["D"]
    if c["op"] == "prenorm":
        h = 2 if c["stream"] == "bf16" else 4
        per_channel = c["scale"] == "channel"
        if c["bwd"]:
            return {"bytes": M * (2 * e + 3 * h + (e if per_channel else 0)) + 8 * c["D"],
                    "flops": 12 * M}
        return {"bytes": M * (2 * e + 2 * h) + 4 * c["D"], "flops": 6 * M}
    rows = (3 if c["bwd"] else 2) + (0 if c["gate"] == "none" else 2 if c["bwd"] else 1)
    rows += 1 if c["residual"] and not c["bwd"] else 0
    return {"bytes": M * rows * e + 8 * c["D"], "flops": (18 if c["bwd"] else 8) * M}


# -------------------------------------------------------------------- exact --
def _bounds(s):
    if s["cu"] is None:
        B, T = s["x"].shape[:2]
        return [(i * T, i * T + T) for i in range(B)]
    c = s["cu"].tolist()
    return list(zip(c[:-1], c[1:]))


def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        return {"conv": _exact_conv, "scan": _exact_scan, "prenorm": _exact_prenorm,
                "postnorm": _exact_postnorm}[case["op"]](s)


def _exact_conv(s):
    """Sequence by sequence and block of channels by block: the convolution written as
    a sum over the joined history; gradients by differentiating it."""
    C, W = s["w"].shape
    B, T = s["x"].shape[:2]
    x = s["x"].reshape(B * T, C)
    y = torch.empty(B * T, C, dtype=torch.float64, device="cuda")
    parts = []
    for lo in range(0, C, 1024):
        ch = slice(lo, min(C, lo + 1024))
        leaf = lambda v: v.double().clone().requires_grad_(s["bwd"])  # noqa: E731
        xs, w, b, init = leaf(x[:, ch]), leaf(s["w"][ch]), leaf(s["b"][ch]), leaf(s["init"][:, :, ch])
        loss, fins = 0, []
        for i, (p, q) in enumerate(_bounds(s)):
            full = torch.cat([init[i], xs[p:q]])
            pre = b + sum(full[j:j + q - p] * w[:, j] for j in range(W))
            o, f = pre / (1 + torch.exp(-pre)), full[q - p:]
            if s["bwd"]:
                loss = loss + (o * s["dout"].reshape(B * T, C)[p:q, ch].double()).sum() \
                    + (f * s["dfin"][i, :, ch].double()).sum()
            else:
                y[p:q, ch] = o
                fins.append(f)
        parts.append(torch.autograd.grad(loss, (xs, w, b, init)) if s["bwd"] else torch.stack(fins))
    if not s["bwd"]:
        y = y.view(B, T, C)
        return [p.contiguous() for p in y.split([o.shape[2] for o in s["out"]], 2)], \
            torch.cat(parts, 2)
    dx, dw, db, di = zip(*parts)
    return {"dx": torch.cat(dx, 1).view(B, T, C), "dweight": torch.cat(dw), "dbias": torch.cat(db),
            "dinitial_state": torch.cat(di, 2)}


def _exact_scan(s):
    """Token by token in 64 bits, all sequences of a batch at once."""
    f = lambda k: s[k].double()  # noqa: E731
    Bq, T, D = s["x"].shape
    n = s["A_log"].shape[1]
    steps = T * (2 if s["bwd"] else 1)
    if steps > 80000 or (s["bwd"] and Bq * T * D * n > 1.2e9):
        return None
    G = s["B"].shape[2]
    A = -torch.exp(f("A_log"))
    Bm, Cm = (s[k].double().repeat_interleave(D // G, 2) if G > 1 else s[k].double() for k in ("B", "C"))
    ends = {q - 1: (i, p) for i, (p, q) in enumerate(_bounds(s)) if q > p} if s["cu"] is not None \
        else {}
    starts = {p: i for i, p in ends.values()}
    batched = s["cu"] is None
    x, v = f("x"), f("dt") + f("dt_bias")
    delta = torch.where(v > 30, v, torch.log1p(torch.exp(v)))
    y = torch.empty_like(x)
    fin = f("init")
    h = fin.clone() if batched else None
    kept = torch.empty(T, Bq, D, n, dtype=torch.float64, device="cuda") if s["bwd"] else None
    for t in range(T):
        if not batched and t in starts:
            h = fin[starts[t]][None]
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * x[:, t])[..., None] * Bm[:, t]
        y[:, t] = (h * Cm[:, t]).sum(-1)
        if s["bwd"]:
            kept[t] = h
        elif not batched and t in ends:
            fin[ends[t][0]] = h[0]
    if batched and T:
        fin = h
    y = y + f("D") * x
    z = f("z")
    sg = 1 / (1 + torch.exp(-z))
    out = y * z * sg
    if not s["bwd"]:
        return out, fin
    dout = f("dout")
    dy = dout * z * sg
    r = {"out": out, "dz": dout * y * sg * (1 + z * (1 - sg)), "dD": (dy * x).sum((0, 1)),
         "dx": dy * f("D"), "ddt": torch.empty_like(x), "dA_log": torch.zeros_like(A),
         "dB": torch.empty(Bq, T, G, n, dtype=torch.float64, device="cuda"),
         "dC": torch.empty(Bq, T, G, n, dtype=torch.float64, device="cuda")}
    dinit = f("dfin")
    g = dinit.clone() if batched else None
    for t in range(T - 1, -1, -1):
        if not batched and t in ends:
            g = dinit[ends[t][0]][None]
        g = g + dy[:, t, :, None] * Cm[:, t]
        if batched:
            prev = kept[t - 1] if t else f("init")
        else:
            prev = s["init"][starts[t]].double()[None] if t in starts else kept[t - 1]
        r["dC"][:, t] = (dy[:, t, :, None] * kept[t]).view(Bq, G, D // G, n).sum(2)
        u = (delta[:, t] * x[:, t])[..., None] * g
        r["dB"][:, t] = u.view(Bq, G, D // G, n).sum(2)
        gb = (g * Bm[:, t]).sum(-1)
        r["dx"][:, t] += gb * delta[:, t]
        g = g * torch.exp(delta[:, t, :, None] * A)
        w = g * prev
        r["ddt"][:, t] = gb * x[:, t] + (w * A).sum(-1)
        r["dA_log"] += (w * delta[:, t, :, None]).sum(0) * A
        if not batched and t in starts:
            dinit[starts[t]] = g[0]
    r["dinitial_state"] = g if batched else dinit
    r["ddt"] = r["ddt"] / (1 + torch.exp(-v))
    r["ddt_bias"] = r["ddt"].sum((0, 1))
    return r


def _exact_prenorm(s):
    sc = s["s"].double() if isinstance(s["s"], torch.Tensor) else s["s"]
    norm = lambda h, w: h / torch.sqrt((h ** 2).mean(-1, keepdim=True) + EPS) * w  # noqa: E731
    if not s["bwd"]:
        h = s["res"].double() + sc * s["x"].double()
        return norm(h, s["w"].double()), h
    h, w = s["h"].double().requires_grad_(), s["w"].double().requires_grad_()
    dh, dw = torch.autograd.grad((norm(h, w) * s["dout"].double()).sum(), (h, w))
    dh = dh + s["dh"].double()
    r = {"dx": dh * sc, "dresidual": dh, "dweight": dw}
    if isinstance(s["s"], torch.Tensor):
        r["dres_scale"] = (dh * s["x"].double()).sum(0)
    return r


def _exact_postnorm(s):
    leaf = lambda v: v.double().requires_grad_(s["bwd"]) if isinstance(v, torch.Tensor) else v  # noqa: E731
    x, w, sc, gate = leaf(s["x"]), leaf(s["w"]), leaf(s["s"]), leaf(s["gate"])
    y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS) * w
    if gate is not None:
        y = y / (1 + torch.exp(-gate)) * (gate if s["act"] == "silu" else 1)
    y = y * sc
    if not s["bwd"]:
        return y if s["res"] is None else y + s["res"].double()
    named = {"dx": x, "dweight": w, "dgate": gate, "dres_scale": sc}
    named = {k: v for k, v in named.items() if isinstance(v, torch.Tensor)}
    return dict(zip(named, torch.autograd.grad((y * s["dout"].double()).sum(), tuple(named.values()))))
