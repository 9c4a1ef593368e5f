"""Arguments of the layer operators that are no tensors are refused as a TypeError that names
them, wherever they stand (no GPU)."""
import pytest
import torch

import kimi_delta_attention_08_gb300 as kda

x, w, b = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(8)
A, B = torch.zeros(8, 16), torch.zeros(2, 5, 1, 16)
CALLS = [
    (kda.kda_conv_fwd, dict(x=x, weight=w, bias=b, out=x, initial_state=None, cu_seqlens=None, workspace=None),
     dict(weight="weight", out="out", bias="bias", initial_state="initial_state", cu_seqlens="cu_seqlens")),
    (kda.kda_conv_bwd, dict(x=x, weight=w, bias=b, dout=x, workspace=None),
     dict(weight="weight", dout="dout", bias="bias", workspace="workspace")),
    (kda.kda_scan_fwd, dict(x=x, dt=x, A_log=A, B=B, C=B, out=x),
     dict(dt="dt", A_log="A_log", B="B", C="C", out="out", z="z", D="D", dt_bias="dt_bias",
          initial_state="initial_state", final_state="initial_state", chunk_states="chunk_states",
          workspace="workspace")),
    (kda.kda_scan_bwd, dict(x=x, dt=x, A_log=A, B=B, C=B, dout=x), dict(dout="dout", z="z", workspace="workspace")),
    (kda.kda_prenorm_fwd, dict(x=x, residual=None, weight=b, out=x),
     dict(residual="residual", weight="weight", out="out")),
    (kda.kda_prenorm_bwd, dict(dout=x, dresidual_out=None, h=x, weight=b), dict(dout="dout", h="h")),
    (kda.kda_postnorm_fwd, dict(x=x, weight=b, gate=None, out=x), dict(weight="weight", gate="gate", out="out")),
    (kda.kda_postnorm_bwd, dict(dout=x, x=x, weight=b), dict(gate="gate")),
]


@pytest.mark.parametrize("call,args,wrong", CALLS, ids=[c[0].__name__ for c in CALLS])
def test_what_is_no_tensor_is_named(call, args, wrong):
    first = next(iter(args))
    for name, said in {first: first, **wrong}.items():
        with pytest.raises(TypeError, match=said):
            call(**{**args, name: 5.0})


def test_lists_of_outputs():
    for outs, error in (([], ValueError), ([x] * 5, ValueError), ([x, None], TypeError), (None, TypeError)):
        with pytest.raises(error):
            kda.kda_conv_fwd(x, w, b, outs)
        with pytest.raises(error):
            kda.kda_conv_bwd(x, w, b, outs)
