"""The buffer of kept pre-activations on the host: its types, shape and device."""
import pytest
import torch

from kimi_delta_attention_08_gb300 import layer

CPU = torch.device("cpu")


def test_types():
    for ty in (torch.int16, torch.bfloat16):
        t = torch.zeros(2, 3, 32, dtype=ty)
        assert layer._pre(t, CPU, None, (2, 3, 32)) == t.data_ptr()
    assert layer._pre(None, CPU, None, (2, 3, 32)) is None
    for bad in (torch.zeros(2, 3, 32), torch.zeros(2, 3, 32, dtype=torch.float16),
                torch.zeros(2, 3, 32, dtype=torch.uint16), torch.zeros(2, 3, 64, dtype=torch.uint8), 3):
        with pytest.raises(TypeError, match="pre"):
            layer._pre(bad, CPU, None, (2, 3, 32))


@pytest.mark.parametrize("ty", [torch.int16, torch.bfloat16])
def test_shapes(ty):
    for bad in (torch.zeros(2, 3, 16, dtype=ty), torch.zeros(2, 3, 64, dtype=ty)[..., ::2],
                torch.zeros(2, 3, 32, dtype=ty, device="meta")):
        with pytest.raises(ValueError, match="pre"):
            layer._pre(bad, CPU, None, (2, 3, 32))
