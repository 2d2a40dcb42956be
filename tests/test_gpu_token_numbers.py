"""GPU: what the experts of a few tokens keep of single values, on either way through
them (each pair by itself, up to 8 tokens; each expert's pairs together)."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O

from test_gpu_token import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [3, 12])
@pytest.mark.parametrize("bits", [0x7FFFFFFF, 0xFFFFFFFF, 0x7F800001, 0x7FC00000])
def test_a_gate_of_any_nan_gives_nan(act, T, bits):
    print(f"\n[case] token NaN gate {T} {bits:#x} {act}", flush=True)
    c = Case(T, 128, 8, 64, 2, act, seed=T)
    c.upload()
    c.run()
    ref = c.y.clone()
    c.g["gate"].view(torch.int32)[1, 1] = np.uint32(bits).astype(np.int32).item()
    c.run()
    assert torch.isnan(c.y[1]).all()
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(c.y[rest], ref[rest])
