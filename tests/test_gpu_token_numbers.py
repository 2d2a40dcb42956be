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


def _weight(shape, codes, scale):
    """e2m1 weights of `shape`, zeros but for codes at (row, column), and a scale byte"""
    code = np.zeros(shape, np.uint8)
    for (row, col), v in codes.items():
        code[..., row, col] = v
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    s = np.zeros((*shape[:-1], O.mx_scale_cols(shape[-1])), np.uint8)
    s[..., :shape[-1] // 32] = scale
    return packed, s, O.mx_values(O.mx_element_values(packed, "e2m1"), s)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [2, 12])
def test_the_hidden_values_are_rounded(act, T):
    """h = 32 (1 + 65535 / 2^23), 24 significant bits, less 32 (1 + 255 / 2^15), 16 of
    them: what is left is 32 * 255 / 2^23, less than half a step of 16 bits off if h is
    rounded to them (a step of 32 is 2^-10), all of it if the rest of h is cut."""
    print(f"\n[case] token rounding of h {T} {act}", flush=True)
    c = Case(T, 64, 4, 64, 1, act, seed=1)
    c.idx[:], c.gate[:] = 2, 1.0
    c.x[:] = 0
    c.x[:, 0], c.x[:, 8], c.x[:, 16] = 1.0, 255 / 2 ** 15, 255 / 2 ** 23
    one, four, minus_one = 2, 6, 10     # codes of 1, 4 and -1
    c.w1 = _weight((4, 64, 64), {(0, 0): four, (1, 0): four}, 127 + 3)   # a = 32: silu(a) = a
    c.w3 = _weight((4, 64, 64), {(0, 0): one, (0, 8): one, (0, 16): one, (1, 0): one, (1, 8): one},
                   127)
    c.w2 = _weight((4, 64, 64), {(n, j): (one, minus_one)[j] for n in range(64) for j in (0, 1)},
                   127)
    c.upload()
    c.run()
    want = 32 * 255 / 2 ** 23
    tol = (2.0 ** -11 + 2.0 ** -8 * want if act == torch.bfloat16 else 64 * 2.0 ** -24)
    off = (c.y.double() - want).abs().max().item()
    print(f"off by {off / want:.3f} of it, bound {tol / want:.3f}", flush=True)
    assert off < tol
