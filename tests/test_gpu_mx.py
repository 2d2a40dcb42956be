"""GPU: rows to and from the block-scaled formats, bit for bit with the oracle
(inputs are exact, dividing by a power of two is exact, one rounding each)."""
import numpy as np
import pytest
import torch

import top_routing_grouped_router_amd as M
from oracle import moe_oracle as O

from _lowp import host64, up

pytestmark = pytest.mark.gpu


def _rows(rng, rows, cols, fmt):
    v = rng.normal(size=(rows, cols)) * 2.0 ** rng.integers(-20, 20, size=(rows, 1))
    flat = v.reshape(-1, 32)
    top = O.MX_FORMATS[fmt][0]
    flat[0] = 0.0
    n = flat.shape[0]
    flat[1 % n, :4] = [top * 4, -top * 4, top * 2, 1e-30]        # exactly the largest
    flat[2 % n, 3] = np.float32(flat[2 % n].max() + 1)
    if n > 8:
        flat[3, 0] = top * (1 + 2.0 ** -7)                       # just above it
        flat[4] = 2.0 ** -149 * np.arange(32)                    # fp32 subnormals
        flat[5] = np.linspace(-1, 1, 32) * 3e38                  # near fp32's largest
        flat[6] = np.r_[6.0, np.arange(31) * 0.25 - 3.5]         # ties of e2m1
        flat[7] = np.r_[448.0, 2.0 ** -9 * (np.arange(31) - 15) / 2]   # subnormals of e4m3, ties
    return v


@pytest.mark.parametrize("rows,cols", [(1, 64), (3, 128), (5, 192), (37, 320), (130, 2048)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_rows_round_trip(fmt, dtype, rows, cols):
    print(f"\n[case] mx {fmt} {dtype} {rows}x{cols}", flush=True)
    rng = np.random.default_rng(rows * cols)
    src = up(_rows(rng, rows, cols, fmt), dtype)
    q = torch.full((rows, cols if fmt == "e4m3" else cols // 2), 0xA5, dtype=torch.uint8,
                   device="cuda")
    scale = torch.full((rows, O.mx_scale_cols(cols)), 0xA5, dtype=torch.uint8, device="cuda")
    M.moe_mx_quantize(src, fmt, q, scale)
    want, s = O.mx_quantize(host64(src), fmt)
    got_s = scale.cpu().numpy()
    assert np.array_equal(got_s[:, :cols // 32], s)
    assert (got_s[:, cols // 32:] == 0).all()
    assert np.array_equal(O.mx_element_values(q.cpu().numpy(), fmt), want)
    back = torch.full_like(src, float("nan"))
    M.moe_mx_dequantize(q, scale, fmt, back)
    ref = torch.from_numpy(O.mx_values(want, s)).to(dtype)   # one rounding (subnormals)
    assert torch.equal(back.cpu(), ref)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_non_finite_blocks_read_as_nan(fmt, dtype):
    print(f"\n[case] mx non-finite {fmt} {dtype}", flush=True)
    src = torch.ones(4, 192, dtype=dtype)
    src[0, 33] = float("nan")
    src[1, 64] = float("inf")
    src[3, 191] = float("-inf")
    src = src.cuda()
    q = torch.empty(4, 192 if fmt == "e4m3" else 96, dtype=torch.uint8, device="cuda")
    scale = torch.empty(4, 8, dtype=torch.uint8, device="cuda")
    M.moe_mx_quantize(src, fmt, q, scale)
    back = torch.empty_like(src)
    M.moe_mx_dequantize(q, scale, fmt, back)
    nan = torch.isnan(back).cpu().reshape(4, 6, 32)
    want = torch.zeros(4, 6, dtype=torch.bool)
    want[0, 1] = want[1, 2] = want[3, 5] = True
    assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)
    assert (back.cpu().reshape(4, 6, 32)[~want] == 1).all()
    assert (scale.cpu()[:, :6][want] == 255).all()


def test_every_element_under_every_scale():
    """all 256 bytes, every scale, both formats, against the definition"""
    print("\n[case] mx all codes", flush=True)
    for fmt in ("e4m3", "e2m1"):
        per = 256 if fmt == "e4m3" else 512
        q = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()
        scale = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, O.mx_scale_cols(per)).cuda()
        out = torch.empty(256, per, device="cuda")
        M.moe_mx_dequantize(q, scale, fmt, out)
        el = O.mx_element_values(q.cpu().numpy(), fmt)
        with np.errstate(over="ignore"):
            want = O.mx_values(el, scale.cpu().numpy()).astype(np.float32)
        assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


def test_no_rows():
    for fmt in ("e4m3", "e2m1"):
        src = torch.empty(0, 128, device="cuda")
        q = torch.empty(0, 128 if fmt == "e4m3" else 64, dtype=torch.uint8, device="cuda")
        scale = torch.empty(0, 4, dtype=torch.uint8, device="cuda")
        M.moe_mx_quantize(src, fmt, q, scale)
        M.moe_mx_dequantize(q, scale, fmt, src)
