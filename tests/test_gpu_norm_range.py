"""GPU: the norm's statistics over the whole range of fp32, and to the last bit that
the 8-bit rows depend on.

rstd is a 64-bit value rounded to fp32: half a step.  y is two fp32 products of it,
rounded to act.
"""
import numpy as np
import pytest
import torch

import top_routing_grouped_router_amd as M
from oracle import moe_oracle as O

from _lowp import U32, U_ACT, host64, up, within
from test_gpu_norm import _bwd, _check_bwd, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 320, 2048, 16448])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e37, 1e30, 3e19, 1.0, 1e-20, 1e-25, 1e-36])
def test_rows_of_any_size(d, dtype, size):
    print(f"\n[case] norm size {size} d={d} {dtype}", flush=True)
    rng = np.random.default_rng(d)
    x = up(np.clip(rng.normal(size=(5, d)), -4, 4) * size, dtype)
    w = up(1 + 0.3 * rng.normal(size=d), torch.float32)
    o = _run(x, None, w, eps=0.0, total=False)
    y, rstd = O.rmsnorm(host64(x), host64(w), 0.0)
    within(host64(o["rstd"]), rstd, rstd * U32 * 1.001, "rstd")
    within(host64(o["y"]), y, np.abs(y) * (U_ACT[dtype] + 4 * U32) + 1e-38, "y")
    v = O.mx_values(O.mx_element_values(o["q"].cpu().numpy(), "e4m3"), o["scale"].cpu().numpy())
    want, scale = O.mx_quantize(y, "e4m3")
    want = O.mx_values(want, scale)
    assert (v != want).sum() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e30, 3e19])
def test_gradients_of_large_rows(dtype, size):
    print(f"\n[case] norm backward size {size} {dtype}", flush=True)
    rng = np.random.default_rng(3)
    x = up(rng.normal(size=(9, 256)) * size, dtype)
    w = up(1 + 0.3 * rng.normal(size=256), torch.float32)
    dy = up(rng.normal(size=(9, 256)), dtype)
    dx, dw = _bwd(x, w, dy, None)
    _check_bwd(x, w, dy, None, dx, dw)


@pytest.mark.parametrize("T,d", [(2, 64), (3, 320), (2, 2048), (2, 4096), (2, 16448), (2, 40000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_elements_next_to_ties_of_any_rows(T, d, dtype):
    """a weight that puts every y of the first row within a rounding of a tie between
    elements, or of its scale's limit; the squares fill more than 24 bits, and so do
    their sums.  y is computed to about 2^-45, and the closest one lies further from
    its tie than that (checked)."""
    print(f"\n[case] norm ties of any rows {T}x{d} {dtype}", flush=True)
    rng = np.random.default_rng(d + T)
    x = up(rng.normal(size=(T, d)), dtype)
    x[x == 0] = 1
    s = host64(x)
    tie = (8 + rng.integers(0, 8, size=d) + 0.5) / 8 * 2.0 ** rng.integers(-3, 8, size=d)
    tie[::32] = rng.choice([448.0, 400.0], size=d // 32)
    tie[tie > 448] = 232.0
    eps = float(np.float32(1e-6))
    w = up(tie / (np.abs(s[0]) / np.sqrt(np.mean(s[0] * s[0]) + eps)), torch.float32)
    y, _ = O.rmsnorm(s, host64(w), eps)
    off = np.abs(np.abs(y[0]) / tie - 1)
    assert (off <= 2.0 ** -24).all() and (off > 2.0 ** -42).all()
    o = _run(x, None, w, total=False)
    want, scale = O.mx_quantize(y, "e4m3")
    assert (o["scale"].cpu().numpy()[:, :d // 32] == scale).all()
    v = O.mx_element_values(o["q"].cpu().numpy(), "e4m3")
    bad = np.argwhere(v != want)
    assert not len(bad), (len(bad), bad[:5], v[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("d", [256, 1024, 20032])
@pytest.mark.parametrize("over", ["x", "residual"])
@pytest.mark.parametrize("total", [False, True])
def test_y_over_an_input(d, over, total):
    """with the sum in the other input, in a tensor of its own, or nowhere"""
    print(f"\n[case] norm y over {over} {total} d={d}", flush=True)
    rng = np.random.default_rng(d)
    x, r = (up(rng.normal(size=(40, d)), torch.bfloat16) for _ in range(2))
    w = up(1 + 0.3 * rng.normal(size=d), torch.float32)
    dims = M.make_dims(40, d, 1, 64, 1, torch.bfloat16)
    ref = _run(x, r, w)
    for own in ([False, True] if total else [False]):
        a, b = x.clone(), r.clone()
        y, other = (a, b) if over == "x" else (b, a)
        s = None if not total else torch.empty_like(x) if own else other
        M.moe_rmsnorm(dims, a, b, w, 1e-6, s, y, None, None, None)
        assert torch.equal(y, ref["y"]) and (s is None or torch.equal(s, ref["sum"]))
