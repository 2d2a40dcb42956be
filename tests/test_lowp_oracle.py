"""Pins of the oracle's norm and block-scaled numbers (CPU): torch's own e4m3
conversion, brute force over the formats' values, finite differences."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_elements_are_the_nearest_of_all_and_ties_are_even(fmt):
    codes = np.arange(256 if fmt == "e4m3" else 8, dtype=np.uint8)
    if fmt == "e4m3":
        vals = O.mx_element_values(codes, fmt)
        ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(vals, ref, equal_nan=True)
        grid = np.unique(vals[np.isfinite(vals)])
    else:
        vals = O.mx_element_values(codes * 0x11, fmt)[::2]
        assert vals.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
        grid = np.unique(np.concatenate([vals, -vals]))
    rng = np.random.default_rng(0)
    mids = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([np.clip(rng.normal(size=4096) * 2, grid[0], grid[-1]), mids, grid])
    v = np.concatenate([v, np.zeros(-v.size % 31)]).reshape(-1, 31)
    top = O.MX_FORMATS[fmt][0]
    v = np.concatenate([np.full((v.shape[0], 1), top), v], 1)      # scale 2^0 in every block
    q, s = O.mx_quantize(v, fmt)
    assert (s == 127).all()
    best = np.abs(v[..., None] - grid).min(-1)
    assert np.array_equal(np.abs(q - v), best)
    if fmt == "e4m3":   # torch rounds ties to even
        assert np.array_equal(q, torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy())
    else:
        tie = {0.25: 0, 0.75: 1, 1.25: 1, 1.75: 2, 2.5: 2, 3.5: 4, 5.0: 4}
        for x, want in tie.items():
            b = np.zeros((1, 32))
            b[0, :2] = 6.0, x
            assert O.mx_quantize(b, fmt)[0][0, 1] == want


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_scale_is_the_smallest_that_fits(fmt):
    top = O.MX_FORMATS[fmt][0]
    for amax, s in ((top, 127), (np.nextafter(top, 1e9), 128), (top / 2, 126), (0.0, 0),
                    (top * 2.0 ** -127, 0), (top * 2.0 ** -140, 0), (top * 2.0 ** 100, 227)):
        b = np.zeros((1, 64))
        b[0, 7] = -amax
        assert O.mx_quantize(b, fmt)[1].tolist() == [[s, 0]]
    for bad in (np.nan, np.inf, -np.inf):
        b[0, 7] = bad
        q, s = O.mx_quantize(b, fmt)
        assert s.tolist() == [[255, 0]] and np.isnan(q[0, :32]).all()
        assert np.isnan(O.mx_values(q, s)[0, :32]).all()


def test_norm_backward_against_differences():
    rng = np.random.default_rng(1)
    s, w, dy = rng.normal(size=(3, 64)), rng.normal(size=64), rng.normal(size=(3, 64))
    dx, dw = O.rmsnorm_bwd(dy, s, w, 1e-3)
    f = lambda a, b: (O.rmsnorm(a, b, 1e-3)[0] * dy).sum()   # noqa: E731
    h = 1e-6
    for at in [(0, 0), (1, 17), (2, 63)]:
        p, m = s.copy(), s.copy()
        p[at] += h
        m[at] -= h
        assert abs((f(p, w) - f(m, w)) / (2 * h) - dx[at]) < 1e-8
        p, m = w.copy(), w.copy()
        p[at[1]] += h
        m[at[1]] -= h
        assert abs((f(s, p) - f(s, m)) / (2 * h) - dw[at[1]]) < 1e-7
    base = O.rmsnorm_bwd(dy, s, w, 1e-3, dsum=s)[0]
    assert np.allclose(base - s, dx)
    y, rstd = O.rmsnorm(s, np.ones(64), 0.0)
    assert np.allclose((y * y).mean(-1), 1.0) and np.allclose(rstd, 1 / np.sqrt((s * s).mean(-1)))


def test_token_experts_are_the_layer():
    rng = np.random.default_rng(2)
    T, d, E, f, k = 5, 64, 6, 64, 3
    x = rng.normal(size=(T, d))
    w1, w3, w2 = rng.normal(size=(E, f, d)), rng.normal(size=(E, f, d)), rng.normal(size=(E, d, f))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    gate = rng.random((T, k))
    wr = rng.normal(size=(E, d)).astype(np.float32)
    ref = O.layer_forward(x, wr, w1, w3, w2, k, routing=(idx, gate))["y"]
    assert np.allclose(O.token_swiglu(x, idx, gate, w1, w3, w2), ref)
    idx[2, 1] = -1
    drop = O.token_swiglu(x, idx, gate, w1, w3, w2)
    assert np.allclose(np.delete(drop, 2, 0), np.delete(ref, 2, 0)) and not np.allclose(drop[2], ref[2])
