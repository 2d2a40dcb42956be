"""Helpers of the low-precision tests: making blocks on the host, uploading them,
and the error terms that the tolerances are built from."""
from __future__ import annotations

import numpy as np
import torch

from oracle import moe_oracle as O

U32 = 2.0 ** -24                     # half a step of fp32, relative
U_ACT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
# An fp32 sum on the matrix cores: each of n terms joins with an error of at
# most one step (2^-23) of the sum of magnitudes.
def gamma(n):   # noqa: E302
    return (n + 8) * 2.0 ** -23


def rnd(a, dtype):
    """fp64 values of `a` rounded to dtype"""
    return torch.from_numpy(np.asarray(a)).to(dtype).double().numpy()


def up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host64(t):
    return t.detach().double().cpu().numpy()


def blocks(v, fmt):
    """(bytes of elements, padded scale bytes, their fp64 values) of v [..., n]"""
    q, s = O.mx_quantize(v, fmt)
    if fmt == "e4m3":
        codes = torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    else:
        table = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
        c = np.searchsorted(table, np.abs(q)).astype(np.uint8) | (np.signbit(q) << 3).astype(np.uint8)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    pad = np.zeros((*s.shape[:-1], O.mx_scale_cols(v.shape[-1])), np.uint8)
    pad[..., :s.shape[-1]] = s
    return codes, pad, O.mx_values(q, s)


def weights(rng, E, n, width, spread=3):
    """e2m1 weights [E, n, width] whose blocks differ in scale"""
    v = rng.normal(size=(E, n, width)) * width ** -0.5
    v = v * 2.0 ** rng.integers(-spread, spread + 1, size=(E, n, width // 32)).repeat(32, -1)
    return blocks(v, "e2m1")


def within(got, want, bound, what):
    """every element within its bound; NaNs only where the oracle has them"""
    got, want, bound = (np.asarray(a, np.float64) for a in (got, want, bound))
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaNs differ"
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    d, b = np.abs(got - want)[fine], np.broadcast_to(bound, want.shape)[fine]
    worst = float(np.max(d / np.maximum(b, 1e-300))) if d.size else 0.0
    print(f"[{what}] worst error / bound {worst:.3f}", flush=True)
    assert (d <= b).all(), f"{what}: {worst:.2f} times its bound"


def random_blocks(rng, shape, fmt, scales=(118, 124)):
    """random elements and scales: (bytes, padded scale bytes, fp64 values)"""
    n = shape[-1]
    if fmt == "e4m3":
        codes = torch.from_numpy(rng.normal(size=shape) * 4).float().to(torch.float8_e4m3fn)
        codes = codes.view(torch.uint8).numpy()
    else:
        codes = rng.integers(0, 256, size=(*shape[:-1], n // 2)).astype(np.uint8)
    scale = np.zeros((*shape[:-1], O.mx_scale_cols(n)), np.uint8)
    scale[..., :n // 32] = rng.integers(scales[0], scales[1], size=(*shape[:-1], n // 32))
    return codes, scale, O.mx_values(O.mx_element_values(codes, fmt), scale)


def block_max(v):
    """largest |value| of each block of 32"""
    return np.abs(v).reshape(*v.shape[:-1], -1, 32).max(-1)


def mx_dot_bound(x, w):
    """error of the block-scaled matrix instruction's x w^T, [n, K] by [N, K].

    It aligns the products of a block to the largest power of two among them and
    drops what lies below 2^-13 of it (two products 2^10 that cancel keep a third
    of 2^-3 and lose one of 2^-4; blocks apart keep each other): each of 32 terms
    loses less than 2^-13 max|x| max|w|.  The blocks' sums then join in fp32."""
    lost = 32 * 2.0 ** -13 * (block_max(x) @ block_max(w).T)
    return lost + gamma(x.shape[1] // 32) * (np.abs(x) @ np.abs(w).T + lost)


def plain_dot_bound(x, w):
    """error of an fp32 sum of exact products"""
    return gamma(x.shape[1]) * (np.abs(x) @ np.abs(w).T)


def hidden_bound(x, w1, w3, a, b, h, dot_bound=plain_dot_bound):
    """error of fp32 h = silu(a) b: |silu'| <= 1.1; the exponential and the
    reciprocal a few steps, the former growing with |a|"""
    ea, eb = dot_bound(x, w1), dot_bound(x, w3)
    with np.errstate(all="ignore"):
        silu = np.abs(a / (1 + np.exp(-a)))
    return 1.1 * ea * (np.abs(b) + eb) + silu * eb + np.abs(h) * (8 + 2 * np.abs(a)) * U32
