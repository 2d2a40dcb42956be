"""GPU: the norm before the layer and its backward against the oracle in 64 bits.

Bounds.  The norm is of the stored sum, so it is given exactly.  mean(s^2) is a
sum of d positive fp32 terms: relative error (d + 2) u, halved by the root; the
root, the division and the two products add a step each.  y is rounded once.
dx: the mean of g n is a sum of d terms, its error n times (d + 4) u mean|g n|;
each factor carries the error of rstd.  dweight: T terms, any order.
"""
import numpy as np
import pytest
import torch

import top_routing_grouped_router_amd as M
from oracle import moe_oracle as O

from _lowp import U32, U_ACT, host64, up, within

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _inputs(T, d, dtype, seed, res=True):
    rng = np.random.default_rng(seed)
    x = up(rng.normal(size=(T, d)), dtype)
    r = up(rng.normal(size=(T, d)) * 2, dtype) if res else None
    w = up(1 + 0.3 * rng.normal(size=d), torch.float32)
    return x, r, w


def _dims(T, d, dtype):
    return M.make_dims(T, d, 1, 64, 1, dtype)


def _run(x, r, w, eps=EPS, quant=True, y=True, total=True):
    T, d = x.shape
    o = {"sum": torch.full_like(x, float("nan")) if total else None,
         "y": torch.full_like(x, float("nan")) if y else None,
         "rstd": torch.full((T,), float("nan"), device="cuda"), "q": None, "scale": None}
    if quant:
        o["q"] = torch.full((T, d), 0xA5, dtype=torch.uint8, device="cuda")
        o["scale"] = torch.full((T, O.mx_scale_cols(d)), 0xA5, dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm(_dims(T, d, x.dtype), x, r, w, eps, o["sum"], o["y"], o["q"], o["scale"],
                  o["rstd"])
    return o


def _stored(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def _check(x, r, w, o, eps=EPS):
    T, d = x.shape
    s = _stored(x, r)
    if o["sum"] is not None:
        assert torch.equal(o["sum"], s)
    with np.errstate(all="ignore"):
        y, rstd = O.rmsnorm(host64(s), host64(w), eps)
    e = (d / 2 + 6) * U32
    within(host64(o["rstd"]), rstd, np.abs(rstd) * e, "rstd")
    if o["y"] is not None:
        within(host64(o["y"]), y, np.abs(y) * (U_ACT[x.dtype] + e + 2 * U32) + 1e-38, "y")
    if o["q"] is not None:
        got_s = o["scale"].cpu().numpy()
        assert (got_s[:, d // 32:] == 0).all()
        sc = 2.0 ** (got_s[:, :d // 32].astype(np.float64) - 127)
        amax = np.abs(y).reshape(T, -1, 32).max(-1)
        ok = np.isfinite(amax)
        assert (got_s[:, :d // 32][~ok] == 255).all()
        with np.errstate(invalid="ignore"):
            fits = (amax <= 448 * sc * (1 + e)) & ((amax >= 224 * sc * (1 - e)) | (got_s[:, :d // 32] == 0))
        assert fits[ok].all(), "scale"
        v = O.mx_values(O.mx_element_values(o["q"].cpu().numpy(), "e4m3"), got_s)
        step = np.repeat(sc, 32, -1) * 2.0 ** -10   # half a step of the subnormal elements
        fine = np.repeat(ok, 32, -1)
        within(np.where(fine, v, 0), np.where(fine, y, 0),
               np.maximum(2.0 ** -4 * np.abs(y), step) + np.abs(y) * 2 * e, "q")
        assert np.isnan(v[~fine]).all()


SHAPES = [(1, 64), (1, 2048), (3, 128), (5, 320), (7, 576), (67, 1024), (33, 2048), (9, 4160),
          (5, 8192), (3, 16384), (2, 16448), (2, 40000)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("res", [True, False])
def test_norm(T, d, dtype, res):
    d = d // 64 * 64
    print(f"\n[case] norm {T}x{d} {dtype} res={res}", flush=True)
    x, r, w = _inputs(T, d, dtype, T + d, res)
    _check(x, r, w, _run(x, r, w, total=res))


@pytest.mark.parametrize("T,d", [(1, 64), (3, 320), (2, 2048), (2, 16448), (2, 40000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_elements_next_to_ties(T, d, dtype):
    """rows of small integers, whose squares add up exactly, and a weight that puts every
    y of the first row within a rounding of a tie between elements, or of its scale's
    limit: each element is still the rounding of y.  rstd is good to 2^-45, y to
    2^-43, and the closest y lies further from its tie than that (checked)."""
    d = d // 64 * 64
    print(f"\n[case] norm ties {T}x{d} {dtype}", flush=True)
    rng = np.random.default_rng(d)
    s = rng.integers(1, 12, size=(T, d)) * rng.choice([-1, 1], size=(T, d))
    tie = (8 + rng.integers(0, 8, size=d) + 0.5) / 8 * 2.0 ** rng.integers(-3, 8, size=d)
    tie[::32] = rng.choice([448.0, 400.0], size=d // 32)
    tie[tie > 448] = 232.0
    rstd = 1 / np.sqrt(np.mean(s[0] * s[0]) + float(np.float32(EPS)))
    w = up(tie / (np.abs(s[0]) * rstd), torch.float32)
    x = up(s, dtype)
    y, _ = O.rmsnorm(s, host64(w), float(np.float32(EPS)))
    off = np.abs(np.abs(y[0]) / tie - 1)
    assert (off <= 2.0 ** -24).all() and (off > 2.0 ** -42).all()
    o = _run(x, None, w, total=False)
    want, scale = O.mx_quantize(y, "e4m3")
    got_s = o["scale"].cpu().numpy()
    assert (got_s[:, :d // 32] == scale).all()
    v = O.mx_element_values(o["q"].cpu().numpy(), "e4m3")
    bad = np.argwhere(v != want)
    assert not len(bad), (len(bad), bad[:5], v[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 64), (torch.float32, 320),
                                     (torch.bfloat16, 448), (torch.float32, 1024),
                                     (torch.bfloat16, 2048), (torch.bfloat16, 2112)])
def test_norm_of_many_rows(dtype, d):
    """the layout of a wavefront per row, with a ragged last workgroup"""
    print(f"\n[case] norm many rows d={d} {dtype}", flush=True)
    x, r, w = _inputs(1027, d, dtype, d)
    _check(x, r, w, _run(x, r, w))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_odd_rows(dtype):
    """rows of zeros (eps decides), large and small rows, infinities and NaNs: each
    row on its own"""
    print(f"\n[case] norm odd rows {dtype}", flush=True)
    x, _, w = _inputs(9, 192, dtype, 3)
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-15
    x[3, 5] = float("nan")
    x[5, 100] = float("inf")
    x[7] = 0
    x[7, 3] = 1
    o = _run(x, None, w, total=False)
    keep = [0, 1, 2, 4, 6, 7, 8]
    part = {n: (None if t is None else t[keep].contiguous()) for n, t in o.items()}
    _check(x[keep].contiguous(), None, w, part)
    assert torch.isnan(o["y"][3]).all() and (o["scale"][3, :6] == 255).all()
    # an infinite value makes rstd 0: that value NaN, the others zeros
    bad = torch.isnan(o["y"][5])
    assert bad[100] and bad.sum() == 1 and (o["y"][5][~bad] == 0).all()
    assert o["scale"][5, :6].tolist() == [0, 0, 0, 255, 0, 0]
    # eps = 0 on a row of zeros: 0 * inf
    z = _run(torch.zeros(2, 64, dtype=dtype, device="cuda"), None, w[:64].contiguous(), eps=0.0,
             total=False)
    assert torch.isinf(z["rstd"]).all() and torch.isnan(z["y"]).all()


@pytest.mark.parametrize("d", [256, 20032])
def test_norm_in_place_and_partial_outputs(d):
    print(f"\n[case] norm in place d={d}", flush=True)
    x, r, w = _inputs(5, d, torch.bfloat16, 11)
    ref = _run(x, r, w)
    dims = _dims(5, d, torch.bfloat16)
    for over in ("x", "r"):
        a, b = x.clone(), r.clone()
        out = torch.empty_like(x)
        M.moe_rmsnorm(dims, a, b, w, EPS, a if over == "x" else b, out, None, None, None)
        assert torch.equal(out, ref["y"]) and torch.equal(a if over == "x" else b, ref["sum"])
        assert torch.equal(b if over == "x" else a, r if over == "x" else x)
    a = x.clone()
    M.moe_rmsnorm(dims, a, r, w, EPS, None, a, None, None, None)
    assert torch.equal(a, ref["y"])
    q, sc = torch.empty_like(ref["q"]), torch.empty_like(ref["scale"])
    M.moe_rmsnorm(dims, x, r, w, EPS, None, None, q, sc, None)
    assert torch.equal(q, ref["q"]) and torch.equal(sc, ref["scale"])


def _bwd(x, w, dy, dsum, dx=None, rstd=None):
    T, d = x.shape
    dims = _dims(T, d, x.dtype)
    if rstd is None:
        rstd = _run(x, None, w, quant=False, total=False)["rstd"]
    dx = torch.full_like(x, float("nan")) if dx is None else dx
    dw = torch.full((d,), float("nan"), device="cuda")
    ws = torch.full((max(M.moe_rmsnorm_bwd_workspace_bytes(dims), 16),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    M.moe_rmsnorm_bwd(dims, dy, x, w, rstd, dsum, dx, dw, ws)
    return dx, dw


def _check_bwd(x, w, dy, dsum, dx, dw):
    T, d = x.shape
    s, w6, g6 = host64(x), host64(w), host64(dy)
    want, dwant = O.rmsnorm_bwd(g6, s, w6, EPS, None if dsum is None else host64(dsum))
    _, rstd = O.rmsnorm(s, w6, EPS)
    n, g = np.abs(s * rstd[:, None]), np.abs(g6 * w6)
    e = (d / 2 + 8) * U32
    c = np.mean(g * n, -1, keepdims=True)
    bound = rstd[:, None] * ((g + n * c) * 3 * e + n * c * (d + 8) * U32) + 4 * U32 * np.abs(want)
    within(host64(dx), want, bound + U_ACT[x.dtype] * np.abs(want) + 1e-38, "dx")
    within(host64(dw), dwant, (np.abs(g6) * n).sum(0) * (T + 8) * U32 + (np.abs(g6) * n).sum(0) * e,
           "dweight")


@pytest.mark.parametrize("T,d", [(1, 64), (2, 2048), (5, 320), (67, 576), (1027, 256), (515, 2048),
                                 (9, 4096), (4, 8192), (11, 8256), (2063, 64), (3, 40000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dsum", [True, False])
def test_norm_backward(T, d, dtype, dsum):
    d = d // 64 * 64
    print(f"\n[case] norm backward {T}x{d} {dtype} dsum={dsum}", flush=True)
    x, ds, w = _inputs(T, d, dtype, T * 7 + d, dsum)
    dy = up(np.random.default_rng(d).normal(size=(T, d)), dtype)
    dx, dw = _bwd(x, w, dy, ds)
    _check_bwd(x, w, dy, ds, dx, dw)
    again = _bwd(x, w, dy, ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("T,d,dtype", [(523, 8256, torch.bfloat16), (523, 4160, torch.float32),
                                       (129, 2112, torch.bfloat16), (513, 1024, torch.float32),
                                       (2051, 2048, torch.bfloat16), (511, 1600, torch.bfloat16)])
def test_norm_backward_of_several_rows_each(T, d, dtype):
    """rows that take a workgroup, more of them than workgroups"""
    print(f"\n[case] norm backward several rows {T}x{d} {dtype}", flush=True)
    x, ds, w = _inputs(T, d, dtype, T + d, True)
    dy = up(np.random.default_rng(d).normal(size=(T, d)), dtype)
    dx, dw = _bwd(x, w, dy, ds)
    _check_bwd(x, w, dy, ds, dx, dw)


@pytest.mark.parametrize("d", [256, 4096, 20032])
def test_norm_backward_in_place(d):
    print(f"\n[case] norm backward in place d={d}", flush=True)
    x, ds, w = _inputs(21, d, torch.bfloat16, 5)
    dy = up(np.random.default_rng(1).normal(size=(21, d)), torch.bfloat16)
    dx, dw = _bwd(x, w, dy, ds)
    a, b = dy.clone(), ds.clone()
    got, gw = _bwd(x, w, a, ds, dx=a)
    assert torch.equal(got, dx) and torch.equal(gw, dw)
    got, gw = _bwd(x, w, dy, b, dx=b)
    assert torch.equal(got, dx) and torch.equal(gw, dw)


def test_norm_gradients_against_differences():
    """central differences of the GPU's own fp32 forward, summed in 64 bits: step h,
    truncation O(h^2), and the forward's rounding over 2 h"""
    print("\n[case] norm differences", flush=True)
    x, _, w = _inputs(3, 128, torch.float32, 8)
    dy = up(np.random.default_rng(4).normal(size=(3, 128)), torch.float32)
    dx, dw = _bwd(x, w, dy, None)

    def loss(a, b):
        return float((host64(_run(a, None, b, quant=False, total=False)["y"]) * host64(dy)).sum())

    h = 2.0 ** -6
    # each y is off by at most (d/2 + 8) u |y|, random in sign and summed over 384
    # products; the third derivative of the loss is of order 10
    tol = 2 * (128 / 2 + 8) * U32 * float((host64(_run(x, None, w, quant=False, total=False)["y"])
                                           * host64(dy)).__abs__().sum()) / (2 * h) + 10 * h * h
    for i, j in ((0, 0), (1, 77), (2, 127)):
        p, m = x.clone(), x.clone()
        p[i, j] += h
        m[i, j] -= h
        assert abs((loss(p, w) - loss(m, w)) / float(p[i, j].double() - m[i, j].double())
                   - float(dx[i, j])) < tol
        p, m = w.clone(), w.clone()
        p[j] += h
        m[j] -= h
        assert abs((loss(x, p) - loss(x, m)) / float(p[j].double() - m[j].double())
                   - float(dw[j])) < tol


def test_no_tokens():
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, device="cuda")
    _run(x, x, w)
    dims = _dims(0, 128, torch.bfloat16)
    dw = torch.full((128,), float("nan"), device="cuda")
    M.moe_rmsnorm_bwd(dims, x, x, w, torch.empty(0, device="cuda"), None, x, dw, None)
    assert (dw == 0).all()   # a sum over no tokens


def test_other_stream_and_graph():
    print("\n[case] norm graph", flush=True)
    x, r, w = _inputs(300, 512, torch.bfloat16, 2)
    dy = up(np.random.default_rng(3).normal(size=(300, 512)), torch.bfloat16)
    dims = _dims(300, 512, torch.bfloat16)
    s, y, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rstd, dw = torch.empty(300, device="cuda"), torch.empty(512, device="cuda")
    ws = torch.empty(M.moe_rmsnorm_bwd_workspace_bytes(dims), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        M.moe_rmsnorm(dims, x, r, w, EPS, s, y, None, None, rstd, stream=stream)
        M.moe_rmsnorm_bwd(dims, dy, s, w, rstd, r, dx, dw, ws, stream=stream)

    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (s, y, dx, rstd, dw)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((s, y, dx, rstd, dw), ref))
        for t in (s, y, dx, rstd, dw, ws):
            t.zero_()
        torch.cuda.synchronize()

    check()
    step(side)
    check()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        check()
