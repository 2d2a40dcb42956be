"""GPU: the norm, the router and the low-precision experts together, as a model
runs them: MoEServeLayer over batches of changing size, and the training layer
with its pre-norm, forward and backward."""
import numpy as np
import pytest
import torch

import top_routing_grouped_router_amd as M
from oracle import moe_oracle as O
from top_routing_grouped_router_amd import MoELayer, MoEServeLayer

from _lowp import (U32, U_ACT, gamma, hidden_bound, host64, mx_dot_bound, plain_dot_bound, up,
                   within)
from _util import TOL, rel_err

pytestmark = pytest.mark.gpu


def _weights(rng, d, E, f, act):
    return {"w1": up(rng.normal(size=(E, f, d)) * d ** -0.5, act),
            "w3": up(rng.normal(size=(E, f, d)) * d ** -0.5, act),
            "w2": up(rng.normal(size=(E, d, f)) * f ** -0.5, act),
            "wr": up(rng.normal(size=(E, d)) * d ** -0.5, torch.float32),
            "nw": up(1 + 0.2 * rng.normal(size=d), torch.float32)}


def _values(q, scale):
    return O.mx_values(O.mx_element_values(q.cpu().numpy(), "e2m1"), scale.cpu().numpy())


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,E,f,k", [(192, 8, 128, 3), (256, 16, 256, 4)])
def test_serving_batches_of_any_size(act, d, E, f, k):
    print(f"\n[case] serve {act} d={d} E={E}", flush=True)
    rng = np.random.default_rng(d)
    w = _weights(rng, d, E, f, act)
    layer = MoEServeLayer(96, d, E, f, k, act, few_slots=64)
    layer.load(w["w1"], w["w3"], w["w2"])
    ref, s = O.mx_quantize(host64(w["w1"]), "e2m1")
    w1, w3, w2 = (_values(getattr(layer, n), getattr(layer, n + "_scale")) for n in ("w1", "w3", "w2"))
    assert np.array_equal(w1, O.mx_values(ref, s))
    for T in (1, 96, 16, 33, 2, 0, 64):
        x, res = up(rng.normal(size=(T, d)), act), up(rng.normal(size=(T, d)), act)
        y, stream = layer.forward(x, w["nw"], w["wr"], residual=res if T % 2 else None)
        torch.cuda.synchronize()
        assert y.shape == (T, d)
        assert torch.equal(stream, (x.float() + res.float()).to(act) if T % 2 else x)
        if T == 0:
            continue
        xn, rstd = O.rmsnorm(host64(stream), host64(w["nw"]), 1e-6)
        within(host64(layer.xn[:T]), xn, np.abs(xn) * (U_ACT[act] + (d / 2 + 8) * U32), "xn")
        idx, gate = layer.topk_idx[:T].cpu().numpy(), host64(layer.topk_gate[:T])
        r = O.route(host64(layer.xn[:T]), w["wr"].cpu().numpy(), k)
        clear = r["margin"] >= 1e-3
        assert np.array_equal(np.sort(idx, 1)[clear], np.sort(r["topk_idx"], 1)[clear])
        few = T * k <= 64
        rows = host64(layer.xn[:T]) if few else O.mx_values(
            O.mx_element_values(layer.xq[:T].cpu().numpy(), "e4m3"), layer.x_scale[:T].cpu().numpy())
        want, bound = np.zeros((T, d)), np.zeros((T, d))
        dot = plain_dot_bound if few else mx_dot_bound
        for t in range(T):
            for j in range(k):
                e, g = idx[t, j], gate[t, j]
                a, b, h = O.swiglu_hidden(rows[t:t + 1], w1[e], w3[e])
                eh = hidden_bound(rows[t:t + 1], w1[e], w3[e], a, b, h, dot)
                if few:
                    eh += np.abs(h) * 2.0 ** -15
                else:   # e4m3: half a step, of the element or of the smallest one
                    top = np.repeat((np.abs(h) + eh).reshape(1, -1, 32).max(-1), 32, -1)
                    eh = eh + np.maximum(2.0 ** -4 * (np.abs(h) + eh), 2.0 ** -10 * top / 224)
                want[t] += g * (h @ w2[e].T)[0]
                bound[t] += g * (eh @ np.abs(w2[e]).T)[0]
                tail = gamma(3 * f) * (np.abs(h) @ np.abs(w2[e]).T) if few else mx_dot_bound(h, w2[e])
                u = 0 if few else U_ACT[act]   # y_perm is stored
                bound[t] += g * (tail + (u + 4 * U32) * (np.abs(h) @ np.abs(w2[e]).T))[0]
        within(host64(y), want, 1.01 * bound + U_ACT[act] * np.abs(want), f"y T={T}")
        # in norm: roundings at random are below their largest.  Few tokens: y's
        # rounding, and the sums of d and of 3 f fp32 terms (each within gamma of its
        # magnitudes, which an fp32 y's own half step does not cover); more: h's
        err = np.linalg.norm(host64(y) - want) / np.linalg.norm(want)
        assert err < (U_ACT[act] + gamma(d) + gamma(3 * f) if few else 2.0 ** -4), err


def test_both_paths_serve_the_same_tokens():
    """8-bit rows against act rows on the same batch: as far apart as two roundings
    to e4m3, of x and of h, each at most 2^-4 of every value"""
    print("\n[case] serve both paths", flush=True)
    rng = np.random.default_rng(1)
    w = _weights(rng, 256, 8, 128, torch.bfloat16)
    x = up(rng.normal(size=(40, 256)), torch.bfloat16)
    out = []
    for few in (0, 256):
        layer = MoEServeLayer(40, 256, 8, 128, 2, torch.bfloat16, few_slots=few)
        layer.load(w["w1"], w["w3"], w["w2"])
        out.append(host64(layer.forward(x, w["nw"], w["wr"])[0]))
    gap = np.linalg.norm(out[0] - out[1]) / np.linalg.norm(out[1])
    # x enters h twice, h once more: at most 2^-4 each in norm, and silu's slope
    assert 0 < gap < 3.2 * 2.0 ** -4, gap


def test_serving_in_a_graph():
    print("\n[case] serve graph", flush=True)
    rng = np.random.default_rng(5)
    w = _weights(rng, 128, 8, 64, torch.bfloat16)
    layer = MoEServeLayer(64, 128, 8, 64, 2, torch.bfloat16, few_slots=16)
    layer.load(w["w1"], w["w3"], w["w2"])
    for T in (4, 64):
        x, res = up(rng.normal(size=(T, 128)), torch.bfloat16), up(rng.normal(size=(T, 128)), torch.bfloat16)
        y, stream = layer.forward(x, w["nw"], w["wr"], res)
        torch.cuda.synchronize()
        ref = y.clone(), stream.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward(x, w["nw"], w["wr"], res)
        for _ in range(3):
            y.zero_()
            stream.zero_()
            layer.workspace.fill_(0xFF)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, ref[0]) and torch.equal(stream, ref[1])


@pytest.mark.parametrize("act,res,kw", [
    (torch.float32, True, {}), (torch.float32, False, dict(gather=True)),
    (torch.bfloat16, True, dict(gather=True, fold_gate=True)),
    (torch.bfloat16, True, dict(gather=True, aux_coef=0.01, z_coef=0.001, capacity_factor=1.25))])
def test_training_layer_with_its_norm(act, res, kw):
    print(f"\n[case] layer pre_norm {act} res={res} {kw}", flush=True)
    T, d, E, f, k = 1024, 256, 16, 256, 4
    rng = np.random.default_rng(3)
    w = _weights(rng, d, E, f, act)
    x, dy, ds = (up(rng.normal(size=(T, d)), act) for _ in range(3))
    r = up(rng.normal(size=(T, d)), act) if res else None
    args = (w["wr"], w["w1"], w["w3"], w["w2"])
    layer = MoELayer(T, d, E, f, k, act, pre_norm=True, **kw)
    layer.step(x, *args, dy, norm_weight=w["nw"], residual=r, dsum=ds)
    torch.cuda.synchronize()
    stream = x if r is None else (x.float() + r.float()).to(act)
    assert torch.equal(layer.stream, stream)
    # the layer behind the norm is the layer without one, on the norm's output
    plain = MoELayer(T, d, E, f, k, act, **kw)
    plain.step(layer.xn, *args, dy)
    torch.cuda.synchronize()
    for n in ("y", "dx", "dw1", "dw3", "dw2", "dwr", "topk_idx"):
        assert torch.equal(getattr(plain, n), getattr(layer, n)), n
    dx, dw = O.rmsnorm_bwd(host64(layer.dx), host64(stream), host64(w["nw"]), 1e-6, host64(ds))
    assert rel_err(host64(layer.dstream), dx) <= (TOL["f32"] if act == torch.float32 else U_ACT[act] * 1.1)
    assert rel_err(host64(layer.dnorm), dw) <= TOL["f32"]
    if act == torch.float32:   # the whole block against the oracle
        xn, _ = O.rmsnorm(host64(stream), host64(w["nw"]), 1e-6)
        routing = (layer.topk_idx.cpu().numpy(), layer.topk_gate.cpu().numpy())
        ws = [host64(w[n]) for n in ("w1", "w3", "w2")]
        wr = w["wr"].cpu().numpy()
        fwd = O.layer_forward(xn, wr, *ws, k, routing=routing)
        bwd = O.layer_backward(xn, wr, *ws, fwd, host64(dy))
        assert rel_err(host64(layer.y), fwd["y"]) <= TOL["f32"]
        dx, dw = O.rmsnorm_bwd(bwd["dx"], host64(stream), host64(w["nw"]), 1e-6, host64(ds))
        assert rel_err(host64(layer.dstream), dx) <= TOL["f32"]
        assert rel_err(host64(layer.dnorm), dw) <= TOL["f32"]


def test_layer_refuses_what_does_not_fit():
    layer = MoELayer(64, 64, 4, 64, 2, torch.float32)
    x = torch.zeros(64, 64, device="cuda")
    with pytest.raises(ValueError, match="pre_norm"):
        layer.forward(x, x, x, x, x, norm_weight=x[0])
    with pytest.raises(ValueError, match="pre_norm"):
        layer.norm(x, x[0])
    layer = MoELayer(64, 64, 4, 64, 2, torch.float32, pre_norm=True)
    with pytest.raises(ValueError, match="pre_norm"):
        layer.forward(x, x, x, x, x)
    with pytest.raises(ValueError, match="before forward"):
        layer.backward(x, x, x, x, x, x, norm_weight=x[0])
    serve = MoEServeLayer(8, 64, 4, 64, 2, torch.float32)
    with pytest.raises(ValueError, match="T <= 8"):
        serve.forward(x, x[0], x[:4])
    with pytest.raises(ValueError, match="w1"):
        serve.load(x, x, x)
    dims = M.make_dims(8, 64, 4, 64, 2, torch.float32)
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_rmsnorm(dims, torch.zeros(64, 8, device="cuda").t(),
                      None, x[0], 1e-6, None, torch.empty(8, 64, device="cuda"), None, None, None)
    with pytest.raises(ValueError, match="hold"):
        M.moe_rmsnorm(dims, x, None, x[0], 1e-6, None, x, None, None, None)
    with pytest.raises(ValueError, match="must be torch.float32"):
        M.moe_rmsnorm(dims, x[:8].bfloat16(), None, x[0], 1e-6, None, x[:8], None, None, None)
    with pytest.raises(ValueError, match="must be on"):
        M.moe_rmsnorm(dims, x[:8], None, x[0].cpu(), 1e-6, None, x[:8], None, None, None)


def test_calls_refuse_other_devices_and_router_shapes():
    serve = MoEServeLayer(8, 64, 4, 64, 2, torch.float32)
    x = torch.zeros(8, 64, device="cuda")
    with pytest.raises(ValueError, match="wr must be"):
        serve.forward(x, x[0], x[:3])

    class Elsewhere:   # a stream of another GPU
        device_index, cuda_stream = torch.cuda.current_device() + 1, 0

    with pytest.raises(ValueError, match="stream must be on"):
        M.moe_rmsnorm(M.make_dims(8, 64, 4, 64, 2, torch.float32), x, None, x[0], 1e-6, None, x,
                      None, None, None, stream=Elsewhere())


@pytest.mark.parametrize("T", [3, 40])
def test_a_layers_outputs_are_its_next_inputs(T):
    """block after block through one layer's buffers: y and the stream are read before
    they are overwritten"""
    print(f"\n[case] serve chain {T}", flush=True)
    rng = np.random.default_rng(7)
    w = _weights(rng, 192, 8, 128, torch.bfloat16)
    layer = MoEServeLayer(40, 192, 8, 128, 2, torch.bfloat16, few_slots=16)
    layer.load(w["w1"], w["w3"], w["w2"])
    y, stream = layer.forward(up(rng.normal(size=(T, 192)), torch.bfloat16), w["nw"], w["wr"],
                              up(rng.normal(size=(T, 192)), torch.bfloat16))
    x, res = y.clone(), stream.clone()
    y2, stream2 = layer.forward(y, w["nw"], w["wr"], stream)
    got = y2.clone(), stream2.clone()
    y3, stream3 = layer.forward(x, w["nw"], w["wr"], res)
    assert torch.equal(y3, got[0]) and torch.equal(stream3, got[1])
    assert torch.equal(stream3, (x.float() + res.float()).to(torch.bfloat16))


def test_two_layers_on_two_streams():
    print("\n[case] serve two streams", flush=True)
    rng = np.random.default_rng(9)
    jobs = []
    for T, d, E, f, k in ((300, 256, 16, 192, 4), (5, 512, 8, 256, 2)):
        w = _weights(rng, d, E, f, torch.bfloat16)
        layer = MoEServeLayer(T, d, E, f, k, torch.bfloat16)
        layer.load(w["w1"], w["w3"], w["w2"])
        x = up(rng.normal(size=(T, d)), torch.bfloat16)
        y = layer.forward(x, w["nw"], w["wr"])[0].clone()
        jobs.append((layer, x, w, y, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, *_ in jobs:
            layer.y.zero_()
        torch.cuda.synchronize()
        for layer, x, w, _, stream in jobs:
            with torch.cuda.stream(stream):
                for _ in range(4):
                    layer.forward(x, w["nw"], w["wr"])
        torch.cuda.synchronize()
        for layer, x, _, y, _ in jobs:
            assert torch.equal(layer.y[:x.shape[0]], y)


def test_training_step_with_its_norm_in_a_graph():
    print("\n[case] layer pre_norm graph", flush=True)
    T, d, E, f, k = 1024, 256, 16, 256, 4
    rng = np.random.default_rng(11)
    w = _weights(rng, d, E, f, torch.bfloat16)
    x, r, dy, ds = (up(rng.normal(size=(T, d)), torch.bfloat16) for _ in range(4))
    layer = MoELayer(T, d, E, f, k, torch.bfloat16, pre_norm=True, gather=True, fold_gate=True)

    def step():
        layer.step(x, w["wr"], w["w1"], w["w3"], w["w2"], dy, norm_weight=w["nw"], residual=r,
                   dsum=ds)

    step()
    torch.cuda.synchronize()
    names = ("y", "stream", "dstream", "dnorm", "dx", "dw1", "dw3", "dw2", "dwr")
    ref = {n: getattr(layer, n).clone() for n in names}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for n in names:
            getattr(layer, n).zero_()
        layer.workspace.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(getattr(layer, n), ref[n]), n
