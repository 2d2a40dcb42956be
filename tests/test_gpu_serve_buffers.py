"""GPU: the layers' own outputs as their next inputs."""
import numpy as np
import pytest
import torch

from top_routing_grouped_router_amd import MoELayer, MoEServeLayer

from _lowp import up

pytestmark = pytest.mark.gpu


def _weights(rng, d, E, f, act):
    return {"w1": up(rng.normal(size=(E, f, d)) * d ** -0.5, act),
            "w3": up(rng.normal(size=(E, f, d)) * d ** -0.5, act),
            "w2": up(rng.normal(size=(E, d, f)) * f ** -0.5, act),
            "wr": up(rng.normal(size=(E, d)) * d ** -0.5, torch.float32),
            "nw": up(1 + 0.2 * rng.normal(size=d), torch.float32)}


def _serve(T, d, E, f, k, act, seed, **kw):
    w = _weights(np.random.default_rng(seed), d, E, f, act)
    layer = MoEServeLayer(T, d, E, f, k, act, **kw)
    layer.load(w["w1"], w["w3"], w["w2"])
    return layer, w


@pytest.mark.parametrize("T,shift", [(7, 1), (6000, 1), (6000, 700)])
def test_rows_that_move_up(T, shift):
    """y and stream of all but the first sequences, as slices, give what copies give"""
    print(f"\n[case] serve rows move up {T} {shift}", flush=True)
    rng = np.random.default_rng(T)
    layer, w = _serve(T, 256, 8, 64, 2, torch.bfloat16, 1)
    x, r = (up(rng.normal(size=(T, 256)), torch.bfloat16) for _ in range(2))

    def again(copies):
        y, stream = layer.forward(x, w["nw"], w["wr"], r)
        y, stream = y[shift:], stream[shift:]
        if copies:
            y, stream = y.clone(), stream.clone()
        y, stream = layer.forward(y, w["nw"], w["wr"], stream)
        return y.clone(), stream.clone()

    want = again(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(again(False), want))


def test_rows_that_move_up_in_a_graph():
    print("\n[case] serve rows move up, graph", flush=True)
    rng = np.random.default_rng(2)
    layer, w = _serve(90, 128, 8, 64, 2, torch.bfloat16, 2, few_slots=16)
    x, r = (up(rng.normal(size=(90, 128)), torch.bfloat16) for _ in range(2))

    def two():
        y, stream = layer.forward(x, w["nw"], w["wr"], r)
        return layer.forward(y[1:], w["nw"], w["wr"], stream[1:])

    ref = [t.clone() for t in two()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = two()
    for _ in range(3):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("T", [3, 300])
def test_the_stream_outlives_the_outputs_that_it_was(T):
    print(f"\n[case] serve y as input {T}", flush=True)
    rng = np.random.default_rng(T)
    layer, w = _serve(T, 192, 8, 128, 2, torch.bfloat16, 3)
    y, _ = layer.forward(up(rng.normal(size=(T, 192)), torch.bfloat16), w["nw"], w["wr"])
    for rows in (y, y[1:], layer.xn[:T], layer.xn[1:T]):
        x = rows.clone()
        want = layer.forward(x, w["nw"], w["wr"])[0].clone()
        rows.copy_(x)
        layer_y, stream = layer.forward(rows, w["nw"], w["wr"])
        assert torch.equal(stream, x) and torch.equal(layer_y, want)


@pytest.mark.parametrize("of", ["y", "xn"])
def test_the_training_layers_outputs_as_its_input(of):
    """gradients are of the input that was there, not of what the forward wrote there"""
    print(f"\n[case] layer {of} as input", flush=True)
    T, d, E, f, k = 128, 128, 8, 64, 2
    rng = np.random.default_rng(4)
    w = _weights(rng, d, E, f, torch.float32)
    args = (w["wr"], w["w1"], w["w3"], w["w2"])
    layer = MoELayer(T, d, E, f, k, torch.float32, pre_norm=True)
    x, dy = (up(rng.normal(size=(T, d)), torch.float32) for _ in range(2))
    layer.step(x, *args, dy, norm_weight=w["nw"])
    ref = {n: getattr(layer, n).clone() for n in ("y", "dstream", "dnorm", "dwr")}
    own = getattr(layer, of)
    own.copy_(x)
    layer.step(own, *args, dy, norm_weight=w["nw"])
    assert torch.equal(layer.stream, x)
    for n, t in ref.items():
        assert torch.equal(getattr(layer, n), t), n


@pytest.mark.parametrize("T", [3, 300])
def test_a_layer_without_weights_gives_nan(T):
    print(f"\n[case] serve before load {T}", flush=True)
    for _ in range(2):   # memory that held other weights
        layer, w = _serve(T, 128, 8, 64, 2, torch.bfloat16, 3)
        del layer
        layer = MoEServeLayer(T, 128, 8, 64, 2, torch.bfloat16)
        y, _ = layer.forward(up(np.ones((T, 128)), torch.bfloat16), w["nw"], w["wr"])
        assert torch.isnan(y).all()


def test_weights_loaded_on_another_stream_stay():
    print("\n[case] serve load on a stream", flush=True)
    layer, w = _serve(5, 512, 64, 512, 2, torch.bfloat16, 6)
    x = up(np.random.default_rng(0).normal(size=(5, 512)), torch.bfloat16)
    ref = layer.forward(x, w["nw"], w["wr"])[0].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 28, device="cuda")
    for _ in range(3):
        for _ in range(8):
            busy.add_(1)   # the current stream is behind
        other = MoEServeLayer(5, 512, 64, 512, 2, torch.bfloat16)
        with torch.cuda.stream(side):
            other.load(w["w1"], w["w3"], w["w2"])
            y = other.forward(x, w["nw"], w["wr"])[0].clone()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,E,f,k,few", [(64, 256, 64, 8, 128), (128, 8, 64, 2, 1024), (64, 3, 64, 1, 0)])
def test_forwards_stay_in_the_workspace(act, d, E, f, k, few):
    print(f"\n[case] serve workspace {d} {E} {k} {act}", flush=True)
    layer, w = _serve(3000, d, E, f, k, act, 8, few_slots=few)
    n = layer.workspace.numel()
    whole = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    layer.workspace = whole[:n]
    for T in (1, 15, 63, 64, 65, 1000, 3000):
        x = up(np.random.default_rng(T).normal(size=(T, d)), act)
        y, _ = layer.forward(x, w["nw"], w["wr"])
        assert torch.isfinite(y).all() and (whole[n:] == 0xA5).all()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [5, 20, 300])
def test_a_bad_token_stays_alone(act, T):
    """a NaN or an infinity in one sequence: the others get the bits they get without it"""
    print(f"\n[case] serve bad token {T} {act}", flush=True)
    layer, w = _serve(T, 128, 8, 64, 2, act, 5)
    x, r = (up(np.random.default_rng(i).normal(size=(T, 128)), act) for i in (1, 2))
    want, stream = (t.clone() for t in layer.forward(x, w["nw"], w["wr"], r))
    x[1, 70], r[3, 5] = float("nan"), float("inf")
    y, _ = layer.forward(x, w["nw"], w["wr"], r)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[3]).any()
    keep = [t for t in range(T) if t not in (1, 3)]
    assert torch.equal(y[keep], want[keep])
