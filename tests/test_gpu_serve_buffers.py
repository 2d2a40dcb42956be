"""GPU: the layers' own outputs as their next inputs."""
import numpy as np
import pytest
import torch

from top_routing_grouped_router_amd import MoEServeLayer

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
