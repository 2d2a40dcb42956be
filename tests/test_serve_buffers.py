"""Host side of the serving layer's buffers (no GPU): the kernels are stood in for by
a norm that takes its rows in either order, so that a row which is overwritten before
it is read shows."""
import numpy as np
import pytest
import torch

from top_routing_grouped_router_amd import MoEServeLayer
from top_routing_grouped_router_amd import _lib as L

T, D, E, F, K = 12, 64, 4, 64, 2


@pytest.fixture
def calls(monkeypatch):
    def norm(dims, x, res, weight, eps, total, y, *rest):
        given = [None if t is None else t.clone() for t in (x, res)]
        want = given[0] if res is None else given[0] + given[1]
        for order in (range(dims.T), reversed(range(dims.T))):
            for t, was in zip((x, res), given):
                if t is not None:
                    t.copy_(was)
            for t in order:
                s = x[t].clone() if res is None else x[t] + res[t]
                assert torch.equal(s, want[t]), f"row {t} was overwritten before it was read"
                if total is not None:
                    total[t] = s
                y[t] = s * weight

    def token(dims, x, *rest):
        rest[8].copy_(x * 3)

    monkeypatch.setattr(L, "moe_rmsnorm", norm)
    monkeypatch.setattr(L, "moe_token_swiglu", token)
    monkeypatch.setattr(L, "moe_route", lambda *a: None)


def _layer():
    layer = MoEServeLayer(T, D, E, F, K, torch.float32, device="cpu")
    for t in (layer.norm_sum, layer.xn, layer.y):
        t.zero_()
    return layer


def _normal(*shape):
    return torch.from_numpy(np.random.default_rng(shape[0]).normal(size=shape)).float()


@pytest.mark.parametrize("shift", [1, 5])
@pytest.mark.parametrize("which", ["residual", "x", "both"])
@pytest.mark.parametrize("of", ["norm_sum", "xn"])
def test_rows_of_the_last_forward_at_other_places(calls, shift, which, of):
    """a sequence has ended: the rows behind it move up, as slices of what the layer
    gave out"""
    layer = _layer()
    weight, wr = torch.full((D,), 2.0), _normal(E, D)
    layer.forward(_normal(T, D), weight, wr, _normal(T, D))
    n = T - shift
    old = getattr(layer, of)[shift:]
    x = old if which != "residual" else _normal(n, D)
    res = old if which != "x" else _normal(n, D)
    want = x + res
    y, stream = layer.forward(x, weight, wr, res)
    assert torch.equal(stream, want) and torch.equal(y, want * 6)


def test_the_same_rows_are_not_copied(calls):
    layer = _layer()
    weight, wr = torch.full((D,), 2.0), _normal(E, D)
    _, stream = layer.forward(_normal(T, D), weight, wr, _normal(T, D))
    seen = []
    inner = L.moe_rmsnorm
    L.moe_rmsnorm = lambda *a: (seen.append((a[1].data_ptr(), a[2].data_ptr())), inner(*a))
    x, res = layer.y[:5], stream[:5]
    want = x + res
    _, got = layer.forward(x, weight, wr, res)
    assert torch.equal(got, want) and seen == [(x.data_ptr(), layer.norm_sum.data_ptr())]


@pytest.mark.parametrize("of", ["y", "xn"])
@pytest.mark.parametrize("shift", [0, 3])
def test_the_stream_outlives_the_outputs_that_it_was(calls, of, shift):
    """rows of an output as the next input, without a residual: they are the stream
    then, and not what the forward writes there"""
    layer = _layer()
    weight, wr = torch.full((D,), 2.0), _normal(E, D)
    layer.forward(_normal(T, D), weight, wr, _normal(T, D))
    x = getattr(layer, of)[shift:]
    want = x.clone()
    y, stream = layer.forward(x, weight, wr)
    assert torch.equal(stream, want) and torch.equal(y, want * 6)


def test_other_inputs_are_the_stream_themselves(calls):
    layer = _layer()
    x = _normal(3, D)
    _, stream = layer.forward(x, torch.ones(D), _normal(E, D))
    assert stream.data_ptr() == x.data_ptr()


def test_weights_are_nan_until_they_are_loaded():
    """a scale byte of 255 makes its block NaN, whatever the elements"""
    layer = _layer()
    for name in ("w1", "w3", "w2"):
        assert (getattr(layer, name + "_scale") == 255).all()


@pytest.mark.parametrize("bad", ["w1", "w3", "w2"])
def test_load_takes_all_weights_or_none(monkeypatch, bad):
    done = []
    monkeypatch.setattr(L, "moe_mx_quantize", lambda *a: done.append(a))
    layer = _layer()
    w = {"w1": torch.zeros(E, F, D), "w3": torch.zeros(E, F, D), "w2": torch.zeros(E, D, F)}
    w[bad] = w[bad][:, :, 1:]
    with pytest.raises(ValueError, match=bad):
        layer.load(**w)
    assert not done


def test_workspace_is_the_forwards_alone():
    """not the training backward's: some percent of the 4-bit weights (214 MB here)"""
    T, d, E, f, k = 16384, 2048, 64, 1024, 6
    layer = MoEServeLayer(T, d, E, f, k, torch.bfloat16, device="meta")
    dims = [L.make_dims(t, d, E, f, k, torch.bfloat16) for t in (1, 21, 63, 64, 4096, T)]
    need = [L.moe_serve_workspace_bytes(dm) for dm in dims]
    assert need == sorted(need) and 0 < need[0]
    # routing sums and counts of 256 tiles, rows of E, and the permutation's of 64 blocks
    assert need[-1] <= 2 * 256 * (E + 64) * 4
    few = L.moe_token_swiglu_workspace_bytes(dims[1])
    assert max(need[-1], few) <= layer.workspace.numel() < 4 << 20
    assert need[-1] <= L.workspace_bytes(dims[-1])
    assert L.moe_serve_workspace_bytes(L.make_dims(4, 96, 4, 64, 2, torch.bfloat16)) == 0
    assert L.moe_serve_workspace_bytes(L.make_dims(0, 64, 4, 64, 2, torch.bfloat16)) > 0


def test_a_router_on_another_device_is_refused(calls, monkeypatch):
    """before anything runs: the router's call would read it there"""
    monkeypatch.setattr(L, "moe_rmsnorm", lambda *a: pytest.fail("the norm ran"))
    layer = _layer()
    with pytest.raises(ValueError, match="wr must be on"):
        layer.forward(_normal(3, D), torch.ones(D), torch.empty(E, D, device="meta"))


@pytest.mark.parametrize("E,k,T,few", [
    (8, 2, 16, True), (8, 2, 32, True), (8, 2, 33, False), (8, 2, 48, False), (8, 2, 64, False),
    (4, 4, 16, True), (4, 4, 17, False), (4, 1, 32, True), (4, 1, 33, False),
    (16, 16, 8, True), (16, 16, 9, False), (64, 6, 21, True), (64, 6, 22, False),
    (256, 8, 16, True), (256, 8, 17, False)])
def test_few_tokens_by_pairs_and_experts(calls, monkeypatch, E, k, T, few):
    """which products a forward takes: by the pairs, and by the pairs of an expert"""
    made = []
    for name in ("moe_permute", "moe_expert_up_mx", "moe_expert_down_mx", "moe_combine"):
        monkeypatch.setattr(L, name, lambda *a, name=name: made.append(name))
    x, wr = _normal(T, D), _normal(E, D)
    for given, want in ((None, few), (T * k, True), (T * k - 1, False), (0, False)):
        kw = {} if given is None else {"few_slots": given}
        layer = MoEServeLayer(T, D, E, F, k, torch.float32, device="cpu", **kw)
        made.clear()
        layer.forward(x, torch.ones(D), wr)
        assert (not made) == want, (given, made)
