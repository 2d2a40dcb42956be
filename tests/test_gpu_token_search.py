"""GPU: more than 8 tokens through their experts, where the pairs of an expert are found
in the router's table: by the expert's number where there are more pairs than experts,
else by the first pair that names it.  Bounds as for any few tokens."""
import numpy as np
import pytest
import torch

from _lowp import random_blocks, up
from test_gpu_token import Case

pytestmark = pytest.mark.gpu
ACTS = [torch.bfloat16, torch.float32]
EXPERTS = [4, 64]   # 36 pairs: by expert, by pair


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("E", EXPERTS)
@pytest.mark.parametrize("T", [9, 12])
def test_dropped_repeated_and_odd_ids(act, E, T):
    print(f"\n[case] token search odd ids {T} E={E} {act}", flush=True)
    c = Case(T, 128, E, 64, 3, act, seed=E + T)
    c.idx[0] = [-1, 2, -1]
    c.idx[1] = [1, 1, 1]
    c.idx[2] = [-1, E, 2147483647]
    c.idx[3] = [3, -2147483648, 3]
    c.idx[5] = [2, 2, 1]
    c.idx[8] = [-1, -1, -1]
    c.upload()
    c.run()
    c.check()
    assert (c.y[[2, 8]] == 0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("E", EXPERTS)
def test_no_token_has_an_expert(act, E):
    print(f"\n[case] token search none E={E} {act}", flush=True)
    c = Case(12, 128, E, 64, 3, act, seed=1)
    c.idx[:] = -1
    c.upload()
    c.run()
    assert (c.y == 0).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("E", EXPERTS)
def test_a_bad_token_stays_alone(act, E):
    """among tokens of its own experts, which share its matrix instructions"""
    print(f"\n[case] token search non-finite E={E} {act}", flush=True)
    c = Case(14, 128, E, 64, 3, act, seed=8)
    c.idx[1] = c.idx[4] = c.idx[9] = c.idx[3] = [2, 0, 1]
    c.upload()
    c.run()
    c.check()
    ref = c.y.clone()
    c.g["x"][1, 7] = float("nan")
    c.g["x"][3, 100] = float("inf")
    c.run()
    assert torch.isnan(c.y[1]).all() and not torch.isfinite(c.y[3]).any()
    keep = [t for t in range(14) if t not in (1, 3)]
    assert torch.equal(c.y[keep], ref[keep])
    c.upload()
    c.g["w2"][1][2, 9, 0] = 255   # one output column of one expert
    c.run()
    bad = torch.zeros(14, 128, dtype=torch.bool)
    bad[(c.idx == 2).any(1), 9] = True
    assert torch.equal(torch.isnan(c.y).cpu(), bad)


@pytest.mark.parametrize("act", ACTS)
def test_scales_at_the_ends(act):
    print(f"\n[case] token search scales {act}", flush=True)
    c = Case(11, 128, 4, 64, 2, act, seed=1, scales=(118, 124))
    rng = np.random.default_rng(0)
    c.w2 = random_blocks(rng, (4, 128, 64), "e2m1", (0, 3))        # products vanish
    c.upload()
    c.run()
    assert (c.y.abs() < 1e-30).all() and torch.isfinite(c.y).all()
    c.w1 = random_blocks(rng, (4, 64, 128), "e2m1", (60, 70))
    c.w3 = random_blocks(rng, (4, 64, 128), "e2m1", (175, 185))
    c.w2 = random_blocks(rng, (4, 128, 64), "e2m1", (120, 130))
    c.upload()
    c.run()
    c.check()


@pytest.mark.parametrize("T,E,k", [(16, 23, 5), (13, 200, 2), (10, 48, 3), (20, 64, 3)])
def test_pairs_named_once_or_often(T, E, k):
    """some experts of several tokens, some of one, most of none"""
    print(f"\n[case] token search {T} {E} {k}", flush=True)
    c = Case(T, 192, E, 128, k, torch.bfloat16, seed=T)
    rng = np.random.default_rng(E)
    c.idx[:] = rng.integers(0, E, size=(T, k)) % max(E // 8, k)
    c.upload()
    c.run()
    c.check()


@pytest.mark.parametrize("E", EXPERTS)
def test_graph_replays_and_streams(E):
    print(f"\n[case] token search graph E={E}", flush=True)
    c = Case(12, 256, E, 128, 3, torch.bfloat16, seed=2)
    c.upload()
    c.run()
    torch.cuda.synchronize()
    ref = c.y.clone()
    side = torch.cuda.Stream()
    c.run(side)
    torch.cuda.synchronize()
    assert torch.equal(c.y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for turn in range(3):
        c.y.zero_()
        c.ws.fill_(turn)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.y, ref)
    # the captured call reads the table anew: other experts, other results
    other = (c.idx + 1) % E
    c.g["idx"].copy_(up(other))
    graph.replay()
    c.idx = other
    c.check()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d,E,f,k", [
    (8, 128, 2, 1152, 2), (8, 128, 2, 1216, 2),     # on either side of the search
    (2, 1024, 16, 512, 16), (3, 1024, 16, 512, 16), (4, 576, 4, 1024, 4), (6, 576, 4, 1024, 4),
    (5, 64, 1, 4096, 1), (1, 128, 1, 16448, 1),
])
def test_up_to_8_tokens_of_few_experts(act, T, d, E, f, k):
    print(f"\n[case] token few experts {T} {d} {E} {f} {k} {act}", flush=True)
    c = Case(T, d, E, f, k, act, seed=T + f)
    c.upload()
    c.run()
    c.check()
