"""GPU: the experts of a few tokens with 4-bit weights against the oracle in 64
bits.

Bounds: a and b are fp32 sums of d terms; h keeps 16 significant bits in a bf16
layer (cut: 2^-15) and 24 in an fp32 one; y is a sum of f terms per slot and of k
slots, rounded once to act.
"""
import numpy as np
import pytest
import torch

import top_routing_grouped_router_amd as M
from oracle import moe_oracle as O

from _lowp import U32, U_ACT, gamma, hidden_bound, host64, random_blocks, rnd, up, within

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, d, E, f, k, act, seed=0, scales=(118, 124)):
        rng = np.random.default_rng(seed)
        self.dims = M.make_dims(T, d, E, f, k, act)
        self.T, self.d, self.E, self.f, self.k, self.act = T, d, E, f, k, act
        self.x = rnd(rng.normal(size=(T, d)), act)
        self.idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        self.gate = rng.random((T, k)).astype(np.float32)
        self.w1 = random_blocks(rng, (E, f, d), "e2m1", scales)
        self.w3 = random_blocks(rng, (E, f, d), "e2m1", scales)
        self.w2 = random_blocks(rng, (E, d, f), "e2m1", scales)

    def upload(self):
        self.g = {n: tuple(up(a) for a in getattr(self, n)[:2]) for n in ("w1", "w3", "w2")}
        self.g["x"] = up(self.x, self.act)
        self.g["idx"], self.g["gate"] = up(self.idx), up(self.gate)
        self.y = torch.full((self.T, self.d), float("nan"), dtype=self.act, device="cuda")
        n = M.moe_token_swiglu_workspace_bytes(self.dims)
        assert n > 0
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaNs

    def run(self, stream=None):
        g = self.g
        M.moe_token_swiglu(self.dims, g["x"], g["idx"], g["gate"], *g["w1"], *g["w3"], *g["w2"],
                           self.y, self.ws, stream=stream)

    def check(self, rows=slice(None)):
        want = O.token_swiglu(self.x, self.idx, self.gate, self.w1[2], self.w3[2], self.w2[2])
        bound = np.zeros_like(want)
        cut = 2.0 ** -15 if self.act == torch.bfloat16 else 2.0 ** -23
        for t in range(self.T):
            x = self.x[t:t + 1]
            for j in range(self.k):
                e = self.idx[t, j]
                if not 0 <= e < self.E:
                    continue
                w1, w3, w2 = self.w1[2][e], self.w3[2][e], np.abs(self.w2[2][e])
                a, b, h = O.swiglu_hidden(x, w1, w3)
                eh = hidden_bound(x, w1, w3, a, b, h) + np.abs(h) * cut
                # the terms of h join one sum: up to three times as many additions
                bound[t] += abs(self.gate[t, j]) * ((eh + gamma(3 * self.f) * np.abs(h)) @ w2.T)[0]
                bound[t] += abs(self.gate[t, j]) * (np.abs(h) @ w2.T)[0] * (self.k + 2) * U32
        within(host64(self.y)[rows], want[rows],
               (bound + U_ACT[self.act] * (np.abs(want) + bound) + 1e-38)[rows], "y")


SHAPES = [   # T, d, E, f, k
    (1, 64, 1, 64, 1), (1, 2048, 64, 1024, 6), (1, 192, 8, 320, 2), (2, 128, 4, 64, 4),
    (7, 256, 8, 256, 2), (16, 576, 16, 192, 4), (33, 128, 2, 192, 2), (100, 64, 3, 128, 1),
    (64, 192, 256, 64, 16), (37, 320, 23, 64, 5), (5, 1088, 64, 128, 7),
    # either side of the two ways, K of several batches, experts of over 16 tokens
    (8, 1600, 4, 1088, 2), (9, 1600, 4, 1088, 2), (8, 64, 16, 64, 16), (60, 1024, 3, 576, 2),
    (9, 2560, 40, 64, 3),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_tokens(shape, act):
    print(f"\n[case] token {shape} {act}", flush=True)
    c = Case(*shape, act, seed=shape[0] + shape[1])
    c.upload()
    c.run()
    c.check()
    first = c.y.clone()
    c.ws.zero_()
    c.run()
    assert torch.equal(c.y, first)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [4, 64])
def test_dropped_repeated_and_odd_ids(act, E):
    """-1 and ids past the end add nothing, a repeated id counts twice, a token
    with no expert is zeros; both ways of finding an expert's pairs"""
    print(f"\n[case] token odd ids E={E} {act}", flush=True)
    c = Case(6, 128, E, 64, 3, act, seed=E)
    c.idx[0] = [-1, 2, -1]
    c.idx[1] = [1, 1, 1]
    c.idx[2] = [-1, E, 2147483647]
    c.idx[3] = [3, -2147483648, 3]
    c.upload()
    c.run()
    c.check()
    assert (c.y[2] == 0).all()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_all_tokens_at_one_expert(act):
    print(f"\n[case] token one expert {act}", flush=True)
    c = Case(50, 192, 8, 128, 1, act, seed=3)
    c.idx[:] = 5
    c.upload()
    c.run()
    c.check()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_a_bad_token_stays_alone(act):
    print(f"\n[case] token non-finite {act}", flush=True)
    c = Case(5, 128, 4, 64, 2, act, seed=8)
    c.upload()
    c.run()
    ref = c.y.clone()
    c.g["x"][1, 7] = float("nan")
    c.g["x"][3, 100] = float("inf")
    c.run()
    assert torch.isnan(c.y[1]).all() and not torch.isfinite(c.y[3]).any()
    keep = [0, 2, 4]
    assert torch.equal(c.y[keep], ref[keep])
    c.upload()
    c.g["w2"][1][int(c.idx[0, 0]), 9, 0] = 255   # one output column of one expert
    c.run()
    bad = torch.zeros(5, 128, dtype=torch.bool)
    bad[(c.idx == c.idx[0, 0]).any(1), 9] = True
    assert torch.equal(torch.isnan(c.y).cpu(), bad)


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_scales_at_the_ends(act):
    """weights near the smallest and the largest powers of two"""
    print(f"\n[case] token scales {act}", flush=True)
    c = Case(3, 128, 4, 64, 2, act, seed=1, scales=(118, 124))
    rng = np.random.default_rng(0)
    c.w2 = random_blocks(rng, (4, 128, 64), "e2m1", (0, 3))        # products vanish
    c.upload()
    c.run()
    torch.cuda.synchronize()
    assert (c.y.abs() < 1e-30).all() and torch.isfinite(c.y).all()
    c.w1 = random_blocks(rng, (4, 64, 128), "e2m1", (60, 70))
    c.w3 = random_blocks(rng, (4, 64, 128), "e2m1", (175, 185))
    c.w2 = random_blocks(rng, (4, 128, 64), "e2m1", (120, 130))
    c.upload()
    c.run()
    c.check()


def test_largest_batch_and_no_tokens():
    print("\n[case] token largest", flush=True)
    c = Case(256, 64, 8, 64, 4, torch.bfloat16, seed=2)
    assert 256 * 4 == M.MOE_TOKEN_MAX_SLOTS
    c.upload()
    c.run()
    c.check()
    z = M.make_dims(0, 64, 8, 64, 4, torch.bfloat16)
    g = c.g
    M.moe_token_swiglu(z, g["x"][:0], g["idx"][:0], g["gate"][:0], *g["w1"], *g["w3"], *g["w2"],
                       c.y[:0], None)


def test_graph_replays_and_streams():
    print("\n[case] token graph", flush=True)
    c = Case(3, 256, 16, 128, 4, torch.bfloat16, seed=2)
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
    other = (c.idx + 1) % 16
    c.g["idx"].copy_(up(other))
    graph.replay()
    c.idx = other
    c.check()
