"""GPU: the experts of a prompt in low precision against the oracle in 64 bits.

UP is held to the exact h: half a step of its e4m3 element under the scale that
the kernel chose, plus the fp32 error of h; the scale itself must be the
smallest that fits, but for that error.  DOWN is held to the exact product of
the h that UP wrote: the instruction's own sum (mx_dot_bound) and one rounding
to act.
"""
import numpy as np
import pytest
import torch

import top_routing_grouped_router_amd as M
from oracle import moe_oracle as O

from _lowp import U_ACT, hidden_bound, host64, mx_dot_bound, random_blocks, up, within

pytestmark = pytest.mark.gpu

GUARD = 0xA5


class Case:
    def __init__(self, T, d, E, f, k, counts, act, seed=0, gather=True):
        rng = np.random.default_rng(seed)
        self.dims = M.make_dims(T, d, E, f, k, act)
        self.T, self.d, self.E, self.f, self.R, self.act = T, d, E, f, T * k, act
        self.offsets = np.r_[0, np.cumsum(counts)].astype(np.int32)
        assert len(counts) == E and self.offsets[-1] <= self.R
        self.rows = int(self.offsets[-1])
        self.src = rng.integers(0, T, size=self.R).astype(np.int32) if gather else None
        n = T if gather else self.R
        self.x = random_blocks(rng, (n, d), "e4m3")
        self.w1 = random_blocks(rng, (E, f, d), "e2m1")
        self.w3 = random_blocks(rng, (E, f, d), "e2m1")
        self.w2 = random_blocks(rng, (E, d, f), "e2m1")

    def upload(self):
        self.g = {n: tuple(up(a) for a in getattr(self, n)[:2]) for n in ("x", "w1", "w3", "w2")}
        self.g["src"] = None if self.src is None else up(self.src)
        self.g["off"] = up(self.offsets)
        self.hq = torch.full((self.R, self.f), GUARD, dtype=torch.uint8, device="cuda")
        self.hs = torch.full((self.R, O.mx_scale_cols(self.f)), GUARD, dtype=torch.uint8,
                             device="cuda")
        self.y = torch.full((self.R, self.d), float("nan"), dtype=self.act, device="cuda")

    def run(self, stream=None):
        g = self.g
        M.moe_expert_up_mx(self.dims, *g["x"], g["src"], g["off"], *g["w1"], *g["w3"], self.hq,
                           self.hs, stream=stream)
        M.moe_expert_down_mx(self.dims, self.hq, self.hs, g["off"], *g["w2"], self.y,
                             stream=stream)

    def check(self):
        torch.cuda.synchronize()
        n, f = self.rows, self.f
        hq, hs = self.hq.cpu().numpy(), self.hs.cpu().numpy()
        assert (hq[n:] == GUARD).all() and (hs[n:] == GUARD).all()
        y = host64(self.y)
        assert np.isnan(y[n:]).all()
        if n == 0:
            return
        hq, hs, y = hq[:n], hs[:n], y[:n]
        assert (hs[:, f // 32:] == 0).all()
        hv = O.mx_values(O.mx_element_values(hq, "e4m3"), hs)
        x = self.x[2][self.src[:n]] if self.src is not None else self.x[2][:n]
        h, eh, yw, ey = (np.zeros((n, c)) for c in (f, f, self.d, self.d))
        for e in range(self.E):
            at = slice(self.offsets[e], self.offsets[e + 1])
            if at.start == at.stop:
                continue
            a, b, h[at] = O.swiglu_hidden(x[at], self.w1[2][e], self.w3[2][e])
            eh[at] = hidden_bound(x[at], self.w1[2][e], self.w3[2][e], a, b, h[at], mx_dot_bound)
            yw[at] = hv[at] @ self.w2[2][e].T
            ey[at] = mx_dot_bound(hv[at], self.w2[2][e])
        sc = 2.0 ** (hs[:, :f // 32].astype(np.float64) - 127)
        low = (np.abs(h) - eh).reshape(n, -1, 32).max(-1)
        high = (np.abs(h) + eh).reshape(n, -1, 32).max(-1)
        assert (low <= 448 * sc).all() and ((high >= 224 * sc) | (hs[:, :f // 32] == 0)).all()
        half = np.maximum(2.0 ** -4 * (np.abs(h) + eh), np.repeat(sc, 32, -1) * 2.0 ** -10)
        within(hv, h, half + eh, "h")
        within(y, yw, ey + U_ACT[self.act] * (np.abs(yw) + ey) + 1e-38, "y_perm")


SHAPES = [   # T, d, E, f, k, rows of each expert
    (1, 64, 1, 64, 1, [1]),
    (5, 192, 4, 64, 2, [0, 9, 0, 1]),
    (8, 128, 4, 128, 2, [0, 0, 0, 0]),
    (70, 320, 5, 192, 4, [65, 64, 63, 1, 87]),
    (64, 64, 3, 448, 3, [33, 0, 95]),
    (129, 1024, 3, 320, 2, [128, 0, 130]),
    (40, 2048, 2, 1024, 2, [31, 49]),
    (96, 256, 256, 64, 2, [1, 0] * 92 + [2, 2] * 4 + [0] * 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:5])))
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_small_tiles(shape, act):
    print(f"\n[case] experts_mx {shape} {act}", flush=True)
    c = Case(*shape, act, seed=shape[0])
    c.upload()
    c.run()
    c.check()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,f", [(1088, 576), (1024, 512)])
def test_large_tiles(act, d, f):
    """16384 rows: the 256 x 256 tiles of both products, with a half K step and a
    partial column tile, and ragged experts"""
    print(f"\n[case] experts_mx large {d} {f} {act}", flush=True)
    c = Case(8192, d, 5, f, 2, [1, 8191, 0, 255, 7900], act, seed=d)
    c.upload()
    c.run()
    c.check()


@pytest.mark.parametrize("T,d,E,f,k,gather", [
    (100000, 64, 3, 64, 2, True),      # K of half a step: every step is a new tile
    (60000, 128, 4, 128, 2, False),    # one step to a tile
    (50000, 192, 5, 64, 3, True),      # two
    (50000, 384, 2, 64, 2, True),      # three: as many as the ring holds
    (2000, 64, 16, 1024, 2, True),     # the small tiles
    (2000, 320, 16, 1024, 2, False),
])
def test_workgroups_with_several_tiles(T, d, E, f, k, gather):
    """more tiles than workgroups on the GPU: the stream of steps runs across them"""
    print(f"\n[case] experts_mx streams {T} {d} {E} {f} {k} {gather}", flush=True)
    R = T * k
    counts = np.random.default_rng(T).multinomial(R - 5, np.ones(E) / E)
    c = Case(T, d, E, f, k, counts, torch.bfloat16, seed=d, gather=gather)
    c.upload()
    c.run()
    c.check()


@pytest.mark.parametrize("T,d,E,f,gather", [(8000, 576, 60, 512, True), (10000, 512, 3, 1088, False)])
def test_large_tiles_of_few_rows(T, d, E, f, gather):
    """large tiles whose second half of wavefronts has no rows, before and after
    full ones, several to a workgroup"""
    print(f"\n[case] experts_mx few rows {T} {d} {E} {f} {gather}", flush=True)
    counts = np.random.default_rng(d).integers(0, 300, size=E)
    counts[::4] = [128, 0, 129, 1, 256][:len(counts[::4])] * 3 if E == 60 else 100
    counts[E // 2] = 2 * T - 3 - (counts.sum() - counts[E // 2])
    c = Case(T, d, E, f, 2, counts, torch.bfloat16, seed=d, gather=gather)
    c.upload()
    c.run()
    c.check()


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_the_down_products_tiles_agree(act):
    """a batch with eight large tiles to a workgroup gives each expert's rows the bits
    that batches of a few tiles give them; rows behind the last expert stay"""
    print(f"\n[case] experts_mx down tiles {act}", flush=True)
    T, d, E, f, k = 16640, 4160, 6, 576, 2
    counts = [129, 16000, 0, 1, 17020, 100]
    off = np.r_[0, np.cumsum(counts)]
    n = int(off[-1])
    gen = torch.Generator(device="cuda").manual_seed(5)

    def codes(*shape, top=256):
        return torch.randint(0, top, shape, dtype=torch.uint8, device="cuda", generator=gen)

    hq = codes(T * k, f)
    hq[(hq & 127) == 127] = 3                                   # no NaN
    hs = codes(T * k, O.mx_scale_cols(f), top=9) + 120
    w2, ws = codes(E, d, f // 2), codes(E, d, O.mx_scale_cols(f), top=9) + 120
    y = torch.full((T * k, d), float("nan"), dtype=act, device="cuda")
    M.moe_expert_down_mx(M.make_dims(T, d, E, f, k, act), hq, hs,
                         torch.tensor(off, dtype=torch.int32, device="cuda"), w2, ws, y)
    assert torch.isnan(y[n:]).all() and torch.isfinite(y[:n]).all()
    for e in range(E):
        for a in range(int(off[e]), int(off[e + 1]), 4096):
            b = min(a + 4096, int(off[e + 1]))
            part = torch.empty(b - a, d, dtype=act, device="cuda")
            M.moe_expert_down_mx(M.make_dims(b - a, d, 1, f, 1, act), hq[a:b].clone(),
                                 hs[a:b].clone(),
                                 torch.tensor([0, b - a], dtype=torch.int32, device="cuda"),
                                 w2[e:e + 1], ws[e:e + 1], part)
            assert torch.equal(y[a:b], part), (e, a)


def test_rows_without_a_table():
    print("\n[case] experts_mx no table", flush=True)
    c = Case(50, 192, 3, 128, 2, [40, 0, 60], torch.bfloat16, seed=1, gather=False)
    c.upload()
    c.run()
    c.check()
    g, hq, hs = c.g, c.hq.clone(), c.hs.clone()
    # the same rows through a table
    d2 = M.make_dims(100, 192, 3, 128, 1, torch.bfloat16)
    M.moe_expert_up_mx(d2, *g["x"], torch.arange(100, dtype=torch.int32, device="cuda"), g["off"],
                       *g["w1"], *g["w3"], c.hq, c.hs)
    assert torch.equal(c.hq, hq) and torch.equal(c.hs, hs)


def test_the_two_tiles_agree():
    """an expert's rows give the same bits whatever the rest of the batch: alone
    (small tile) and among 16384 rows (large tile)"""
    print("\n[case] experts_mx tiles agree", flush=True)
    c = Case(8192, 1024, 2, 512, 2, [100, 16284], torch.bfloat16, seed=4)
    c.upload()
    c.run()
    alone = M.make_dims(50, 1024, 2, 512, 2, torch.bfloat16)
    off = torch.tensor([0, 100, 100], dtype=torch.int32, device="cuda")
    rows = c.g["src"][:100].long()
    hq, hs, y = c.hq[:100].clone().fill_(0), c.hs[:100].clone().fill_(0), c.y[:100].clone().fill_(0)
    x, xs = (t[rows].contiguous() for t in c.g["x"])
    M.moe_expert_up_mx(alone, x, xs, None, off, *c.g["w1"], *c.g["w3"], hq, hs)
    M.moe_expert_down_mx(alone, hq, hs, off, *c.g["w2"], y)
    assert torch.equal(hq, c.hq[:100]) and torch.equal(hs, c.hs[:100]) and torch.equal(y, c.y[:100])


def test_non_finite_blocks_stay_in_their_row_and_expert():
    print("\n[case] experts_mx non-finite", flush=True)
    c = Case(40, 192, 2, 128, 2, [30, 50], torch.float32, seed=9)
    c.upload()
    c.run()
    hq, hs, y = c.hq.clone(), c.hs.clone(), c.y.clone()
    bad_token = int(c.src[3])
    c.g["x"][1][bad_token, 2] = 255          # one block of one token
    c.g["w1"][1][1, 70, 0] = 255             # one block of one weight row of expert 1
    c.run()
    torch.cuda.synchronize()
    hit = torch.from_numpy(c.src == bad_token).cuda()
    second = torch.arange(80, device="cuda") >= 30
    nan = (c.hs[:, :4] == 255)
    assert nan[hit].all()
    assert torch.equal(nan[~hit & ~second], torch.zeros_like(nan[~hit & ~second]))
    assert torch.equal(nan[~hit & second], torch.tensor([0, 0, 1, 0], device="cuda").bool()
                       .expand_as(nan[~hit & second]))
    fine = ~hit & ~second
    assert torch.equal(c.hq[fine], hq[fine]) and torch.equal(c.y[fine], y[fine])
    assert torch.isnan(c.y[hit | second]).all() and not torch.isnan(c.y[fine]).any()


def test_large_values_and_silu_tails():
    """a and b far out: silu of large negative a vanishes, large products keep
    their scale"""
    print("\n[case] experts_mx tails", flush=True)
    c = Case(32, 128, 2, 128, 1, [16, 16], torch.float32, seed=5)
    rng = np.random.default_rng(6)
    c.x = random_blocks(rng, (32, 128), "e4m3", scales=(126, 132))
    c.w1 = random_blocks(rng, (2, 128, 128), "e2m1", scales=(123, 130))
    c.upload()
    c.run()
    c.check()


def test_graph_replays():
    print("\n[case] experts_mx graph", flush=True)
    c = Case(300, 256, 4, 192, 2, [100, 0, 300, 200], torch.bfloat16, seed=2)
    c.upload()
    c.run()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (c.hq, c.hs, c.y)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    c.run(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        for t in (c.hq, c.hs, c.y):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((c.hq, c.hs, c.y), ref))
