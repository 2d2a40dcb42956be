"""GPU: the low-precision experts on numbers whose products and sums are exact: within a
block the instruction keeps 13 bits below its largest product, and fp32 holds every sum
of these, so one lost, doubled or misplaced product of a long K shows.

x is 0, 1 or 2 or their negatives, the weights are any e2m1 value, scales four neighbouring powers of two:
products are multiples of 2^-1 up to 12 times the scales', and the sum of 2048 of them
takes fewer than 24 bits.
"""
import pytest
import torch

import top_routing_grouped_router_amd as M

from _lowp import U32

pytestmark = pytest.mark.gpu


class Numbers:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def integers(self, lo, hi, *shape):
        return torch.randint(lo, hi, shape, device="cuda", generator=self.gen)

    def scale(self, *shape, low):
        """bytes for 2^low and the next power of two, and their values"""
        s = torch.zeros(*shape[:-1], M.moe_mx_scale_cols(shape[-1]), dtype=torch.uint8, device="cuda")
        n = shape[-1] // 32
        s[..., :n] = self.integers(127 + low, 129 + low, *shape[:-1], n).byte()
        return s, torch.exp2(s[..., :n].float() - 127).repeat_interleave(32, -1)

    def rows(self, *shape, low=-1):
        code = torch.tensor([0x00, 0x38, 0x40, 0xB8, 0xC0], dtype=torch.uint8, device="cuda")
        value = torch.tensor([0.0, 1.0, 2.0, -1.0, -2.0], device="cuda")
        at = self.integers(0, 5, *shape)
        s, power = self.scale(*shape, low=low)
        return code[at], s, value[at] * power

    def weights(self, *shape, low=-1):
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
        at = self.integers(0, 16, *shape)
        s, power = self.scale(*shape, low=low)
        v = torch.where(at >= 8, -value[at & 7], value[at & 7]) * power
        return (at[..., 0::2] | (at[..., 1::2] << 4)).byte(), s, v


SHAPES = [   # rows of each expert, columns (of the down product, of the up product), K
    ([70, 0, 129], 320, 192, 2048),           # small tiles
    ([1, 300], 64, 128, 1088),
    ([3000, 0, 1, 257, 4934], 1088, 512, 2048),   # large ones
    ([20000, 13281], 4160, 576, 576),         # and the widest
]


@pytest.mark.parametrize("counts,N,_,K", SHAPES)
@pytest.mark.parametrize("act", [torch.float32, torch.bfloat16])
def test_down_is_exact(counts, N, _, K, act):
    print(f"\n[case] exact down {counts} {N} {K} {act}", flush=True)
    R, E = sum(counts), len(counts)
    g = Numbers(K)
    hq, hs, h = g.rows(R, K)
    w2, ws, w = g.weights(E, N, K)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    y = torch.full((R, N), float("nan"), dtype=act, device="cuda")
    M.moe_expert_down_mx(M.make_dims(R, N, E, K, 1, act), hq, hs, off, w2, ws, y)
    at = 0
    for e, n in enumerate(counts):
        want = (h[at:at + n] @ w[e].t()).to(act)
        assert torch.equal(y[at:at + n], want), (e, (y[at:at + n] != want).sum())
        at += n


def _e4m3(v):
    """nearest element values of fp64 v, |v| <= 448"""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp_min(-6).double() - 3)
    return torch.round(v / step) * step


@pytest.mark.parametrize("counts,_,f,K", SHAPES[:3])
@pytest.mark.parametrize("gather", [True, False])
def test_up_rounds_the_exact_products(counts, _, f, K, gather):
    """a and b are exact, h = silu(a) b good to a few steps of fp32: each element is the
    rounding of one of the two ends of that range"""
    print(f"\n[case] exact up {counts} {f} {K} {gather}", flush=True)
    R, E = sum(counts), len(counts)
    g = Numbers(f)
    xq, xs, x = g.rows(R, K, low=-4)
    w1, s1, a = g.weights(E, f, K, low=-2)
    w3, s3, b = g.weights(E, f, K, low=-2)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    src = g.integers(0, R, R).int() if gather else None
    hq = torch.empty(R, f, dtype=torch.uint8, device="cuda")
    hs = torch.empty(R, M.moe_mx_scale_cols(f), dtype=torch.uint8, device="cuda")
    M.moe_expert_up_mx(M.make_dims(R, K, E, f, 1, torch.bfloat16), xq, xs, src, off, w1, s1, w3, s3,
                       hq, hs)
    if gather:
        x = x[src.long()]
    av, bv = torch.empty(R, f, device="cuda"), torch.empty(R, f, device="cuda")
    at = 0
    for e, n in enumerate(counts):
        av[at:at + n], bv[at:at + n] = x[at:at + n] @ a[e].t(), x[at:at + n] @ b[e].t()
        at += n
    av, bv = av.double(), bv.double()
    h = av / (1 + torch.exp(-av)) * bv
    err = h.abs() * (8 + 2 * av.abs()) * U32
    blocks = h.abs().unflatten(-1, (-1, 32))
    top, off_by = blocks.amax(-1), err.unflatten(-1, (-1, 32)).amax(-1)
    s = torch.exp2(hs[:, :f // 32].double() - 127)
    assert ((top - off_by <= 448 * s) & (top + off_by > 224 * s)).all()
    s = s.repeat_interleave(32, -1)
    got = hq.view(torch.float8_e4m3fn).double()
    low, high = (_e4m3(((h + d) / s).clamp(-448, 448)) for d in (-err, err))
    ok = (got == low) | (got == high)
    print(f"{(low != high).float().mean().item():.2e} of the elements lie at a tie", flush=True)
    assert ok.all(), ((~ok).sum(), got[~ok][:4], low[~ok][:4], high[~ok][:4])
