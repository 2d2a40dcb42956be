"""GPU: tensors of more than 2^31 values: the last rows get the bits that they get
alone, in the norm, the quantiser and the low-precision experts."""
import pytest
import torch

import top_routing_grouped_router_amd as M
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu

ROWS, D, TAIL = (1 << 20) + 4100, 2048, 133      # 2^31 + 8.4M values


def _bytes(*shape, top=256):
    return torch.randint(0, top, shape, dtype=torch.uint8, device="cuda")


@pytest.fixture(scope="module")
def x():
    torch.manual_seed(3)
    return torch.randn(ROWS, D, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("backward", [False, True])
def test_norm(x, backward):
    print(f"\n[case] large norm backward={backward}", flush=True)
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    last = slice(ROWS - TAIL, ROWS)
    big, small = (M.make_dims(n, D, 1, 64, 1, torch.bfloat16) for n in (ROWS, TAIL))
    rstd, rstd_t = (torch.empty(n, device="cuda") for n in (ROWS, TAIL))
    y, tail = torch.empty_like(x), x[last].clone()
    y_t = torch.empty_like(tail)
    if not backward:
        q, q_t = (torch.empty(n, D, dtype=torch.uint8, device="cuda") for n in (ROWS, TAIL))
        s, s_t = (torch.empty(n, O.mx_scale_cols(D), dtype=torch.uint8, device="cuda")
                  for n in (ROWS, TAIL))
        M.moe_rmsnorm(big, x, None, w, 1e-6, None, y, q, s, rstd)
        M.moe_rmsnorm(small, tail, None, w, 1e-6, None, y_t, q_t, s_t, rstd_t)
        assert torch.equal(q[last], q_t) and torch.equal(s[last], s_t)
        assert torch.equal(rstd[last], rstd_t) and torch.equal(y[last], y_t)
        return
    M.moe_rmsnorm(big, x, None, w, 1e-6, None, y, None, None, rstd)
    dy = x.flip(0)
    dw = torch.empty(D, device="cuda")
    ws = torch.empty(M.moe_rmsnorm_bwd_workspace_bytes(big), dtype=torch.uint8, device="cuda")
    M.moe_rmsnorm_bwd(big, dy, x, w, rstd, None, y, dw, ws)
    # dx of a row by the formula, in 64 bits.  The kernel's mean of g n adds 32 products a
    # lane, then 6 levels of lanes, in fp32: at most 42 roundings of a sum, each of the
    # products 3; 6 more make dx, and one rounds it to bf16
    r = rstd[last].double()[:, None]
    n, g = tail.double() * r, dy[last].double() * w.double()
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    err = 2.0 ** -24 * r * (52 * n.abs() * (g * n).abs().mean(1, keepdim=True) + 8 * g.abs())
    assert ((y[last].double() - dx).abs() <= 2.0 ** -8 * (dx.abs() + err) + err).all()


def test_quantiser(x):
    print("\n[case] large quantiser", flush=True)
    last = slice(ROWS - TAIL, ROWS)
    q, q_t = (torch.empty(n, D // 2, dtype=torch.uint8, device="cuda") for n in (ROWS, TAIL))
    s, s_t = (torch.empty(n, O.mx_scale_cols(D), dtype=torch.uint8, device="cuda")
              for n in (ROWS, TAIL))
    M.moe_mx_quantize(x, "e2m1", q, s)
    M.moe_mx_quantize(x[last].clone(), "e2m1", q_t, s_t)
    assert torch.equal(q[last], q_t) and torch.equal(s[last], s_t)
    back, back_t = torch.empty_like(x), torch.empty_like(x[last])
    M.moe_mx_dequantize(q, s, "e2m1", back)
    M.moe_mx_dequantize(q_t, s_t, "e2m1", back_t)
    assert torch.equal(back[last], back_t)


def test_experts():
    print("\n[case] large experts", flush=True)
    f, E = 64, 2
    torch.manual_seed(5)
    xq, xs = _bytes(ROWS, D, top=127), _bytes(ROWS, O.mx_scale_cols(D), top=9) + 110
    w1, w3, w2 = _bytes(E, f, D // 2), _bytes(E, f, D // 2), _bytes(E, D, f // 2)
    s1, s3 = (_bytes(E, f, O.mx_scale_cols(D), top=9) + 120 for _ in range(2))
    s2 = _bytes(E, D, O.mx_scale_cols(f), top=9) + 120

    def run(xq, xs, offsets):
        n = xq.shape[0]
        dims = M.make_dims(n, D, E, f, 1, torch.bfloat16)
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        hq = torch.empty(n, f, dtype=torch.uint8, device="cuda")
        hs = torch.empty(n, O.mx_scale_cols(f), dtype=torch.uint8, device="cuda")
        y = torch.empty(n, D, dtype=torch.bfloat16, device="cuda")
        M.moe_expert_up_mx(dims, xq, xs, None, off, w1, s1, w3, s3, hq, hs)
        M.moe_expert_down_mx(dims, hq, hs, off, w2, s2, y)
        return hq, hs, y

    whole = run(xq, xs, [0, 5000, ROWS])
    alone = run(xq[-TAIL:].clone(), xs[-TAIL:].clone(), [0, 0, TAIL])
    for a, b in zip(whole, alone):
        assert torch.equal(a[-TAIL:], b)
