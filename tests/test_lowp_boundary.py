"""Host-side checks of the norm's and the low-precision experts' entry points (no
GPU): bad arguments get the documented status before anything is enqueued.
Pointers are fake and used only where validation must fail."""
import ctypes

import pytest
import torch

import top_routing_grouped_router_amd as M
from top_routing_grouped_router_amd import _lib as L
from oracle import moe_oracle as O

INVALID, UNSUP, WS = 1, 2, 3
FAKE = 1 << 20


def dims(T=64, d=64, E=8, f=64, k=2, act=1):
    return L.moe_dims(T, d, E, f, k, act)


def call(name, *args):
    st = getattr(L.lib(), name)(*args)
    return st, L.last_error()


def norm(dm, x=FAKE, res=None, w=FAKE, eps=1e-6, s=None, y=FAKE, q=None, qs=None, rstd=None):
    return call("moe_rmsnorm", ctypes.byref(dm), x, res, w, eps, s, y, q, qs, rstd, None)


def norm_bwd(dm, *p, ws=FAKE, n=1 << 30):
    p = list(p) + [FAKE] * (7 - len(p))
    return call("moe_rmsnorm_bwd", ctypes.byref(dm), *p, ws, n, None)


def test_header_limits_match_the_binding():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "moe.h")).read()
    assert int(re.search(r"#define MOE_TOKEN_MAX_SLOTS (\d+)", text)[1]) == M.MOE_TOKEN_MAX_SLOTS
    assert "MOE_MX_E4M3 = 0, MOE_MX_E2M1 = 1" in text


@pytest.mark.parametrize("n", [1, 63, 64, 128, 192, 320, 2048, 0, -64])
def test_scale_cols(n):
    want = O.mx_scale_cols(n) if n > 0 and n % 64 == 0 else 0
    assert M.moe_mx_scale_cols(n) == want


@pytest.mark.parametrize("kw", [dict(d=96), dict(E=257), dict(T=-1), dict(act=7), dict(k=9)])
def test_bad_dims(kw):
    dm = dims(**kw)
    want = INVALID if kw.get("T", 0) < 0 else UNSUP
    assert norm(dm)[0] == want
    assert norm_bwd(dm)[0] == want
    b = ctypes.byref(dm)
    assert call("moe_expert_up_mx", b, *([FAKE] * 10), None)[0] == want
    assert call("moe_expert_down_mx", b, *([FAKE] * 6), None)[0] == want
    assert call("moe_token_swiglu", b, *([FAKE] * 10), FAKE, 1 << 30, None)[0] == want
    assert L.lib().moe_rmsnorm_bwd_workspace_bytes(b) == 0
    assert L.lib().moe_token_swiglu_workspace_bytes(b) == 0


def test_norm_arguments():
    assert norm(dims(), x=None)[0] == INVALID
    assert norm(dims(), w=None)[0] == INVALID
    st, why = norm(dims(), y=None)
    assert st == INVALID and "'y' or 'q'" in why
    st, why = norm(dims(), q=FAKE)
    assert st == INVALID and "together" in why
    assert norm(dims(), qs=FAKE)[0] == INVALID
    for eps in (-1e-6, float("nan"), float("inf")):
        st, why = norm(dims(), eps=eps)
        assert st == INVALID and "eps" in why
    st, why = norm(dims(), res=FAKE + 4)
    assert st == INVALID and "aligned" in why
    st, why = norm(dims(), s=FAKE, y=FAKE)
    assert st == INVALID and "one tensor" in why
    for at in range(7):
        p = [FAKE] * 7
        p[at] = None
        if at != 4:   # dsum may be missing
            assert norm_bwd(dims(), *p)[0] == INVALID, at
    dm = dims(T=4096, d=2048)
    need = L.lib().moe_rmsnorm_bwd_workspace_bytes(ctypes.byref(dm))
    assert 0 < need <= L.lib().moe_workspace_bytes(ctypes.byref(dm), 1)
    assert norm_bwd(dm, n=need - 1)[0] == WS
    assert norm_bwd(dm, ws=None)[0] == WS


def test_mx_arguments():
    def quant(rows=4, cols=64, dt=0, src=FAKE, fmt=0, q=FAKE, s=FAKE):
        return call("moe_mx_quantize", rows, cols, dt, src, fmt, q, s, None)

    def dequant(rows=4, cols=64, fmt=0, q=FAKE, s=FAKE, dt=0, dst=FAKE):
        return call("moe_mx_dequantize", rows, cols, fmt, q, s, dt, dst, None)

    for f in (quant, dequant):
        assert f(rows=-1)[0] == INVALID and f(cols=0)[0] == INVALID
        assert f(cols=96)[0] == UNSUP and f(dt=2)[0] == UNSUP and f(fmt=2)[0] == UNSUP
        assert f(rows=1 << 40)[0] == UNSUP
        assert f(q=None)[0] == INVALID and f(s=None)[0] == INVALID
        assert f(s=FAKE + 1)[0] == INVALID
    assert quant(src=None)[0] == INVALID and dequant(dst=None)[0] == INVALID


def test_mx_sizes_end_where_a_launch_does():
    """2^35 values of 4 bytes are 2^31 threads of 4 pieces; one row more is refused"""
    rows = (1 << 35) // 64 + 1
    for cols, dt in ((64, 0), (64, 1)):
        for fn, args in (("moe_mx_quantize", (dt, FAKE, 0)), ("moe_mx_dequantize", (0, FAKE, FAKE))):
            tail = (FAKE, FAKE, None) if fn == "moe_mx_quantize" else (dt, FAKE, None)
            st, why = call(fn, rows, cols, *args, *tail)
            assert st == UNSUP and "2^35" in why


def test_experts_arguments():
    for at in range(10):
        p = [FAKE] * 10
        p[at] = None
        if at != 2:   # src_token may be missing
            assert call("moe_expert_up_mx", ctypes.byref(dims()), *p, None)[0] == INVALID, at
        p[at] = FAKE + 8
        assert call("moe_expert_up_mx", ctypes.byref(dims()), *p, None)[0] == INVALID, at
    for at in range(6):
        p = [FAKE] * 6
        p[at] = None
        assert call("moe_expert_down_mx", ctypes.byref(dims()), *p, None)[0] == INVALID, at
    st, why = call("moe_expert_up_mx", ctypes.byref(dims(T=1 << 20, d=2048)), *([FAKE] * 10), None)
    assert st == UNSUP and "2 GiB" in why
    for kw in (dict(d=1 << 21), dict(f=1 << 21), dict(T=(1 << 30) - 1, k=2, f=4096)):
        p = [FAKE] * 10
        p[2] = None
        assert call("moe_expert_up_mx", ctypes.byref(dims(**kw)), *p, None)[0] == UNSUP
        assert call("moe_expert_down_mx", ctypes.byref(dims(**kw)), *([FAKE] * 6), None)[0] == UNSUP


def test_token_arguments():
    b = ctypes.byref(dims(T=8))
    for at in range(10):
        p = [FAKE] * 10
        p[at] = None
        assert call("moe_token_swiglu", b, *p, FAKE, 1 << 30, None)[0] == INVALID, at
    need = L.lib().moe_token_swiglu_workspace_bytes(b)
    assert call("moe_token_swiglu", b, *([FAKE] * 10), FAKE, need - 1, None)[0] == WS
    assert call("moe_token_swiglu", b, *([FAKE] * 10), None, need, None)[0] == WS
    big = dims(T=513, k=2)
    st, why = call("moe_token_swiglu", ctypes.byref(big), *([FAKE] * 10), FAKE, 1 << 30, None)
    assert st == UNSUP and "1024" in why
    assert L.lib().moe_token_swiglu_workspace_bytes(ctypes.byref(big)) == 0
    assert L.lib().moe_token_swiglu_workspace_bytes(ctypes.byref(dims(T=512, k=2))) > 0


def test_binding_refuses_host_tensors_and_formats():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        M.moe_rmsnorm(M.make_dims(2, 64, 1, 64, 1, torch.float32), x, None, x[0], 1e-6, None, x,
                      None, None, None)
    with pytest.raises(ValueError, match="format"):
        M.moe_mx_quantize(x, "e5m2", x, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        M.moe_mx_quantize(x, "e4m3", x, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        M.moe_token_swiglu(M.make_dims(2, 64, 1, 64, 1, torch.float32), *([None] * 11))
