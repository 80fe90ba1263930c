"""The ends of eps, products of sums beyond fp32's range, and tokens of every size one after another
in a team, in the block around the experts.  Bounds as in test_block_range."""

import ctypes

import numpy as np
import pytest
import torch

from test_block import BF, F32, FAKE, OPS, SUM, U, Block, f64, forward, inputs, moe, near
from test_block_range import check_after, check_before, signs


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


def test_eps_beyond_the_ends_is_refused():
    """Below 2^-126 its reciprocal, which the gradients take, passes fp32's range; above 2^127 it does
    with a mean square beside it."""
    m = moe()
    L = m.lib()
    cfg = lambda eps: ctypes.byref(m.BlockCfg(1, eps, 1.0))
    norm = lambda eps: L.moe_norm(FAKE, 0, 0, 64, None, eps, FAKE, None)
    comb = lambda eps: L.moe_combine_norm(FAKE, 8, FAKE, FAKE, 0, 2, 64, None, FAKE, 0, None, None, cfg(eps), FAKE, None,
                                          None, FAKE, 256, None)
    cbwd = lambda eps: L.moe_combine_norm_backward(FAKE, 0, FAKE, 8, FAKE, FAKE, 0, 2, 64, None, None, None, cfg(eps),
                                                   FAKE, FAKE, None, None, None, None, 0, FAKE, 256, None)
    nbwd = lambda eps: L.moe_norm_backward(FAKE, 8, FAKE, 2, None, FAKE, 0, 0, 64, None, eps, None, 1.0, FAKE, None,
                                           None, 0, FAKE, 256, None)
    for f in (norm, comb, cbwd, nbwd):
        assert [f(e) for e in (2.0 ** -127, 1e-44, 2.0 ** 127 * 1.01, 3e38)] == [1] * 4
        assert [f(e) for e in (2.0 ** -126, 1e-12, 2.0 ** 127)] == [0] * 3


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_smallest_eps(dt):
    """eps = 2^-126: rows of zeros keep finite gradients, r u weight with r = 2^63."""
    m = moe()
    T, H, k, eps = 3, 264, 2, 2.0 ** -126
    s = inputs(T, H, k, dt, False, True, True, 0, seed=40)
    ws, sc = m.new_workspace(T, k, 1), m.new_norm_scratch(T, H)
    x, gx, gw = torch.zeros(T, H, dtype=dt, device="cuda"), torch.empty(T, H, dtype=dt, device="cuda"), torch.empty(H, device="cuda")
    x[1] = 1e-20
    m.moe_norm_backward(s["add"], x, s["weight"], eps, gx, gw, ws, sc)
    u, wt, v = f64(s["add"]), f64(s["weight"]), f64(x)
    e, r = u * wt, 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    mean, mag = (e * v).mean(1, keepdims=True), np.abs(e * v).mean(1, keepdims=True)
    want = r * (e - v * r * r * mean)
    near(gx, want, (SUM + 4 * OPS) * r * (np.abs(e) + np.abs(v) * r * r * mag), "x")
    near(gw, (u * v * r).sum(0), (SUM + OPS) * np.abs(u * v * r).sum(0), "weight")
    # after the experts: nothing arrives and nothing is shared
    dest = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    zero, gs = torch.zeros(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    rows, w = torch.zeros_like(s["yp"]), torch.empty(T, k, device="cuda")
    m.moe_combine_norm_backward(s["gy"], s["yp"], dest, s["w"], m.BlockCfg(1, eps, 1.0), rows, w, ws, sc, shared=zero,
                                weight=s["weight"], grad_shared=gs, grad_weight=gw)
    m.moe_check_device_status(ws)
    want = f64(s["gy"]) * wt * 2.0 ** 63
    near(gs, want, 4 * OPS * np.abs(want), "shared")
    assert (gw == 0).all() and (w == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H", [1024, 16384])
def test_product_of_sums_beyond_the_range(H, dt):
    """e . Y = 0, e . c and c . Y within the range, their product beyond it, and a gate that brings the
    weight's gradient back."""
    T, k = 3, 2
    s = inputs(T, H, k, dt, True, True, True, 0, seed=41)
    s["gy"][1, :H // 2] = (1e20 * s["gy"][1, :H // 2].float()).to(dt)
    s["gy"][1, H // 2:] = 0
    row = s["dest"][1, 0].long()
    s["yp"][row, :H // 2] = 0
    s["yp"][row, H // 2:] = (1e20 * s["yp"][row, H // 2:].float()).to(BF)
    s["w"][1, 0], s["gate"][1] = 1e-22, 1e-12
    check_after(s)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,k,dt", [(8000, 256, 2, BF), (5000, 264, 5, F32), (700, 8192, 3, BF), (400, 12288, 2, F32)])
def test_tokens_of_every_size_in_turn(T, H, k, dt):
    """Several tokens a team, those with sums beyond the range among others."""
    m = moe()
    s = inputs(T, H, k, dt, True, True, True, 0.1, seed=42)
    kind = torch.randint(0, 4, (T,), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    factor = torch.tensor([1.0, 1e25, 1e-12, 1e30], device="cuda")[kind]
    small = torch.tensor([1.0, 1.0, 1.0, 1e-25], device="cuda")[kind]
    live = s["dest"] >= 0
    for name, f in (("yp", factor), ("grad", torch.tensor([1.0, 1.0, 1e10, 1e-10], device="cuda")[kind])):
        rows = s[name][s["dest"][live].long()].float() * f[:, None].expand(T, k)[live][:, None]
        s[name][s["dest"][live].long()] = rows.to(BF)
    s["w"] = (s["w"] * small[:, None]).contiguous()
    s["x"] = (s["x"].float() * factor[:, None]).to(dt)
    for i in range(0, T, 97):
        s["x"][i] = (3e38 * signs(H)).to(dt)
    y, nx, ws = forward(s, True, 0.5)
    m.moe_check_device_status(ws)
    near(y, *Block(s, T, H, True, 0.5).forward(), "y")
    check_after(s)
    check_before(s)
