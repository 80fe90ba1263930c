"""Rows at the ends of fp32's range in the block around the experts: norms of the largest rows and
their gradients, sums of products that pass the range where the results do not.

The bounds are those of test_block (they are relative to the terms' magnitudes, and a power of two
that is taken out and put back changes none of them); gradients among fp32's smallest numbers add
2^-130, half a step of the bf16 ones there and more than the reciprocal's own rounding."""

import numpy as np
import pytest
import torch

from test_block import BF, EPS, F32, OPS, SUM, U, Block, Norm, backward, f64, forward, inputs, moe, near, norm_backward, take

TINY = 2.0 ** -130


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


def check_before(s, scale=1.0, residual=False):
    """moe_norm_backward against the formula, with add and the copies' gradients."""
    gx, gw, ws = norm_backward(s, False, scale, residual=residual)
    moe().moe_check_device_status(ws)
    T, H = s["x"].shape
    terms = take(f64(s["grad"]), s["dest"].cpu().numpy())
    u, du = terms.sum(1) + f64(s["add"]), SUM * (np.abs(terms).sum(1) + np.abs(f64(s["add"])))
    wt, n = f64(s["weight"]), Norm(f64(s["x"]))
    d, dd, _ = n.back(u * wt, np.abs(wt) * du + OPS * np.abs(u * wt))
    near(gx, d, dd + OPS * np.abs(d) + TINY, "x")
    hat, dhat = n.out(np.ones(H))
    near(gw, (u * hat).sum(0), (du * np.abs(hat) + np.abs(u) * dhat + (T * U + OPS) * np.abs(u * hat)).sum(0), "weight")


def check_after(s, post=True):
    out, ws = backward(s, post)
    moe().moe_check_device_status(ws)
    T, H = s["x"].shape
    want = Block(s if post else {**s, "weight": None}, T, H, post, 1.0).backward()
    live = s["dest"].cpu().numpy() >= 0
    near(out["rows"][s["dest"][s["dest"] >= 0].long()], want["rows"][0][live], want["rows"][1][live] + TINY, "rows")
    near(out["w"], *want["w"], "w")
    near(out["shared"], want["shared"][0], want["shared"][1] + TINY, "shared")
    near(out["gate"], *want["gate"], "gate")
    if post:
        near(out["weight"], *want["weight"], "weight")


def signs(*shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    return 1.0 - 2.0 * torch.randint(0, 2, shape, generator=gen, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H", [1024, 4104, 8192, 16384])
def test_largest_rows(H, dt):
    """3e38 in every place of a row, in one place only, and rows next to them of ordinary size."""
    m = moe()
    T, k = 4, 2
    s = inputs(T, H, k, dt, True, True, True, 0, seed=30)
    s["x"][0] = (3e38 * signs(H)).to(dt)
    s["x"][1, H - 3] = 3e38
    n = torch.empty(T, H, dtype=BF, device="cuda")
    m.moe_norm(s["x"], s["weight"], EPS, n)
    near(n, *Norm(f64(s["x"])).out(f64(s["weight"])), "norm")
    check_before(s)
    # the next block's norm, of y as it is held, and the norm of the experts' sum
    s["w"][2] = 0.5
    s["yp"][s["dest"][2].long()] = (3e38 * signs(H)).to(BF)
    s["shared"][2] = 0
    y, nx, ws = forward(s, True, 1.0)
    m.moe_check_device_status(ws)
    near(y, *Block(s, T, H, True, 1.0).forward(), "y")
    near(nx, *Norm(f64(y)).out(f64(s["next_weight"])), "next")
    check_after(s)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_large_eps_beside_large_rows(dt):
    """eps counts next to squares that pass the range as it does next to others."""
    m = moe()
    H, eps = 8, 1e38
    x = (1e19 * signs(3, H)).to(dt)
    out = torch.empty(3, H, dtype=BF, device="cuda")
    m.moe_norm(x, None, eps, out)
    v = f64(x)
    want = v / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    near(out, want, (SUM + OPS) * np.abs(want), "norm")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_no_norm_and_large_rows(dt):
    """Without a norm the gradients do not depend on the sum c: products with it may pass the range,
    and c itself may be infinite."""
    T, H, k = 4, 4096, 3
    s = inputs(T, H, k, dt, True, True, False, 0, seed=31)
    r = s["dest"][1].long()
    s["yp"][r] = (s["yp"][r].float() * 1e18).to(BF)
    out, ws = backward(s, False)
    moe().moe_check_device_status(ws)
    want = Block(s, T, H, False, 1.0).backward()
    near(out["w"], *want["w"], "w")
    near(out["rows"][s["dest"].long()], *want["rows"], "rows")
    near(out["shared"], *want["shared"], "shared")
    bad = s["dest"][2, 1].long()
    s["yp"][bad, 9] = float("inf")
    got, _ = backward(s, False)
    assert torch.equal(got["rows"][s["landed"]], out["rows"][s["landed"]])
    assert torch.equal(got["shared"], out["shared"])
    keep = torch.ones(T, k, dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(got["w"][keep], out["w"][keep]) and not torch.isfinite(got["w"][2, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H,k", [(256, 2), (4096, 8), (8192, 3), (16384, 12)])
def test_products_past_the_range_beside_a_norm(H, k, dt):
    """Sums of squares within fp32's range, products with the rows or with the gradient beyond it."""
    T = 5
    s = inputs(T, H, k, dt, True, True, True, 0, seed=32)
    # experts' rows far larger than their weighted sum
    r = s["dest"][1].long()
    s["yp"][r] = (s["yp"][r].float() * 1e30).to(BF)
    s["w"][1] *= 1e-25
    # one of them alone, with the others' rows of ordinary size or small
    s["yp"][s["dest"][2, 0].long()] = (s["yp"][s["dest"][2, 0].long()].float() * 1e33).to(BF)
    s["w"][2, 0] = 1e-28
    s["yp"][s["dest"][2, 1].long()] = (s["yp"][s["dest"][2, 1].long()].float() * 1e-20).to(BF)
    check_after(s)
    # a large sum and a large gradient
    r = s["dest"][3].long()
    s["yp"][r] = (s["yp"][r].float() * 1e16).to(BF)
    s["gy"][3] = (s["gy"][3].float() * 1e24).to(dt)
    check_after(s)
    s["x"][0] = (s["x"][0].float() * 1e16).to(dt)
    g = s["dest"][0].long()
    s["grad"][g] = (s["grad"][g].float() * 1e24).to(BF)
    check_before(s)
