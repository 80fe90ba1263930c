"""SwiGLU of the FP4 product over the whole range of gate and up values.

Every sum here is exact (small integers, factors that are powers of two), so
a result is silu(g) u up to the epilogue's own arithmetic: relative 2^-19 for
exponential, division and products in fp32 (the exponent -g log2 e of up to
126 carries an error of 126 * 2^-24, below 2^-17 in the result; counted with
the rest as 2^-16), and one rounding to bf16, 2 * 2^-8 as in test_fp4_product.
What e^-g beyond 2^126 takes from a result is at most 2^-119 |u|.
"""

import numpy as np
import pytest
import torch

from test_fp4_rows import MX, NV


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


def run(alpha, fmt, out_t):
    """Row r, column c of expert e: g = alpha_e G[r, c], u = alpha_e U[r, c]."""
    m = moe()
    E, K, I, R = len(alpha), 64, 32, 16
    rng = np.random.default_rng(1)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    signed = np.concatenate((grid, -grid))
    xc = rng.integers(0, 3, (R, K))                      # 0, 0.5, 1
    wc = rng.integers(0, 16, (2 * I, K))
    wc[:I // 2] |= 8                                     # gates of half the columns below zero
    X, W = signed[xc], signed[wc]
    one = 127 if fmt == MX else 0x38                     # the scale 1
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    pack = lambda c: (c[..., 0::2] + 16 * c[..., 1::2]).astype(np.uint8)
    ld = m.moe_fp4_scale_ld(K, fmt)
    sf = np.zeros((1, ld), np.uint8)
    sf[:, :K // (32 if fmt == MX else 16)] = one
    w = m.pack_weights_fp4(cu(np.tile(pack(wc), (E, 1, 1))), cu(np.tile(sf, (E, 2 * I, 1))), fmt, m.MOE_EPI_SWIGLU)
    out = torch.empty(E * R, I, dtype=out_t, device="cuda")
    ws = m.new_workspace(E * R, 1, E)
    m.moe_grouped_product_fp4(cu(np.tile(pack(xc), (E, 1))), cu(np.tile(sf, (E * R, 1))),
                              torch.arange(0, E * R + 1, R, dtype=torch.int32, device="cuda"),
                              torch.arange(E, dtype=torch.int32, device="cuda"), w,
                              torch.tensor(alpha, dtype=torch.float32, device="cuda"), out, ws)
    m.moe_check_device_status(ws)
    y = X @ W.T
    a = np.repeat(np.array(alpha), R)[:, None]
    return out.float().cpu().numpy().astype(np.float64), a * np.tile(y[:, :I], (E, 1)), a * np.tile(y[:, I:], (E, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("out_t", [torch.bfloat16, torch.float32])
def test_gates_of_every_size(out_t, fmt):
    alpha = [2.0 ** j for j in range(-20, 100, 2)] + [2.0 ** j for j in (-1, 0, 1)]
    got, g, u = run(alpha, fmt, out_t)
    with np.errstate(over="ignore"):
        y = g / (1 + np.exp(-g)) * u
    top = float(torch.finfo(torch.bfloat16).max)
    tol = (2 * 2.0 ** -8 if out_t == torch.bfloat16 else 0) * np.abs(y) + 2.0 ** -16 * np.abs(y) \
        + 2.0 ** -119 * np.abs(u) + 2.0 ** -125
    assert (g < -2.0 ** 60).any() and ((g < -50) & (g > -80)).any()
    small = np.abs(y) < top / 2
    bad = small & ~(np.abs(got - y) <= tol)
    assert not bad.any(), [(g[i], u[i], y[i], got[i]) for i in map(tuple, np.argwhere(bad)[:6])]
    big = np.abs(y) > 2 * top
    assert big.any() and (got[big] == np.sign(y[big]) * np.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("out_t", [torch.bfloat16, torch.float32])
def test_nan_and_infinity_stay_with_their_values(out_t):
    """A row with the NaN scale beside others; a factor that makes gates infinite."""
    m = moe()
    rng = np.random.default_rng(4)
    n, K, I = 40, 128, 32
    cu = lambda a: torch.from_numpy(a).cuda()
    wc, xc = (rng.integers(0, 256, s).astype(np.uint8) for s in ((1, 2 * I, K // 2), (n, K // 2)))
    ld = m.moe_fp4_scale_ld(K, NV)
    xs, wsf = np.zeros((n, ld), np.uint8), np.zeros((1, 2 * I, ld), np.uint8)
    xs[:, :K // 16], wsf[:, :, :K // 16] = 0x38, 0x30
    w = m.pack_weights_fp4(cu(wc), cu(wsf), NV, m.MOE_EPI_SWIGLU)
    ws = m.new_workspace(n, 1, 1)
    offs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    expert = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(scales, alpha):
        out = torch.empty(n, I, dtype=out_t, device="cuda")
        m.moe_grouped_product_fp4(cu(xc), cu(scales), offs, expert, w, torch.tensor([alpha], device="cuda"), out, ws)
        m.moe_check_device_status(ws)
        return out.float().cpu()

    plain = call(xs, 0.01)
    assert torch.isfinite(plain).all()
    for r in (0, 7, 18, 39):
        bad = xs.copy()
        bad[r, 2] = 127
        got = call(bad, 0.01)
        keep = torch.arange(n) != r
        assert torch.isnan(got[r]).all() and torch.equal(got[keep], plain[keep])
    # g = -inf is NaN as in g / (1 + e^-g), g = +inf times u is infinite; 0 stays 0
    got = call(xs, 3e38)
    assert not torch.isfinite(got).all() and torch.isnan(got).any() and torch.isinf(got).any()
