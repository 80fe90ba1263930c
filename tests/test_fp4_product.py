"""The grouped product of FP4 rows with FP4 expert weights against the
definition in moe.h, in 64 bits.

Tolerance: the products are exact in fp32; K / 64 sums of 64 products follow
one another, each cut to 24 bits or better at the size of what it adds, so a
result is within (K / 64 + 64) * 2^-23 of the sum of its terms' magnitudes,
and a bf16 result adds 2^-8 of its value.  SwiGLU passes the errors of g and u
on (|silu'| <= 1.1) and adds 2^-19 of the value for exponential and division
(fp32; the bf16 form's are below half a bf16 step, counted once more).  Where
every sum is exact in fp32, results are equal.
"""

import ctypes

import numpy as np
import pytest
import torch

from test_fp4_rows import E4M3, GRID, MX, NV

SIGNED = np.concatenate((GRID, -GRID))


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
ODD = ctypes.c_void_p(0x10008)


def test_refusals():
    L = moe().lib()

    def f(c=FAKE, s=FAKE, n=8, so=FAKE, se=FAKE, S=4, E=4, w=FAKE, N=16, K=64, fmt=0, ep=0, o=FAKE, t=1, ws=FAKE,
          b=256):
        return L.moe_grouped_product_fp4(c, s, n, so, se, S, E, w, N, K, fmt, ep, None, o, t, ws, b, None)

    assert f(n=0) == 0
    assert all(v == 1 for v in (f(c=None), f(s=None), f(so=None), f(se=None), f(w=None), f(o=None), f(n=-1), f(S=0),
                                f(E=0), f(N=0), f(K=0), f(fmt=2), f(ep=2), f(t=2), f(c=ODD), f(s=ODD), f(w=ODD),
                                f(o=ODD)))
    assert all(v == 2 for v in (f(S=1025), f(K=48), f(N=12), f(N=24, ep=1), f(n=2 ** 31 - 16),
                                f(N=2 ** 30, n=2 ** 20)))
    assert f(ws=None) == 6 and f(ws=ODD) == 6 and f(b=64) == 6


# ------------------------------------------------------------------ GPU
def fp4_tensor(shape, fmt, rng, lo, hi, exact=False):
    """Codes and scales [.., K/2], [.., ld] as uint8 arrays, and their values in 64 bits."""
    *lead, K = shape
    blk = 32 if fmt == MX else 16
    ld = -(-K // 256) * (8 if fmt == MX else 16)
    c = rng.choice([0, 1, 2, 9, 10], (*lead, K)) if exact else rng.integers(0, 16, (*lead, K))
    sf = np.zeros((*lead, ld), np.uint8)
    if fmt == MX:
        e = rng.integers(lo, hi + 1, (*lead, K // blk))
        sf[..., :K // blk] = e + 127
        scale = 2.0 ** e
    else:
        b = rng.integers((lo + 7) * 8, (hi + 7) * 8 + 8, (*lead, K // blk))
        if exact:
            b = b // 8 * 8
        sf[..., :K // blk] = b
        scale = E4M3[b]
    val = SIGNED[c] * np.repeat(scale, blk, -1)
    return (c[..., 0::2] + 16 * c[..., 1::2]).astype(np.uint8), sf, val


def product(x, w, bounds, experts, alpha, I):
    """Result and error bound factor (the terms' magnitudes) in 64 bits, for every row in a segment."""
    n, K = x.shape
    N = w.shape[1]
    y, mag = np.full((n, N), np.nan), np.zeros((n, N))
    for s, e in enumerate(experts):
        lo, hi = bounds[s], bounds[s + 1]
        a = 1.0 if alpha is None else float(alpha[e])
        y[lo:hi] = a * (x[lo:hi] @ w[e].T)
        mag[lo:hi] = abs(a) * (np.abs(x[lo:hi]) @ np.abs(w[e]).T)
    err = (K / 64 + 64) * 2.0 ** -23 * mag
    if not I:
        return y, err
    g, u, eg, eu = y[:, :I], y[:, I:], err[:, :I], err[:, I:]
    with np.errstate(over="ignore"):
        sg = g / (1 + np.exp(-g))
    return sg * u, 1.1 * eg * (np.abs(u) + eu) + np.abs(sg) * eu + 2.0 ** -19 * np.abs(sg * u)


CASES = [  # rows per segment, first row, E, N, K, swiglu, alpha
    ((1,), 0, 1, 8, 32, False, False),
    ((3, 0, 17), 0, 4, 264, 288, False, True),
    ((0, 0, 112, 113, 0, 1), 5, 6, 256, 256, False, True),
    ((40, 16, 15), 0, 3, 272, 1440, True, True),
    ((500, 0, 1), 2, 3, 48, 96, True, False),
    ((225,), 0, 2, 520, 512, False, True),
    ((8, 8, 8, 8), 0, 5, 512, 7168, True, True),
    ((1,) * 300, 0, 7, 16, 64, False, True),
]


def setup(case, fmt, seed, exact=False):
    counts, first, E, N, K, swiglu, has_alpha = case
    m = moe()
    rng = np.random.default_rng(seed)
    bounds = (first + np.concatenate(([0], np.cumsum(counts)))).astype(np.int32)
    n = int(bounds[-1]) + 3                       # rows after the last segment
    experts = rng.integers(0, E, len(counts)).astype(np.int32)
    span = (0, 0) if exact else (-2, 1)
    xc, xs, xv = fp4_tensor((n, K), fmt, rng, *span, exact)
    wc, wsf, wv = fp4_tensor((E, N, K), fmt, rng, *span, exact)
    size = np.sqrt(K) * (1 if exact else 20)
    alpha = (2.0 ** -np.round(np.log2(size)) * (1 if exact else rng.uniform(0.5, 2, E))).astype(np.float32) \
        * np.ones(E, np.float32) if has_alpha else None
    cu = lambda a: torch.from_numpy(a).cuda()
    w = m.pack_weights_fp4(cu(wc), cu(wsf), fmt, m.MOE_EPI_SWIGLU if swiglu else m.MOE_EPI_NONE)
    args = [cu(xc), cu(xs), cu(bounds), cu(experts), w, None if alpha is None else cu(alpha)]
    return args, (xv, wv, bounds, experts, alpha, N // 2 if swiglu else 0), n


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("case", CASES)
def test_exact_sums(case, fmt):
    """Small integers under one scale: every sum is exact, the result too."""
    args, ref, n = setup(case[:5] + (False,) + case[6:], fmt, 1, exact=True)
    m = moe()
    out = torch.full((n, case[3]), float("nan"), device="cuda")
    ws = m.new_workspace(n, 1, len(case[0]))
    m.moe_grouped_product_fp4(*args, out, ws)
    m.moe_check_device_status(ws)
    y, _ = product(*ref)
    assert np.array_equal(out.cpu().numpy(), y.astype(np.float32), equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("case", CASES)
def test_product(case, fmt, out_t):
    args, ref, n = setup(case, fmt, 2)
    m = moe()
    y, err = product(*ref)
    out = torch.full((n, y.shape[1]), float("nan"), dtype=out_t, device="cuda")
    ws = m.new_workspace(n, 1, len(case[0]))
    m.moe_grouped_product_fp4(*args, out, ws)
    m.moe_check_device_status(ws)
    got = out.float().cpu().numpy().astype(np.float64)
    lo, hi = ref[2][0], ref[2][-1]
    assert np.isnan(got[:lo]).all() and np.isnan(got[hi:]).all()
    tol = err + (2 * 2.0 ** -8 * np.abs(y) if out_t == torch.bfloat16 else 0) + 2.0 ** -100
    bad = np.abs(got - y)[lo:hi] > tol[lo:hi]
    assert not bad.any(), (np.argwhere(bad)[:5], (np.abs(got - y) / tol)[lo:hi].max())
    # rows do not depend on their neighbours, nor calls on one another
    again = torch.full_like(out, float("nan"))
    m.moe_grouped_product_fp4(*args, again, ws)
    assert torch.equal(again[lo:hi], out[lo:hi])


LONG = [  # many rows a segment: tiles of more than 112 rows, mixed with small ones
    ((300, 0, 113, 112, 224, 225, 1, 700), 3, 4, 264, 288, False, True),
    ((129, 448, 16, 97, 336), 0, 2, 272, 512, True, True),
    ((1000, 240), 0, 3, 1040, 160, False, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("case", LONG)
def test_long_segments(case, fmt, out_t):
    test_product(case, fmt, out_t)
    test_exact_sums(case, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("S", [767, 768, 1024])
def test_many_segments(S):
    """As many segments as the kernel's tables hold, empty ones among them."""
    rng = np.random.default_rng(S)
    counts = tuple(int(c) for c in rng.choice([0, 0, 1, 2, 17, 130], S))
    test_exact_sums((counts, 1, 9, 40, 96, False, True), NV)


@pytest.mark.gpu
def test_nan_stays_in_its_row():
    m = moe()
    args, ref, n = setup(((20, 20), 0, 2, 64, 128, False, False), NV, 3)
    args[1][7, 2] = 127
    out = torch.empty(n, 64, device="cuda")
    ws = m.new_workspace(n, 1, 2)
    m.moe_grouped_product_fp4(*args, out, ws)
    nan = torch.isnan(out[:40]).cpu()
    assert nan[7].all() and int(nan.sum()) == 64


@pytest.mark.gpu
def test_bad_segments_are_reported_and_skipped():
    m = moe()
    args, ref, n = setup(((4, 4, 4), 0, 3, 16, 64, False, False), MX, 4)
    ws = m.new_workspace(n, 1, 3)
    experts = args[3]
    for bad in (-1, 3):
        args[3] = experts.clone()
        args[3][1] = bad
        out = torch.full((n, 16), 5.0, device="cuda")
        m.moe_grouped_product_fp4(*args, out, ws)
        with pytest.raises(m.MoeError) as e:
            m.moe_check_device_status(ws)
        assert e.value.status == 4 and e.value.info == 1
        assert (out[4:8] == 5.0).all() and not (out[:4] == 5.0).all() and not (out[8:12] == 5.0).all()
    args[3] = experts
    for offs, info, written in (([0, 4, 8, n + 1], 2, 8), ([-4, 4, 8, 12], 0, 12), ([0, 8, 4, 12], 1, 0)):
        args[2] = torch.tensor(offs, dtype=torch.int32, device="cuda")
        out = torch.full((n, 16), 5.0, device="cuda")
        m.moe_grouped_product_fp4(*args, out, ws)
        with pytest.raises(m.MoeError) as e:
            m.moe_check_device_status(ws)
        assert e.value.status == 4 and e.value.info == info
        first = 4 if offs[0] < 0 else 0
        assert (out[:first] == 5.0).all() and (out[written:] == 5.0).all()
        assert written == 0 or not (out[first:written] == 5.0).any()


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    m = moe()
    args, ref, n = setup(((30, 0, 50), 0, 3, 272, 512, True, True), NV, 5)
    ws = m.new_workspace(n, 1, 3)
    out = torch.zeros(n, 136, dtype=torch.bfloat16, device="cuda")
    m.moe_grouped_product_fp4(*args, out, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = torch.zeros_like(out)
    side.wait_stream(torch.cuda.current_stream())
    m.moe_grouped_product_fp4(*args, other, ws, side)
    side.synchronize()
    assert torch.equal(out, other)
    other.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_grouped_product_fp4(*args, other, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, other)
    # other segment sizes, same graph
    args[2].copy_(torch.tensor([0, 1, 70, 80], dtype=torch.int32))
    graph.replay()
    m.moe_grouped_product_fp4(*args, out, ws)
    assert torch.equal(out[:80], other[:80])


@pytest.mark.gpu
@pytest.mark.parametrize("out_t", [torch.float32, torch.bfloat16])
def test_offsets_past_32_bits(out_t):
    """Results more than 4 GiB into the output: the last rows against the same rows alone."""
    m = moe()
    rng = np.random.default_rng(9)
    n, N, K = 1_200_000, 2048, 64
    wc, wsf, _ = fp4_tensor((2, N, K), MX, rng, -2, 1)
    xc, xs, _ = fp4_tensor((300, K), MX, rng, -2, 1)
    w = m.pack_weights_fp4(torch.from_numpy(wc).cuda(), torch.from_numpy(wsf).cuda(), MX, m.MOE_EPI_NONE)
    codes, sf = m.new_fp4(n, K, MX)
    codes.zero_(), sf.fill_(127)
    codes[-300:], sf[-300:] = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda()
    ws = m.new_workspace(n, 1, 2)
    experts = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, n - 200, n], dtype=torch.int32, device="cuda")
    out = torch.full((n, N), 3.0, dtype=out_t, device="cuda")
    m.moe_grouped_product_fp4(codes, sf, offs, experts, w, None, out, ws)
    m.moe_check_device_status(ws)
    few = torch.empty(300, N, dtype=out_t, device="cuda")
    offs = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    m.moe_grouped_product_fp4(codes[-300:].contiguous(), sf[-300:].contiguous(), offs, experts, w, None, few, ws)
    assert torch.equal(out[-300:], few) and few.abs().max() > 0 and not out[:-300].any()
