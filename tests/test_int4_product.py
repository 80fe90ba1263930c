"""The grouped product of bf16 rows with 4-bit integer weights against the
definition in moe.h, in 64 bits.

Tolerance: x (q - z) has at most 8 + 7 bits and is exact in fp32; the sums of a
group's products and of the groups follow one another in fp32, each cut to 24
bits or better at the size of what it adds: K / 16 steps of 16 products that add
in 8 levels at most, and 32 more for groups and warps, so a result is within
(K / 16 + 64) * 2^-23 of the sum of its terms' magnitudes, and a bf16 result adds
2^-8 of its value.  SwiGLU passes the errors of g and u on (|silu'| <= 1.1) and
adds 2^-19 of the value for exponential and division.  Where every sum is exact
in fp32, results are equal.
"""

import ctypes

import numpy as np
import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
ODD = ctypes.c_void_p(0x10008)


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


def test_refusals():
    L = moe().lib()

    def f(x=FAKE, n=8, so=FAKE, se=FAKE, S=4, E=4, w=FAKE, N=16, K=128, g=32, z=0, ep=0, o=FAKE, t=1, ws=FAKE, b=256):
        return L.moe_grouped_product_int4(x, n, so, se, S, E, w, N, K, g, z, ep, o, t, ws, b, None)

    def p(c=FAKE, s=FAKE, z=None, E=4, N=16, K=128, g=32, ep=0, o=ctypes.c_void_p(0x20000)):
        return L.moe_pack_weights_int4(c, s, z, E, N, K, g, ep, o, None)

    assert f(n=0) == 0
    bad = [f(x=None), f(so=None), f(se=None), f(w=None), f(o=None), f(n=-1), f(S=0), f(E=0), f(N=0), f(K=0), f(g=16),
           f(g=0), f(z=2), f(ep=2), f(t=2), f(x=ODD), f(w=ODD), f(o=ODD)]
    bad += [p(c=None), p(s=None), p(o=None), p(E=0), p(N=0), p(K=0), p(g=48), p(ep=2), p(c=ODD), p(o=ODD), p(o=FAKE),
            p(s=ctypes.c_void_p(0x10001))]
    assert all(v == 1 for v in bad), bad
    big = [f(S=1025), f(K=48), f(K=96, g=64), f(N=12), f(N=24, ep=1), f(n=2 ** 31 - 64), f(N=2 ** 30, n=2 ** 20),
           f(K=2 ** 24 + 128), p(K=48), p(K=96, g=64), p(N=12), p(N=24, ep=1)]
    assert all(v == 2 for v in big), big
    assert f(ws=None) == 6 and f(ws=ODD) == 6 and f(b=64) == 6
    n = L.moe_int4_packed_bytes
    assert n(1, 32, 128, 128, 0, 0) == 2048 + 64 and n(2, 40, 160, 32, 1, 0) == 2 * 2 * 2 * (2048 + 256 + 128)
    assert n(1, 16, 64, 64, 0, 1) == 2048 + 128
    assert n(0, 32, 128, 128, 0, 0) == 0 and n(1, 12, 128, 128, 0, 0) == 0 and n(1, 32, 128, 16, 0, 0) == 0


def test_binding_refusals():
    m = moe()
    with pytest.raises(TypeError):
        m.pack_weights_int4(torch.zeros(1, 8, 16, dtype=torch.uint8), torch.zeros(1, 8, 1).bfloat16(), None, 0)


# ------------------------------------------------------------------ GPU
CASES = [  # rows per segment, first row, E, N, K, group, zeros, swiglu
    ((1,), 0, 1, 8, 32, 32, False, False),
    ((3, 0, 17), 0, 4, 264, 288, 32, True, False),
    ((0, 0, 8, 9, 0, 1), 5, 6, 256, 256, 64, True, False),
    ((40, 16, 15), 0, 3, 272, 1440, 32, False, True),
    ((100, 0, 1), 2, 3, 48, 64, 64, True, True),
    ((33,), 0, 2, 520, 512, 128, False, False),
    ((8, 8, 8, 8), 0, 5, 512, 7168, 128, True, True),
    ((1,) * 300, 0, 7, 16, 64, 32, False, False),
    ((2, 1), 0, 2, 72, 8192, 128, False, False),
    ((7,), 1, 3, 1000, 192, 64, True, False),
    # most segments empty, none of them first or last alone
    ((0,) * 500 + (3,) + (0,) * 100 + (1, 2) + (0,) * 400 + (9,) + (0,) * 20, 0, 9, 144, 128, 32, False, True),
]


def setup(case, seed, exact=False):
    counts, first, E, N, K, group, has_zeros, swiglu = case
    m = moe()
    rng = np.random.default_rng(seed)
    bounds = (first + np.concatenate(([0], np.cumsum(counts)))).astype(np.int32)
    n = int(bounds[-1]) + 3                       # rows after the last segment
    experts = rng.integers(0, E, len(counts)).astype(np.int32)
    codes = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
    zeros = rng.integers(0, 20, (E, N, K // group)).astype(np.uint8) if has_zeros else None
    if exact:
        x = rng.integers(-2, 3, (n, K)).astype(np.float32)
        scales = 2.0 ** rng.integers(-2, 2, (E, N, K // group))
    else:
        x = rng.standard_normal((n, K))
        scales = 0.3 / np.sqrt(K) * np.exp(0.3 * rng.standard_normal((E, N, K // group)))
    x = torch.from_numpy(x).bfloat16()
    scales = torch.from_numpy(scales).bfloat16()
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, -1)
    w = (codes - z) * np.repeat(scales.double().numpy(), group, -1)
    packed = m.pack_weights_int4(torch.from_numpy(codes[..., 0::2] + 16 * codes[..., 1::2]).cuda(), scales.cuda(),
                                 None if zeros is None else torch.from_numpy(zeros).cuda(),
                                 m.MOE_EPI_SWIGLU if swiglu else m.MOE_EPI_NONE)
    args = [x.cuda(), torch.from_numpy(bounds).cuda(), torch.from_numpy(experts).cuda(), packed]
    return args, (x.double().numpy(), w, bounds, experts, N // 2 if swiglu else 0), n


def product(x, w, bounds, experts, I):
    n, K = x.shape
    y, mag = np.full((n, w.shape[1]), np.nan), np.zeros((n, w.shape[1]))
    for s, e in enumerate(experts):
        lo, hi = bounds[s], bounds[s + 1]
        y[lo:hi] = x[lo:hi] @ w[e].T
        mag[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w[e]).T
    err = (K / 16 + 64) * 2.0 ** -23 * mag
    if not I:
        return y, err
    g, u, eg, eu = y[:, :I], y[:, I:], err[:, :I], err[:, I:]
    with np.errstate(over="ignore"):
        sg = g / (1 + np.exp(-g))
    return sg * u, 1.1 * eg * (np.abs(u) + eu) + np.abs(sg) * eu + 2.0 ** -19 * np.abs(sg * u)


def call(args, n, dtype=torch.float32, ws=None, stream=None):
    m = moe()
    w = args[3]
    own = ws is None
    ws = m.new_workspace(max(n, 1), 1, 1, stream=stream) if own else ws
    with torch.cuda.stream(stream):
        out = torch.full((n, w.N // 2 if w.epilogue else w.N), 7.0, dtype=dtype, device="cuda")
    m.moe_grouped_product_int4(*args, out, ws, stream)
    if own:
        m.moe_check_device_status(ws, stream)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_exact_sums(case):
    case = (*case[:7], False)
    args, ref, n = setup(case, 1, exact=True)
    y, _ = product(*ref)
    got = call(args, n).cpu().numpy()
    inside = ~np.isnan(y)
    assert np.array_equal(got[inside], y[inside])
    assert (got[~inside] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_against_64_bits(case, dtype):
    args, ref, n = setup(case, 2)
    y, err = product(*ref)
    got = call(args, n, dtype)
    again = call(args, n, dtype)
    assert torch.equal(got, again)
    got = got.double().cpu().numpy()
    inside = ~np.isnan(y)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    bad = np.abs(got - y)[inside] > (err + half * (np.abs(y) + err))[inside]
    assert not bad.any(), np.abs(got - y)[inside][bad].max()
    assert (got[~inside] == 7.0).all()


@pytest.mark.gpu
def test_a_row_does_not_depend_on_the_others():
    """The same row alone, among few and among many of its segment: the same bits (as long as the
    number of tasks does not change how K is split)."""
    case = ((100,), 0, 1, 72, 640, 64, True, False)
    args, _, n = setup(case, 3)
    x, _, experts, w = args
    bounds = lambda k: torch.tensor([0, k], dtype=torch.int32, device="cuda")
    one = call([x[:1].contiguous(), bounds(1), experts, w], 1)
    for k in (2, 8, 9, 16, 17, 33, 100):
        assert torch.equal(call([x[:k].contiguous(), bounds(k), experts, w], k)[:1], one), k


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_row():
    case = ((5, 12), 0, 2, 64, 256, 64, False, True)
    args, _, n = setup(case, 4)
    want = call(args, n)
    args[0][3, 17], args[0][9, 200] = float("inf"), float("nan")
    got = call(args, n)
    keep = [i for i in range(17) if i not in (3, 9)]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[9]).all() and not torch.isfinite(got[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("wrong", ["expert", "low", "high", "order"])
def test_bad_segments_are_reported_and_skipped(wrong):
    m = moe()
    case = ((4, 3, 20), 0, 3, 40, 128, 128, False, False)
    args, _, n = setup(case, 5)
    want = call(args, n)
    ws = m.new_workspace(n, 1, 3)
    off, exp = args[1].clone(), args[2].clone()
    skipped = slice(4, 7)
    if wrong == "expert":
        exp[1] = 3
    elif wrong == "low":
        off[0], skipped = -1, slice(0, 4)
    elif wrong == "high":
        off[3], skipped = n + 1, slice(7, 27)
    else:
        off[1], skipped = 9, slice(0, 27)
    got = call([args[0], off, exp, args[3]], n, ws=ws)
    with pytest.raises(m.MoeError) as e:
        m.moe_check_device_status(ws)
    assert e.value.status == 4
    assert (got[skipped] == 7.0).all()
    if wrong != "order":
        keep = torch.ones(n, dtype=torch.bool)
        keep[skipped] = False
        assert torch.equal(got[keep], want[keep])


@pytest.mark.gpu
def test_no_rows_another_stream_and_a_replayed_graph():
    m = moe()
    case = ((2, 0, 5), 0, 3, 48, 256, 32, True, True)
    args, _, n = setup(case, 6)
    want = call(args, n)
    assert call([args[0][:0], torch.zeros_like(args[1]), args[2], args[3]], 0).shape == (0, 24)
    zero = call([args[0], torch.full_like(args[1], 4), args[2], args[3]], n)
    assert (zero == 7.0).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(args, n, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws, out = m.new_workspace(n, 1, 3), torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_grouped_product_int4(*args, out, ws, torch.cuda.current_stream())
    for _ in range(3):
        out.fill_(7.0)
        g.replay()
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_weights_and_rows_past_32_bits():
    """Packed weights more than 4 GiB into their planes, rows more than 4 GiB into x."""
    m = moe()
    E, N, K, n = 9, 16384, 65536, 40000
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    codes = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(E, N, K // 128, dtype=torch.bfloat16, device="cuda")
    codes[8] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda").to(torch.uint8)
    scales[8] = 2.0 ** -4
    w = m.pack_weights_int4(codes, scales, None, m.MOE_EPI_NONE)
    alone = m.pack_weights_int4(codes[8:].contiguous(), scales[8:].contiguous(), None, m.MOE_EPI_NONE)
    del codes, scales
    assert w.data.numel() > 4.5 * 2 ** 30
    x = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, generator=gen, device="cuda").bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    want = call([x[-3:].contiguous(), i32(0, 3), i32(0), alone], 3)
    ws = m.new_workspace(n, 1, 1)
    out = torch.empty(n, N, device="cuda")
    m.moe_grouped_product_int4(x, i32(n - 3, n), i32(8), w, out, ws)
    m.moe_check_device_status(ws)
    assert torch.equal(out[-3:], want)
