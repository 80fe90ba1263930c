"""Rows in microscaled FP4 and the weight layout of the grouped product,
against a 64-bit implementation of the definition in moe.h.

Codes, scales and restored values are those of real arithmetic, so everything
here is compared exactly (the sign of a zero aside).
"""

import ctypes

import numpy as np
import pytest
import torch

MX, NV = 0, 1
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


# ------------------------------------------------------------------ 64-bit definition
E4M3 = np.array([(c % 8) * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])


def nearest_even(v, grid):
    """Index of the grid value nearest to v >= 0, halves to the even index."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    d0, d1 = v - grid[lo], grid[hi] - v
    return np.where((d1 < d0) | ((d1 == d0) & (hi % 2 == 0)), hi, lo)


def reference(x, fmt, exp):
    """codes 0..15 [n, K], scale bytes [n, K/block], values [n, K] (64 bits)."""
    blk = 32 if fmt == MX else 16
    b = x.astype(np.float64).reshape(x.shape[0], -1, blk)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0, b)
    amax = np.abs(b).max(2)
    if fmt == MX:
        m, q = np.frexp(amax)                   # amax = m 2^q, m in [0.5, 1); 6 = 0.75 * 2^3
        e = np.where(amax == 0, -127, np.clip(q - 3 + (m > 0.75), -127, 127))
        byte, unit = e + 127, 2.0 ** e
    else:
        byte = nearest_even(amax / 2.0 ** exp / 6, E4M3)
        unit = E4M3[byte] * 2.0 ** exp
    safe = np.where(unit > 0, unit, 1)
    y = np.where(unit[:, :, None] > 0, np.abs(b) / safe[:, :, None], 0)
    idx = nearest_even(y, GRID)
    val = np.sign(b) * GRID[idx] * unit[:, :, None]
    val[bad] = np.nan
    byte = np.where(bad, 255 if fmt == MX else 127, byte)
    code = idx + 8 * (b < 0)
    return code.reshape(x.shape), byte.astype(np.uint8), val.reshape(x.shape)


def unpack(codes):
    c = codes.cpu().numpy()
    return np.stack((c % 16, c // 16), -1).reshape(c.shape[0], -1)


def same_codes(got, ref):
    zero = lambda c: np.where(c % 8 == 0, 0, c)
    return np.array_equal(zero(got), zero(ref))


# ------------------------------------------------------------------ CPU: refusals
FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
ODD = ctypes.c_void_p(0x10008)


def test_refusals():
    L = moe().lib()
    q = lambda x=FAKE, t=1, ld=64, n=4, K=64, f=0, e=0, c=FAKE, s=FAKE: \
        L.moe_quantize_fp4(x, t, ld, n, K, f, e, c, s, None)
    assert q(n=0) == 0
    assert all(v == 1 for v in (q(x=None), q(c=None), q(s=None), q(t=2), q(ld=63), q(n=-1), q(K=0), q(f=2),
                                q(e=1), q(x=ODD), q(c=ODD), q(s=ODD), q(ld=68), q(t=0, ld=65)))
    assert q(K=48) == 2 and q(f=1, e=101) == 2 and q(f=1, e=-101) == 2 and q(K=2 ** 25, ld=2 ** 25) == 2
    p = lambda x=FAKE, T=4, K=64, k=2, d=FAKE, n=8, f=0, e=0, c=FAKE, s=FAKE, ws=FAKE, b=256: \
        L.moe_permute_fp4(x, T, K, k, d, n, f, e, c, s, ws, b, None)
    assert p(T=0) == 0
    assert all(v == 1 for v in (p(x=None), p(d=None), p(c=None), p(s=None), p(k=0), p(n=-1), p(T=-1), p(f=7),
                                p(x=ODD), p(c=ODD)))
    assert p(K=40) == 2 and p(ws=None) == 6 and p(b=8) == 6 and p(ws=ODD) == 6
    d = lambda c=FAKE, s=FAKE, n=4, K=64, f=0, e=0, o=FAKE, t=1: L.moe_dequant_fp4(c, s, n, K, f, e, o, t, None)
    assert d(n=0) == 0
    assert all(v == 1 for v in (d(c=None), d(s=None), d(o=None), d(t=5), d(f=-1), d(o=ODD), d(e=3)))
    assert d(K=31) == 2
    w = lambda c=FAKE, s=FAKE, E=1, N=16, K=64, f=0, ep=0, o=ctypes.c_void_p(0x20000): \
        L.moe_pack_weights_fp4(c, s, E, N, K, f, ep, o, None)
    assert all(v == 1 for v in (w(c=None), w(s=None), w(o=None), w(E=0), w(N=0), w(K=0), w(f=2), w(ep=2),
                                w(o=FAKE), w(c=ODD)))
    assert w(N=12) == 2 and w(N=24, ep=1) == 2 and w(K=16) == 2


def test_sizes():
    L = moe().lib()
    assert [L.moe_fp4_scale_ld(K, f) for K, f in ((32, 0), (256, 0), (288, 0), (7168, 1), (1440, 1))] == \
        [8, 8, 16, 448, 96]
    assert L.moe_fp4_scale_ld(33, 0) == 0 and L.moe_fp4_scale_ld(64, 2) == 0 and L.moe_fp4_scale_ld(0, 0) == 0
    assert L.moe_fp4_packed_bytes(2, 256, 512, NV, 0) == 2 * 2 * 36864
    assert L.moe_fp4_packed_bytes(3, 264, 32, MX, 0) == 3 * 2 * 34816
    assert L.moe_fp4_packed_bytes(1, 272, 256, MX, 1) == 2 * 34816
    assert L.moe_fp4_packed_bytes(0, 256, 512, NV, 0) == 0 and L.moe_fp4_packed_bytes(1, 256, 512, NV, 2) == 0


# ------------------------------------------------------------------ GPU
def rows(n, K, seed, dtype):
    """Rows whose blocks reach from the smallest floats to the largest, with
    zero blocks, exact borders between codes and their neighbours."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, K)).astype(np.float32)
    x *= np.exp2(rng.integers(-6, 7, (n, K // 16)).astype(np.float32)).repeat(16, 1)
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32)
    for r in range(0, n, 3):            # a block whose largest value is 6 * m: quotients on borders
        for b in range(0, K // 32, 2):
            m = np.float32(rng.integers(8, 16) * 2.0 ** rng.integers(-9, 3))
            v = rng.choice(mid, 32) * m * rng.choice([-1, 1], 32)
            v[rng.integers(0, 16)] = 6 * m
            v[rng.integers(16, 32)] = -6 * m
            x[r, 32 * b:32 * b + 32] = v
    if dtype == torch.float32:          # one step beside the borders
        step = rng.integers(-1, 2, x.shape)
        x = np.where(step > 0, np.nextafter(x, np.float32(np.inf)),
                     np.where(step < 0, np.nextafter(x, np.float32(-np.inf)), x))
    x[0, :32] = 0
    if n > 4:
        x[1] *= np.float32(2.0 ** -130)
        x[2] *= np.float32(2.0 ** 115)
        x[3, :16] = 0
        x[4, 0] = np.finfo(np.float32).max
    t = torch.from_numpy(x).to(dtype)
    if n > 4 and dtype == torch.bfloat16:
        t[4, 0] = torch.finfo(torch.bfloat16).max
    return t, t.float().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,exp", [(MX, 0), (NV, 0), (NV, -8), (NV, 100), (NV, -100)])
@pytest.mark.parametrize("n,K", [(1, 32), (7, 96), (33, 256), (19, 1440), (5, 7168)])
def test_quantize_and_back(n, K, fmt, exp, dtype):
    m = moe()
    t, x = rows(n, K, n + K, dtype)
    codes, sf = m.new_fp4(n, K, fmt)
    codes.fill_(0xAB), sf.fill_(0xCD)
    wide = torch.zeros(n, K + 16, dtype=dtype, device="cuda")   # rows further apart than their length
    wide[:, :K] = t
    m.moe_quantize_fp4(wide[:, :K], fmt, exp, codes, sf)
    rc, rs, rv = reference(x, fmt, exp)
    s = sf.cpu().numpy()
    assert np.array_equal(s[:, :rs.shape[1]], rs) and (s[:, rs.shape[1]:] == 0).all()
    assert same_codes(unpack(codes), rc)
    for out_t in (torch.float32, torch.bfloat16):
        out = torch.full((n, K), 7.0, dtype=out_t, device="cuda")
        m.moe_dequant_fp4(codes, sf, fmt, exp, out)
        exact = torch.from_numpy(rv).float().to(out_t)
        assert torch.equal(out.cpu() + 0.0, exact + 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nonfinite_blocks(fmt, dtype):
    m = moe()
    t = torch.randn(6, 128).to(dtype)
    t[0, 5], t[1, 40], t[2, 127], t[3] = float("nan"), float("inf"), -float("inf"), float("nan")
    codes, sf = m.new_fp4(6, 128, fmt)
    m.moe_quantize_fp4(t.cuda(), fmt, 0, codes, sf)
    rc, rs, rv = reference(t.float().numpy(), fmt, 0)
    assert np.array_equal(sf.cpu().numpy()[:, :rs.shape[1]], rs)
    assert same_codes(unpack(codes), np.where(np.isnan(rv), 0, rc))
    out = torch.empty(6, 128, device="cuda")
    m.moe_dequant_fp4(codes, sf, fmt, 0, out)
    assert np.array_equal(out.cpu().numpy() + 0.0, rv.astype(np.float32) + 0.0, equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [MX, NV])
def test_every_code_and_scale(fmt):
    """Restoring codes that this library did not write: all 16 codes under every scale byte."""
    m = moe()
    blk = 32 if fmt == MX else 16
    codes, sf = m.new_fp4(256, 32, fmt)
    c = np.tile(np.arange(16), 2)
    codes[:] = torch.from_numpy((c[0::2] + 16 * c[1::2]).astype(np.uint8)).cuda()
    sf[:] = torch.arange(256, dtype=torch.uint8).cuda()[:, None]
    out = torch.empty(256, 32, device="cuda")
    m.moe_dequant_fp4(codes, sf, fmt, 0, out)
    if fmt == MX:
        scale = np.where(np.arange(256) == 255, np.nan, 2.0 ** (np.arange(256) - 127.0))
    else:
        scale = np.array([(-1.0 if b > 127 else 1.0) * (np.nan if b % 128 == 127 else E4M3[b % 128])
                          for b in range(256)])
    signed = np.concatenate((GRID, -GRID))
    with np.errstate(over="ignore"):
        ref = (signed[c][None, :] * scale[:, None]).astype(np.float32)
    assert np.array_equal(out.cpu().numpy() + 0.0, ref + 0.0, equal_nan=True) and blk


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,exp", [(MX, 0), (NV, -5)])
@pytest.mark.parametrize("T,K,k", [(1, 32, 1), (5, 1440, 3), (64, 256, 8), (130, 96, 2)])
def test_permute(T, K, k, fmt, exp):
    m = moe()
    t, x = rows(T, K, 3 * T + K, torch.bfloat16)
    n = T * k + 3
    rng = np.random.default_rng(T)
    dest = rng.permutation(n)[:T * k].astype(np.int32)
    dest[0] = -1
    codes, sf = m.new_fp4(n, K, fmt)
    codes.fill_(0x5A), sf.fill_(0x5A)
    ws = m.new_workspace(T, k, 1)
    m.moe_permute_fp4(t.cuda(), k, torch.from_numpy(dest).cuda(), fmt, exp, codes, sf, ws)
    m.moe_check_device_status(ws)
    rc, rs, _ = reference(x, fmt, exp)
    gc, gs = unpack(codes), sf.cpu().numpy()
    hit = np.zeros(n, bool)
    for a, d in enumerate(dest):
        if d >= 0:
            hit[d] = True
            assert same_codes(gc[d], rc[a // k]) and np.array_equal(gs[d, :rs.shape[1]], rs[a // k])
            assert (gs[d, rs.shape[1]:] == 0).all()
    assert (codes.cpu().numpy()[~hit] == 0x5A).all() and (gs[~hit] == 0x5A).all()
    # a row out of range is reported and skipped
    dest[-1] = n
    m.moe_permute_fp4(t.cuda(), k, torch.from_numpy(dest).cuda(), fmt, exp, codes, sf, ws)
    with pytest.raises(m.MoeError) as e:
        m.moe_check_device_status(ws)
    assert e.value.status == 4 and e.value.info == T * k - 1


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("E,N,K,epi", [(1, 8, 32, 0), (2, 264, 288, 0), (3, 272, 1440, 1), (1, 512, 256, 1)])
def test_pack_layout(E, N, K, epi, fmt):
    m = moe()
    rng = np.random.default_rng(N + K)
    ld = m.moe_fp4_scale_ld(K, fmt)
    codes = rng.integers(0, 256, (E, N, K // 2)).astype(np.uint8)
    sf = rng.integers(1, 120, (E, N, ld)).astype(np.uint8)
    w = m.pack_weights_fp4(torch.from_numpy(codes).cuda(), torch.from_numpy(sf).cuda(), fmt, epi)
    sb, blk = (16, 16) if fmt == NV else (8, 32)
    nkb = -(-K // 256)
    nbn = -(-(N // 2) // 128) if epi else -(-N // 256)
    got = w.data.cpu().numpy().reshape(E, nbn, nkb, 32768 + 256 * sb)
    assert (w.E, w.N, w.K, w.fmt, w.epilogue) == (E, N, K, fmt, epi)
    full_c = np.zeros((E, 2 * nbn * 128, nkb * 128), np.uint8)   # rows in tile order, halves one after the other
    full_s = np.zeros((E, 2 * nbn * 128, nkb * sb), np.uint8)
    for nb in range(nbn):
        for h in range(2):
            for r in range(128):
                f = (h * (N // 2) + nb * 128 + r) if epi else nb * 256 + h * 128 + r
                ok = nb * 128 + r < N // 2 if epi else f < N
                if ok:
                    full_c[:, (nb * 2 + h) * 128 + r, :K // 2] = codes[:, f]
                    full_s[:, (nb * 2 + h) * 128 + r, :K // blk] = sf[:, f, :K // blk]
    c = got[..., :32768].reshape(E, nbn, nkb, 2, 128, 8, 16)
    un = np.empty_like(c)
    for r in range(128):
        for j in range(8):
            un[..., r, j, :] = c[..., r, j ^ (r % 8), :]
    un = un.reshape(E, nbn, nkb, 2, 128, 128).transpose(0, 1, 3, 4, 2, 5).reshape(full_c.shape)
    assert np.array_equal(un, full_c)
    s = got[..., 32768:].reshape(E, nbn, nkb, 2, sb // 4, 32, 4, 4)      # half, group, r % 32, r / 32, byte
    s = s.transpose(0, 1, 3, 6, 5, 2, 4, 7).reshape(full_s.shape)
    assert np.array_equal(s, full_s)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Codes, rows and logits more than 4 GiB into their buffers."""
    m = moe()
    n, K = 1_100_000, 8192                              # 18 GB of rows, 4.5 GB of codes
    x = torch.zeros(n, K, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, K, device="cuda").bfloat16()
    x[-5:] = tail
    codes, sf = m.new_fp4(n, K, NV)
    m.moe_quantize_fp4(x, NV, -4, codes, sf)
    rc, rs, rv = reference(tail.float().cpu().numpy(), NV, -4)
    assert same_codes(unpack(codes[-5:]), rc) and np.array_equal(sf[-5:].cpu().numpy()[:, :rs.shape[1]], rs)
    x.fill_(1)
    m.moe_dequant_fp4(codes, sf, NV, -4, x)
    assert torch.equal(x[-5:].float().cpu() + 0.0, torch.from_numpy(rv).float() + 0.0) and not x[:-5].any()
    del x, sf
    # dispatched rows beyond 4 GiB of codes
    sf = torch.zeros(n, m.moe_fp4_scale_ld(K, MX), dtype=torch.uint8, device="cuda")
    ws = m.new_workspace(5, 1, 1)
    dest = torch.arange(n - 5, n, dtype=torch.int32, device="cuda").flip(0).contiguous()
    m.moe_permute_fp4(tail, 1, dest, MX, 0, codes, sf, ws)
    m.moe_check_device_status(ws)
    rc, rs, _ = reference(tail.float().cpu().numpy(), MX, 0)
    assert same_codes(unpack(codes[-5:].flip(0)), rc)
