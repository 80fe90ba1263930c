"""The block around the experts: norms before and after them with gate and
residual, and the gradients, against the definitions of moe.h in 64 bits.

Tolerances.  With u = 2^-24 (half an fp32 step) a sum of n terms in fp32 is
within d u of the terms' magnitudes, d the longest chain of additions that one
term goes through: at most 32 in a thread, 10 across warp and CTA, and 16 for
the fma chain over experts, so 64 covers each sum here.  Operations outside the
sums add a few u each, 16 in all.  ``Block`` carries these bounds through the
formulas: dx is the bound of an error of x, A_x the sum of the magnitudes of
the terms of x.  Results held in bf16 add half a step, 2^-8 of the value.
"""

import ctypes

import numpy as np
import pytest
import torch

U = 2.0 ** -24
SUM = 64 * U
OPS = 16 * U
BF16 = 2.0 ** -8
EPS = 1e-6

F32, BF = torch.float32, torch.bfloat16
FAKE = ctypes.c_void_p(0x10000)   # never dereferenced
ODD = ctypes.c_void_p(0x10008)


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


# ------------------------------------------------------------------ refusals
def test_refusals():
    m = moe()
    L = m.lib()
    cfg = lambda post=1, eps=EPS, scale=1.0: ctypes.byref(m.BlockCfg(post, eps, scale))
    nan = float("nan")

    def norm(x=FAKE, t=0, T=4, H=64, w=None, eps=EPS, o=FAKE):
        return L.moe_norm(x, t, T, H, w, eps, o, None)

    def comb(yp=FAKE, n=8, d=FAKE, w=FAKE, T=4, k=2, H=64, sh=None, res=FAKE, t=0, wt=None, c=None, y=FAKE, nw=None,
             no=None, ws=FAKE, b=256):
        return L.moe_combine_norm(yp, n, d, w, T, k, H, sh, res, t, wt, None, c or cfg(), y, nw, no, ws, b, None)

    def cbwd(gy=FAKE, t=0, yp=FAKE, n=8, d=FAKE, w=FAKE, T=4, k=2, H=64, gyp=FAKE, gw=FAKE, ws=FAKE, b=256):
        return L.moe_combine_backward(gy, t, yp, n, d, w, T, k, H, gyp, gw, ws, b, None)

    def nbwd(gy=FAKE, t=0, yp=FAKE, n=8, d=FAKE, w=FAKE, T=4, k=2, H=64, sh=None, wt=None, c=None, gyp=FAKE, gw=FAKE,
             gs=None, gwt=None, sc=None, sb=0, ws=FAKE, b=256):
        return L.moe_combine_norm_backward(gy, t, yp, n, d, w, T, k, H, sh, wt, None, c or cfg(), gyp, gw, gs, gwt,
                                           None, sc, sb, ws, b, None)

    def xbwd(g=FAKE, n=8, d=FAKE, k=2, add=None, x=FAKE, t=0, T=4, H=64, w=None, eps=EPS, rg=None, s=1.0, gx=FAKE,
             gw=None, sc=None, sb=0, ws=FAKE, b=256):
        return L.moe_norm_backward(g, n, d, k, add, x, t, T, H, w, eps, rg, s, gx, gw, sc, sb, ws, b, None)

    def pbwd(g=FAKE, n=8, d=FAKE, add=None, T=4, k=2, H=64, gx=FAKE, t=0, ws=FAKE, b=256):
        return L.moe_permute_backward(g, n, d, add, T, k, H, gx, t, ws, b, None)

    assert all(f(T=0) == 0 for f in (norm, comb, cbwd, nbwd, xbwd, pbwd))
    for f in (norm, comb, cbwd, nbwd, xbwd, pbwd):
        assert f(T=-1) == 1 and f(H=0) == 1 and f(t=2) == 1 and f(t=-1) == 1
        assert f(H=12) == 2 and f(H=16392) == 2
    for f in (comb, cbwd, nbwd, xbwd, pbwd):
        assert f(k=0) == 1 and f(n=-1) == 1 and f(k=17) == 2 and f(n=2 ** 31) == 2 and f(T=2 ** 30, k=2) == 2
        assert f(ws=None) == 6 and f(ws=ODD) == 6 and f(b=64) == 6
    assert norm(T=2 ** 31) == 2
    bad = [norm(x=None), norm(o=None), norm(x=ODD), norm(o=ODD), norm(w=ODD), norm(eps=0.0), norm(eps=-1.0),
           norm(eps=nan), norm(eps=float("inf"))]
    bad += [comb(yp=None), comb(d=None), comb(w=None), comb(res=None), comb(y=None), comb(yp=ODD), comb(sh=ODD),
            comb(res=ODD), comb(wt=ODD), comb(y=ODD), comb(no=FAKE, nw=ODD), comb(no=ODD), comb(nw=FAKE),
            comb(c=cfg(post=2)), comb(c=cfg(eps=0.0)), comb(c=cfg(scale=nan)), comb(c=cfg(post=0), wt=FAKE),
            L.moe_combine_norm(FAKE, 8, FAKE, FAKE, 4, 2, 64, None, FAKE, 0, None, None, None, FAKE, None, None, FAKE,
                               256, None)]
    bad += [cbwd(gy=None), cbwd(yp=None), cbwd(d=None), cbwd(w=None), cbwd(gyp=None), cbwd(gw=None), cbwd(gy=ODD),
            cbwd(yp=ODD), cbwd(gyp=ODD)]
    bad += [nbwd(gy=None), nbwd(yp=None), nbwd(d=None), nbwd(w=None), nbwd(gyp=None), nbwd(gw=None), nbwd(gy=ODD),
            nbwd(sh=ODD), nbwd(wt=ODD), nbwd(gs=ODD), nbwd(gwt=ODD), nbwd(c=cfg(post=0), wt=FAKE),
            nbwd(c=cfg(post=0), gwt=FAKE), nbwd(c=cfg(eps=nan))]
    bad += [xbwd(g=None), xbwd(x=None), xbwd(gx=None), xbwd(g=ODD), xbwd(add=ODD), xbwd(x=ODD), xbwd(w=ODD),
            xbwd(rg=ODD), xbwd(gx=ODD), xbwd(gw=ODD), xbwd(eps=0.0), xbwd(s=nan), xbwd(d=None)]
    bad += [pbwd(g=None), pbwd(d=None), pbwd(gx=None), pbwd(g=ODD), pbwd(add=ODD), pbwd(gx=ODD)]
    assert all(v == 1 for v in bad), bad
    # the gradient of a norm's weight needs scratch
    assert nbwd(gwt=FAKE) == 6 and nbwd(gwt=FAKE, sc=ODD, sb=1 << 40) == 6 and nbwd(gwt=FAKE, sc=FAKE, sb=16) == 6
    assert xbwd(gw=FAKE) == 6 and xbwd(gw=FAKE, sc=ODD, sb=1 << 40) == 6 and xbwd(gw=FAKE, sc=FAKE, sb=16) == 6
    assert L.moe_norm_scratch_bytes(0, 64) == 0 and L.moe_norm_scratch_bytes(4, 12) == 0
    assert L.moe_norm_scratch_bytes(4, 16392) == 0


def test_binding_refusals():
    m = moe()
    z = lambda *s, t=BF: torch.zeros(*s, dtype=t)
    ws = z(256, t=torch.uint8)
    with pytest.raises(TypeError):
        m.moe_norm(z(2, 8), None, EPS, z(2, 8))
    with pytest.raises(TypeError):
        m.moe_norm(z(2, 8, t=torch.float16), None, EPS, z(2, 8))
    with pytest.raises(TypeError):
        m.moe_combine_norm(z(4, 8), z(2, 2, t=torch.int32), z(2, 2, t=F32), z(2, 8), m.BlockCfg(), z(2, 8), ws)
    with pytest.raises(TypeError):
        m.moe_combine_backward(z(2, 8), z(4, 8), z(2, 2, t=torch.int32), z(2, 2, t=F32), z(4, 8), z(2, 2, t=F32), ws)
    with pytest.raises(TypeError):
        m.moe_permute_backward(z(4, 8), z(2, 2, t=torch.int32), z(2, 8), ws)
    with pytest.raises(TypeError):
        m.moe_norm_backward(z(2, 8), z(2, 8), None, EPS, z(2, 8), None, ws)


# ------------------------------------------------------------------ 64 bits
def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rms(c):
    return 1 / np.sqrt((c * c).mean(1, keepdims=True) + EPS)


class Norm:
    """1 / rms of rows and the gradient through them, with error bounds."""

    def __init__(self, c, dc=0.0):
        self.c, self.dc = c, dc + 0 * c
        self.r = rms(c)
        # r moves with the length of the error, over the length of the row with eps in it
        self.dr = self.r * (SUM + OPS + np.sqrt((self.dc ** 2).mean(1, keepdims=True)) * self.r)

    def out(self, w):
        y = self.c * self.r * w
        return y, np.abs(w) * (self.dc * self.r + np.abs(self.c) * self.dr) + OPS * np.abs(y)

    def back(self, e, de):
        c, r, dr = self.c, self.r, self.dr
        s2, A = (e * c).mean(1, keepdims=True), np.abs(e * c).mean(1, keepdims=True)
        ds2 = SUM * A + (np.abs(e) * self.dc + de * np.abs(c)).mean(1, keepdims=True)
        m = r * r * s2
        dm = r * r * ds2 + 2 * dr * r * np.abs(s2) + OPS * np.abs(m)
        g = r * (e - c * m)
        mag = np.abs(e) + np.abs(c * m)
        dg = dr * mag + r * (de + self.dc * np.abs(m) + np.abs(c) * dm + OPS * mag)
        return g, dg, m


def take(rows, dest):
    out = np.zeros((*dest.shape, rows.shape[1]))
    out[dest >= 0] = rows[dest[dest >= 0]]
    return out


class Block:
    """moe_combine_norm and its gradient in 64 bits: value and bound of each output."""

    def __init__(self, s, T, H, post, scale):
        self.s, self.post, self.scale = s, post, scale
        self.dest = s["dest"].cpu().numpy()
        self.w = f64(s["w"])
        self.rows = take(f64(s["yp"]), self.dest)
        self.sh = f64(s["shared"])
        self.g = f64(s["gate"])[:, None] if s["gate"] is not None else np.ones((T, 1))
        self.wt = f64(s["weight"]) if s["weight"] is not None else np.ones(H)
        terms = self.w[..., None] * self.rows
        self.c = terms.sum(1) + (0 if self.sh is None else self.sh)
        mag = np.abs(terms).sum(1) + (0 if self.sh is None else np.abs(self.sh))
        self.dc = SUM * mag
        self.norm = Norm(self.c, self.dc)

    def forward(self):
        f, df = self.norm.out(self.wt) if self.post else (self.c, self.dc)
        x = self.scale * f64(self.s["x"])
        y = x + self.g * f
        return y, np.abs(self.g) * df + OPS * (np.abs(x) + np.abs(self.g * f))

    def backward(self):
        gy = f64(self.s["gy"])
        e = gy * self.wt
        de = OPS * np.abs(e)
        if self.post:
            d, dd, m = self.norm.back(e, de)
            mag = self.norm.r * (np.abs(e) + np.abs(self.c * m))
            f, df = self.norm.out(np.ones_like(self.wt))
        else:
            d, dd, mag, f, df = e, de, np.abs(e), self.c, self.dc
        out = {}
        dc, ddc = self.g * d, np.abs(self.g) * (dd + OPS * np.abs(d))
        out["shared"] = dc, ddc
        out["rows"] = self.w[..., None] * dc[:, None], (np.abs(self.w)[..., None] * (ddc + OPS * np.abs(dc))[:, None])
        a = np.abs(self.rows)
        err = (ddc[:, None] + SUM * (np.abs(self.g) * mag)[:, None]) * a
        out["w"] = (dc[:, None] * self.rows).sum(2), err.sum(2)
        T = gy.shape[0]
        t = self.g * gy * f
        out["weight"] = t.sum(0), (np.abs(self.g * gy) * df + (T * U + OPS) * np.abs(t)).sum(0)
        t = e * f
        out["gate"] = t.sum(1), (np.abs(e) * df + de * np.abs(f) + SUM * np.abs(t)).sum(1)
        return out


def near(got, want, err, name=""):
    half = BF16 if got.dtype == BF else U
    got = f64(got)
    tiny = 2.0 ** -133 if half == BF16 else 2.0 ** -149
    bad = ~(np.abs(got - want) <= err + half * (np.abs(want) + err) + tiny)
    assert not bad.any(), (name, int(bad.sum()), np.abs(got - want)[bad].max(), err[bad].max())


def inputs(T, H, k, dt, gate, shared, weight, drop, seed=0, rows=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    n = rows or T * k + 5
    dest = torch.randperm(n, generator=gen, device="cuda")[:T * k].to(torch.int32).view(T, k)
    if drop:
        dest = dest.masked_fill(torch.rand(T, k, generator=gen, device="cuda") < drop, -1)
    dest = dest.contiguous()
    scale = torch.exp(0.5 * rn(H))
    yp, grad = (rn(n, H) * scale).to(BF), rn(n, H).to(BF)
    # rows that nothing lands on are never read
    landed = torch.zeros(n, dtype=torch.bool, device="cuda")
    landed[dest[dest >= 0].long()] = True
    yp[~landed] = float("nan")
    grad[~landed] = float("nan")
    return dict(dest=dest, yp=yp, w=torch.rand(T, k, generator=gen, device="cuda") + 0.1,
                shared=rn(T, H).to(BF) if shared else None, x=(rn(T, H) * scale).to(dt), gy=rn(T, H).to(dt),
                gate=rn(T) if gate else None, weight=1 + 0.3 * rn(H) if weight else None, grad=grad,
                add=rn(T, H).to(BF), landed=landed, next_weight=1 + 0.3 * rn(H))


def forward(s, post, scale, next=True, y=None, stream=None):
    m = moe()
    T, H = s["x"].shape
    ws = m.new_workspace(T, s["w"].shape[1], 1, stream=stream)
    y = torch.empty_like(s["x"]) if y is None else y
    nx = torch.empty(T, H, dtype=BF, device="cuda") if next else None
    m.moe_combine_norm(s["yp"], s["dest"], s["w"], s["x"], m.BlockCfg(int(post), EPS, scale), y, ws,
                       shared=s["shared"], weight=s["weight"] if post else None, gate=s["gate"],
                       next_weight=s["next_weight"] if next else None, next_out=nx, stream=stream)
    return y, nx, ws


def backward(s, post, scale=1.0, stream=None):
    m = moe()
    T, H = s["x"].shape
    ws = m.new_workspace(T, s["w"].shape[1], 1, stream=stream)
    e = lambda *n, t=F32: torch.full(n, 7.0, dtype=t, device="cuda")
    out = dict(rows=torch.full_like(s["yp"], 7.0), w=e(*s["w"].shape), shared=e(T, H, t=BF), gate=e(T),
               weight=e(H) if post else None)
    sc = m.new_norm_scratch(T, H, stream=stream) if post else None
    m.moe_combine_norm_backward(s["gy"], s["yp"], s["dest"], s["w"], m.BlockCfg(int(post), EPS, scale), out["rows"],
                                out["w"], ws, sc, shared=s["shared"], weight=s["weight"] if post else None,
                                gate=s["gate"], grad_shared=out["shared"], grad_weight=out["weight"],
                                grad_gate=out["gate"], stream=stream)
    return out, ws


def norm_backward(s, direct, scale, residual=True, gx=None, stream=None):
    m = moe()
    T, H = s["x"].shape
    ws = m.new_workspace(T, s["w"].shape[1], 1, stream=stream)
    gx = torch.empty_like(s["x"]) if gx is None else gx
    gw = torch.empty(H, device="cuda")
    m.moe_norm_backward(s["add"] if direct else s["grad"], s["x"], s["weight"], EPS, gx, gw, ws,
                        m.new_norm_scratch(T, H, stream=stream), dest_row=None if direct else s["dest"],
                        add=None if direct else s["add"], residual_grad=s["gy"] if residual else None,
                        residual_scale=scale, stream=stream)
    return gx, gw, ws


CASES = [  # T, H, k, type, post, gate, shared, weight, drop, scale
    (1, 8, 1, BF, True, False, True, True, 0, 1.0),
    (1, 7168, 8, BF, False, False, True, False, 0, 1.0),
    (3, 264, 2, F32, True, True, False, True, 0, 0.5),
    (37, 1440, 6, BF, True, True, True, True, 0.3, 2.0),
    (64, 72, 16, F32, True, False, True, False, 0.6, -1.0),
    (5, 4104, 3, F32, False, True, False, False, 0.5, 1.0),
    (9, 8192, 4, BF, True, True, False, True, 0, 1.0),
    (7, 8200, 8, F32, True, True, True, True, 0.2, 0.25),
    (2, 16384, 16, BF, True, False, False, True, 0, 1.0),
    (700, 136, 5, BF, True, True, True, True, 0.1, 1.0),
    # rows of which half have a place in shared memory at a time, or one team instead of two
    (3, 8192, 16, F32, True, True, True, True, 0.2, 1.0),
    (5, 4096, 16, F32, True, False, True, True, 0.2, 1.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    T, H, k, dt, post, gate, shared, weight, drop, scale = case
    m = moe()
    s = inputs(T, H, k, dt, gate, shared, weight, drop)
    y, nx, ws = forward(s, post, scale)
    m.moe_check_device_status(ws)
    near(y, *Block(s if post else {**s, "weight": None}, T, H, post, scale).forward(), "y")
    near(nx, *Norm(f64(y)).out(f64(s["next_weight"])), "next")
    # the next block's norm is moe_norm of y, and y does not depend on it
    n2 = torch.empty_like(nx)
    m.moe_norm(y, s["next_weight"], EPS, n2)
    assert torch.equal(n2, nx)
    assert torch.equal(forward(s, post, scale, next=False)[0], y)
    n3 = torch.empty_like(nx)
    m.moe_norm(s["x"], None, EPS, n3)
    near(n3, *Norm(f64(s["x"])).out(np.ones(H)), "norm without weight")


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    T, H, k, dt, post, gate, shared, weight, drop, scale = case
    m = moe()
    s = inputs(T, H, k, dt, gate, shared, weight, drop, seed=1)
    out, ws = backward(s, post, scale)
    m.moe_check_device_status(ws)
    want = Block(s if post else {**s, "weight": None}, T, H, post, scale).backward()
    dest = s["dest"].cpu().numpy()
    live = dest >= 0
    rows = out["rows"][s["dest"][s["dest"] >= 0].long()]
    near(rows, want["rows"][0][live], want["rows"][1][live], "rows")
    assert (out["rows"][~s["landed"]] == 7.0).all()
    assert (out["w"][s["dest"] < 0] == 0).all()
    near(out["w"], *want["w"], "w")
    near(out["shared"], *want["shared"], "shared")
    near(out["gate"], *want["gate"], "gate")
    if post:
        near(out["weight"], *want["weight"], "weight")
    again, _ = backward(s, post, scale)
    assert all(a is None or torch.equal(a, again[n]) for n, a in out.items())


@pytest.mark.gpu
@pytest.mark.parametrize("direct", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_norm_backward(case, direct):
    T, H, k, dt, _, _, _, weight, drop, scale = case
    m = moe()
    s = inputs(T, H, k, dt, False, False, weight, drop, seed=2)
    gx, gw, ws = norm_backward(s, direct, scale)
    m.moe_check_device_status(ws)
    terms = take(f64(s["grad"]), s["dest"].cpu().numpy())
    u, mag = f64(s["add"]), np.abs(f64(s["add"]))
    if not direct:
        u, mag = u + terms.sum(1), mag + np.abs(terms).sum(1)
    du = SUM * mag
    wt = f64(s["weight"]) if weight else np.ones(H)
    n = Norm(f64(s["x"]))
    d, dd, _ = n.back(u * wt, np.abs(wt) * du + OPS * np.abs(u * wt))
    r = scale * f64(s["gy"])
    near(gx, r + d, dd + OPS * (np.abs(r) + np.abs(d)), "x")
    hat, dhat = n.out(np.ones(H))
    near(gw, (u * hat).sum(0), (du * np.abs(hat) + np.abs(u) * dhat + (T * U + OPS) * np.abs(u * hat)).sum(0), "weight")
    gx2, gw2, _ = norm_backward(s, direct, scale)
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_sort_backward(case):
    T, H, k, dt, _, _, _, _, drop, _ = case
    m = moe()
    s = inputs(T, H, k, dt, False, False, False, drop, seed=3)
    ws = m.new_workspace(T, k, 1)
    rows, gw, gx = torch.full_like(s["yp"], 7.0), torch.empty_like(s["w"]), torch.empty_like(s["x"])
    m.moe_combine_backward(s["gy"], s["yp"], s["dest"], s["w"], rows, gw, ws)
    m.moe_permute_backward(s["grad"], s["dest"], gx, ws, add=s["add"])
    m.moe_check_device_status(ws)
    b = Block({**s, "weight": None}, T, H, False, 1.0).backward()
    live = s["dest"].cpu().numpy() >= 0
    near(rows[s["dest"][s["dest"] >= 0].long()], b["rows"][0][live], b["rows"][1][live], "rows")
    assert (rows[~s["landed"]] == 7.0).all() and (gw[s["dest"] < 0] == 0).all()
    near(gw, *b["w"], "w")
    terms = take(f64(s["grad"]), s["dest"].cpu().numpy())
    mag = np.abs(terms).sum(1) + np.abs(f64(s["add"]))
    near(gx, terms.sum(1) + f64(s["add"]), SUM * mag, "x")
    m.moe_permute_backward(s["grad"], s["dest"], gx, ws)
    near(gx, terms.sum(1), SUM * np.abs(terms).sum(1), "x without add")


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of the 64-bit forward along random directions: a
    difference over 2h is off by h^2/6 of the third derivative, far below the
    gradients' own rounding at h = 1e-4."""
    T, H, k = 4, 24, 3
    s = inputs(T, H, k, F32, True, True, True, 0, seed=4)
    out, _ = backward(s, True, 0.5)
    gx, gpre, _ = norm_backward(s, False, 0.5)
    rng = np.random.default_rng(0)
    gy = f64(s["gy"])

    def after(q):
        c = (q["w"][..., None] * take(q["rows"], s["dest"].cpu().numpy())).sum(1) + q["shared"]
        return (gy * (q["gate"][:, None] * c * rms(c) * q["weight"])).sum()

    base = dict(w=f64(s["w"]), rows=np.nan_to_num(f64(s["yp"])), shared=f64(s["shared"]), gate=f64(s["gate"]),
                weight=f64(s["weight"]))
    for name, v in base.items():
        d = rng.standard_normal(v.shape)
        if name == "rows":
            d[~s["landed"].cpu().numpy()] = 0
        h = 1e-4
        num = (after({**base, name: v + h * d}) - after({**base, name: v - h * d})) / (2 * h)
        got = f64(out[name])
        if name == "rows":
            got[~s["landed"].cpu().numpy()] = 0
        assert abs(num - (got * d).sum()) <= 2 * BF16 * np.abs(got * d).sum() + 1e-5, name
    u = take(f64(s["grad"]), s["dest"].cpu().numpy()).sum(1) + f64(s["add"])
    before = lambda x, w: (u * (x * rms(x) * w)).sum() + 0.5 * (gy * x).sum()
    x, w = f64(s["x"]), f64(s["weight"])
    d, h = rng.standard_normal(x.shape), 1e-4
    num = (before(x + h * d, w) - before(x - h * d, w)) / (2 * h)
    assert abs(num - (f64(gx) * d).sum()) <= 1e-4 * np.abs(f64(gx) * d).sum()
    d = rng.standard_normal(H)
    num = (before(x, w + h * d) - before(x, w - h * d)) / (2 * h)
    assert abs(num - (f64(gpre) * d).sum()) <= 1e-4 * np.abs(f64(gpre) * d).sum()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_of_any_size(dt):
    """Rows whose squares pass fp32's range are normalised all the same (2^70 is
    exact, so the bounds hold), rows of zeros stay zero, and an infinity or NaN
    stays in its row."""
    m = moe()
    T, H, k = 6, 520, 2
    s = inputs(T, H, k, dt, False, True, True, 0, seed=5)
    s["x"][0] *= 1e25
    s["x"][1] = s["x"][1].float().clamp(-1, 1).to(dt) * 3e38
    s["x"][2] = 0
    clean = s["x"].clone()
    s["x"][4, 3], s["x"][5, 7] = float("inf"), float("nan")
    out = torch.empty(T, H, dtype=BF, device="cuda")
    m.moe_norm(s["x"], s["weight"], EPS, out)
    near(out[:4], *Norm(f64(clean[:4])).out(f64(s["weight"])), "norm")
    assert torch.isnan(out[4, 3]) and torch.isnan(out[5]).all() and torch.isfinite(out[4, :3]).all()
    gx, gw, _ = norm_backward({**s, "x": clean}, False, 1.0, residual=False)
    u = take(f64(s["grad"]), s["dest"].cpu().numpy()).sum(1) + f64(s["add"])
    du = SUM * (np.abs(take(f64(s["grad"]), s["dest"].cpu().numpy())).sum(1) + np.abs(f64(s["add"])))
    wt = f64(s["weight"])
    n = Norm(f64(clean))
    d, dd, _ = n.back(u * wt, np.abs(wt) * du + OPS * np.abs(u * wt))
    # the gradient of a huge row lies among fp32's smallest numbers: half a step of those too
    near(gx, d, dd + 2.0 ** -130, "x")
    # after the experts
    r0 = s["dest"][0].long()
    s["yp"][r0] = (s["yp"][r0].float() * 1e25).to(BF)
    s["shared"][0] = 0
    s["shared"][3] = 0
    s["dest"][3] = -1                    # nothing arrives and nothing is shared: c = 0
    s["x"] = inputs(T, H, k, dt, False, True, True, 0, seed=5)["x"]
    y, nx, _ = forward(s, True, 1.0)
    near(y, *Block(s, T, H, True, 1.0).forward(), "y")
    got, _ = backward(s, True)
    want = Block(s, T, H, True, 1.0).backward()
    live = s["dest"].cpu().numpy() >= 0
    near(got["rows"][s["dest"][s["dest"] >= 0].long()], want["rows"][0][live], want["rows"][1][live] + 2.0 ** -130)
    near(got["w"], *want["w"], "w")
    near(got["shared"], want["shared"][0], want["shared"][1] + 2.0 ** -130, "shared")
    near(got["weight"], *want["weight"], "weight")
    s["yp"][s["dest"][1, 0].long(), 5] = float("nan")
    y2, _, _ = forward(s, True, 1.0)
    assert torch.isnan(y2[1]).all() and torch.equal(y2[[0, 2, 3, 4, 5]], y[[0, 2, 3, 4, 5]])


@pytest.mark.gpu
def test_in_place():
    s = inputs(9, 264, 3, BF, True, True, True, 0, seed=6)
    y, nx, _ = forward(s, True, 0.5)
    t = {**s, "x": s["x"].clone()}
    y2, nx2, _ = forward(t, True, 0.5, y=t["x"])
    assert torch.equal(y, y2) and torch.equal(nx, nx2)
    gx, gw, _ = norm_backward(s, False, 0.5)
    t = {**s, "gy": s["gy"].clone()}
    gx2, gw2, _ = norm_backward(t, False, 0.5, gx=t["gy"])
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)
    n = torch.empty_like(s["x"])
    m = moe()
    m.moe_norm(s["x"], s["weight"], EPS, n)
    m.moe_norm(s["x"], s["weight"], EPS, s["x"])
    assert torch.equal(n, s["x"])


@pytest.mark.gpu
def test_no_tokens_and_no_gradient_of_the_weight():
    m = moe()
    s = inputs(3, 64, 2, BF, False, False, True, 0, seed=7)
    ws = m.new_workspace(3, 2, 1)
    gw = torch.full((64,), 7.0, device="cuda")
    e = {n: v[:0] if n in ("dest", "w", "x", "gy", "add") else v for n, v in s.items() if v is not None}
    m.moe_norm_backward(e["grad"], e["x"], s["weight"], EPS, e["x"], gw, ws, m.new_norm_scratch(0, 64),
                        dest_row=e["dest"])
    assert (gw == 0).all()
    gw.fill_(7.0)
    m.moe_combine_norm_backward(e["gy"], e["yp"], e["dest"], e["w"], m.BlockCfg(), torch.empty_like(s["yp"]), e["w"],
                                ws, grad_weight=gw)
    assert (gw == 0).all()
    gx, want = torch.empty_like(s["x"]), norm_backward(s, False, 1.0)[0]
    m.moe_norm_backward(s["grad"], s["x"], s["weight"], EPS, gx, None, ws, dest_row=s["dest"], add=s["add"],
                        residual_grad=s["gy"])
    assert torch.equal(gx, want)


@pytest.mark.gpu
def test_rows_outside_are_reported_and_skipped():
    m = moe()
    s = inputs(6, 136, 3, BF, False, False, True, 0, seed=8)
    ref = {**s, "dest": s["dest"].clone()}
    ref["dest"][2, 1] = -1
    ref["dest"][4, 0] = -1
    s["dest"][2, 1] = s["yp"].shape[0]
    s["dest"][4, 0] = -2
    calls = [lambda q: forward(q, True, 1.0), lambda q: backward(q, True), lambda q: norm_backward(q, False, 1.0)]
    for f in calls:
        got, want = f(s), f(ref)
        with pytest.raises(m.MoeError) as e:
            m.moe_check_device_status(got[-1])
        assert e.value.status == 4 and e.value.info in (7, 12)
        m.moe_check_device_status(want[-1])
        for a, b in zip(got[:-1], want[:-1]):
            for x, y in (zip(a.values(), b.values()) if isinstance(a, dict) else [(a, b)]):
                live = ~torch.isnan(x.float())
                assert torch.equal(x[live], y[live]) and torch.equal(live, ~torch.isnan(y.float()))


@pytest.mark.gpu
def test_another_stream_and_a_replayed_graph():
    m = moe()
    s = inputs(33, 1032, 4, BF, True, True, True, 0.1, seed=9)
    want = [*forward(s, True, 1.0)[:2], *backward(s, True)[0].values(), *norm_backward(s, False, 1.0)[:2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [*forward(s, True, 1.0, stream=side)[:2], *backward(s, True, stream=side)[0].values()]
    torch.cuda.synchronize()
    T, H = s["x"].shape
    ws, sc = m.new_workspace(T, 4, 1), m.new_norm_scratch(T, H)
    outs = [torch.zeros_like(t) for t in want]
    cfg = m.BlockCfg(1, EPS, 1.0)

    def step():
        st = torch.cuda.current_stream()
        m.moe_combine_norm(s["yp"], s["dest"], s["w"], s["x"], cfg, outs[0], ws, shared=s["shared"],
                           weight=s["weight"], gate=s["gate"], next_weight=s["next_weight"], next_out=outs[1],
                           stream=st)
        m.moe_combine_norm_backward(s["gy"], s["yp"], s["dest"], s["w"], cfg, outs[2], outs[3], ws, sc,
                                    shared=s["shared"], weight=s["weight"], gate=s["gate"], grad_shared=outs[4],
                                    grad_gate=outs[5], grad_weight=outs[6], stream=st)
        m.moe_norm_backward(s["grad"], s["x"], s["weight"], EPS, outs[7], outs[8], ws, sc, dest_row=s["dest"],
                            add=s["add"], residual_grad=s["gy"], stream=st)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for o in outs:
            o.fill_(7.0)
        g.replay()
        for i, (a, b) in enumerate(zip(outs, want)):
            keep = slice(None) if i != 2 else s["landed"]
            assert torch.equal(a[keep], b[keep]), i
    for a, b in zip(got, want):
        keep = slice(None) if a.shape != s["yp"].shape else s["landed"]
        assert torch.equal(a[keep], b[keep])


@pytest.mark.gpu
def test_no_expert_rows_at_all():
    """An empty dispatched buffer: every assignment is dropped."""
    s = inputs(5, 72, 2, BF, True, True, True, 0, seed=11)
    s["dest"].fill_(-1)
    e = {**s, "yp": s["yp"][:0], "grad": s["grad"][:0], "landed": s["landed"][:0]}
    for f in (lambda q: forward(q, True, 0.5)[:2], lambda q: backward(q, True)[0].values(),
              lambda q: norm_backward(q, False, 0.5)[:2]):
        for a, b in zip(f(s), f(e)):
            assert torch.equal(a[:b.shape[0]], b) and (a.shape == b.shape or (a == 7.0).all())


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused(monkeypatch):
    """Calls launch on the current device (here it is said to be another one than the tensors')."""
    m = moe()
    s = inputs(3, 64, 2, BF, False, False, True, 0, seed=12)
    ws, sc = m.new_workspace(3, 2, 1), m.new_norm_scratch(3, 64)
    y, gw = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    codes, scales = torch.zeros(1, 8, 16, dtype=torch.uint8, device="cuda"), torch.ones(1, 8, 1, device="cuda").to(BF)
    w = m.pack_weights_int4(codes, scales, None, m.MOE_EPI_NONE)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    x4, o4, off, exp = torch.zeros(1, 32, device="cuda").to(BF), torch.zeros(1, 8, device="cuda"), i32(0, 1), i32(0)
    torch.cuda.synchronize()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for f in (lambda: m.moe_norm(s["x"], None, EPS, y),
              lambda: m.moe_combine_norm(s["yp"], s["dest"], s["w"], s["x"], m.BlockCfg(), y, ws),
              lambda: m.moe_combine_backward(s["gy"], s["yp"], s["dest"], s["w"], torch.empty_like(s["yp"]), gw, ws),
              lambda: m.moe_permute_backward(s["grad"], s["dest"], y, ws),
              lambda: m.moe_combine_norm_backward(s["gy"], s["yp"], s["dest"], s["w"], m.BlockCfg(),
                                                  torch.empty_like(s["yp"]), gw, ws, sc),
              lambda: m.moe_norm_backward(s["grad"], s["x"], None, EPS, y, None, ws, sc, dest_row=s["dest"]),
              lambda: m.pack_weights_int4(codes, scales, None, m.MOE_EPI_NONE),
              lambda: m.moe_grouped_product_int4(x4, off, exp, w, o4, ws)):
        with pytest.raises(ValueError, match="device"):
            f()


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    m = moe()
    qs = [inputs(400, 2048, 4, BF, True, True, True, 0.1, seed=20 + i) for i in range(2)]
    want = [[*backward(q, True)[0].values(), *norm_backward(q, False, 1.0)[:2]] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for q, st in zip(qs, streams):
            with torch.cuda.stream(st):
                got.append([*backward(q, True, stream=st)[0].values(), *norm_backward(q, False, 1.0, stream=st)[:2]])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.gpu
def test_rows_past_32_bits():
    """Rows more than 2^32 bytes (and 2^31 elements) into the dispatched buffers."""
    m = moe()
    T, H, k, n = 3, 8192, 2, 270000
    s = inputs(T, H, k, BF, False, False, True, 0, seed=10)
    far = torch.tensor([[n - 1, 7], [n - 2, n - 5], [262150, n - 9]], dtype=torch.int32, device="cuda")
    big = {**s, "dest": far}
    for name in ("yp", "grad"):
        big[name] = torch.zeros(n, H, dtype=BF, device="cuda")
        big[name][far.flatten().long()] = s[name][s["dest"].flatten().long()]
    y, _, _ = forward(s, True, 1.0)
    y2, _, _ = forward(big, True, 1.0)
    assert torch.equal(y, y2)
    a, b = backward(s, True)[0], backward(big, True)[0]
    assert torch.equal(a["rows"][s["dest"].flatten().long()], b["rows"][far.flatten().long()])
    assert torch.equal(a["w"], b["w"]) and torch.equal(a["weight"], b["weight"])
    assert (b["rows"][262144 + 100:n - 100] == 7.0).all()
    p, q = norm_backward(s, False, 1.0), norm_backward(big, False, 1.0)
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
