"""The router with a balance bias: refusals on the CPU; choice, weights,
gradient and bias update on the GPU against a 64-bit implementation of the
definition in moe.h.

Tolerances.  Ids are equal.  A weight is within a few fp32 operations of its
exact value: 16 half steps of fp32 (16 * 2^-24) relative, as is each term of a
gradient, which subtracts two of them, so 32 * 2^-24 of the terms' sizes; a
bf16 gradient adds its own rounding, 2^-8 of the value.
"""

import ctypes

import numpy as np
import pytest
import torch

SOFTMAX, SIGMOID = 0, 1
HALF32, HALF16 = 2.0 ** -24, 2.0 ** -8


def moe():
    from grouped_ffn_gb300 import moe as m
    return m


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


# ------------------------------------------------------------------ 64-bit definition
def scores(l, fn):
    l = np.where(np.isnan(l), -np.inf, np.minimum(l.astype(np.float64), np.finfo(np.float32).max))
    with np.errstate(over="ignore", invalid="ignore"):
        if fn == SIGMOID:
            return 1 / (1 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.where(np.isneginf(l), 0, np.exp(l - np.where(np.isneginf(m), 0, m)))
        z = e.sum(1, keepdims=True)
        return np.where(z > 0, e / np.where(z > 0, z, 1), 0)


def reference(l, bias, fn, k, G, kept, topn, renorm, scale):
    l = np.asarray(l, np.float64)
    T, E = l.shape
    off = ~(l > -np.inf)
    s = scores(l, fn)
    c = s + (0 if bias is None else np.asarray(bias, np.float64))
    ids = np.empty((T, k), np.int32)
    per = E // G
    for t in range(T):
        gs = []
        for g in range(G):
            v = sorted((c[t, e] for e in range(g * per, (g + 1) * per) if not off[t, e]), reverse=True)
            gs.append(sum(v[:topn]) if v else -np.inf)
        order = sorted(range(G), key=lambda g: (-gs[g], g))[:kept]
        cand = [e for e in range(E) if e // per in order]
        cand.sort(key=lambda e: (off[t, e], 0.0 if off[t, e] else -c[t, e], e))
        ids[t] = cand[:k]
    return ids, weights(l, ids, fn, renorm, scale)


def weights(l, ids, fn, renorm, scale):
    s = np.take_along_axis(scores(l, fn), ids, 1)
    if not renorm:
        return scale * s
    # log scores keep ratios of scores too small for a float
    ls = np.take_along_axis(l, ids, 1)
    ls = np.where(np.isnan(ls), -np.inf, np.minimum(ls, np.finfo(np.float32).max))
    logs = ls if fn == SOFTMAX else np.where(ls > -30, -np.log1p(np.exp(-np.maximum(ls, -30))), ls)
    m = logs.max(1, keepdims=True)
    e = np.where(np.isneginf(logs), 0, np.exp(logs - np.where(np.isneginf(m), 0, m)))
    z = e.sum(1, keepdims=True)
    return np.where(z > 0, scale * e / np.where(z > 0, z, 1), 0)


def gradient(l, ids, g, fn, renorm, scale):
    """Formula, and the size of the terms each entry subtracts."""
    s_all = scores(l, fn)
    s = np.take_along_axis(s_all, ids, 1)
    T, E = l.shape
    dl, size = np.zeros((T, E)), np.zeros((T, E))
    if renorm:
        v = weights(l, ids, fn, True, 1.0)
        f = v * ((1 - s) if fn == SIGMOID else 1)
        dot, adot = (g * v).sum(1, keepdims=True), (np.abs(g) * v).sum(1, keepdims=True)
        np.put_along_axis(dl, ids, scale * (g - dot) * f, 1)
        np.put_along_axis(size, ids, scale * (np.abs(g) + adot) * f, 1)
    elif fn == SIGMOID:
        np.put_along_axis(dl, ids, scale * g * s * (1 - s), 1)
        size = np.abs(dl)
    else:
        G = np.zeros((T, E))
        np.put_along_axis(G, ids, scale * g, 1)
        dl = s_all * (G - (G * s_all).sum(1, keepdims=True))
        size = s_all * (np.abs(G) + (np.abs(G) * s_all).sum(1, keepdims=True))
    return dl, size


# ------------------------------------------------------------------ CPU: refusals
FAKE = ctypes.c_void_p(0x10000)   # never dereferenced


def test_refusals():
    m = moe()
    L = m.lib()

    def gate(T=8, E=64, ld=64, kind=0, logits=FAKE, ids=FAKE, w=FAKE, **kw):
        a = dict(score_fn=0, k=2, n_groups=1, topk_groups=1, group_topn=1, renormalize=1, scale=1.0)
        a.update(kw)
        cfg = m.GateCfg(**a)
        return L.moe_gate(logits, kind, ld, T, E, None, ctypes.byref(cfg), ids, w, None)

    assert gate(T=0) == 0
    for kw in (dict(T=-1), dict(E=0), dict(ld=63), dict(kind=2), dict(logits=None), dict(ids=None),
               dict(w=None), dict(score_fn=2), dict(k=0), dict(E=4, ld=4, k=5), dict(renormalize=2),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(n_groups=0),
               dict(n_groups=8, topk_groups=9), dict(n_groups=8, topk_groups=0),
               dict(n_groups=8, group_topn=9), dict(n_groups=8, topk_groups=1, k=9)):
        assert gate(**kw) == 1, kw
    for kw in (dict(E=513, ld=513), dict(k=17), dict(n_groups=33), dict(n_groups=7),
               dict(group_topn=9, n_groups=2)):
        assert gate(**kw) == 2, kw
    cfg = m.GateCfg(0, 2, 1, 1, 1, 1, 1.0)
    back = lambda g=FAKE, out=FAKE, ws=FAKE, n=256: L.moe_gate_backward(
        FAKE, 0, 64, 8, 64, FAKE, g, ctypes.byref(cfg), out, ws, n, None)
    assert back(g=None) == 1 and back(out=None) == 1
    assert back(ws=None) == 6 and back(n=16) == 6
    up = lambda E=64, c=FAKE, b=FAKE, r=0.1, o=FAKE: L.moe_gate_update_bias(c, E, b, r, o, None)
    assert up(E=0) == 1 and up(c=None) == 1 and up(b=None) == 1 and up(o=None) == 1
    assert up(r=-1.0) == 1 and up(r=float("nan")) == 1 and up(E=513) == 2


def test_python_refusals():
    m = moe()
    cfg = m.GateCfg(0, 2, 1, 1, 1, 1, 1.0)
    with pytest.raises(TypeError):
        m.moe_gate(torch.zeros(4, 8), None, cfg, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))


# ------------------------------------------------------------------ GPU
CASES = [  # T, E, fn, k, groups, kept, topn, renorm, scale, bias, dtype
    (1, 1, SOFTMAX, 1, 1, 1, 1, 1, 1.0, True, "f32"),
    (3, 5, SIGMOID, 5, 1, 1, 1, 0, 2.5, True, "f32"),
    (257, 32, SOFTMAX, 4, 1, 1, 1, 0, 1.0, False, "f32"),
    (100, 33, SOFTMAX, 16, 1, 1, 1, 1, 1.0, True, "bf16"),
    (65, 60, SOFTMAX, 4, 6, 2, 2, 0, 1.0, True, "bf16"),
    (130, 64, SIGMOID, 8, 32, 8, 2, 1, 2.5, True, "f32"),
    (77, 120, SIGMOID, 6, 6, 3, 2, 1, 1.0, False, "bf16"),
    (129, 256, SIGMOID, 8, 8, 4, 2, 1, 2.5, True, "f32"),
    (64, 256, SOFTMAX, 8, 8, 4, 8, 0, 1.0, True, "bf16"),
    (33, 257, SIGMOID, 3, 1, 1, 1, 0, 1.0, True, "f32"),
    (31, 512, SOFTMAX, 16, 4, 1, 3, 1, 1.0, True, "f32"),
    (40, 384, SIGMOID, 8, 8, 8, 1, 1, 1.0, True, "bf16"),
]


def make(T, E, dtype, seed, spread=1.0, edit=None):
    rng = np.random.default_rng(seed)
    l = (spread * rng.standard_normal((T, E))).astype(np.float32)
    if edit is not None:
        edit(l, rng)
    t = torch.from_numpy(l).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t, t.float().numpy().astype(np.float64), rng


def run_gate(t, bias, cfg):
    m = moe()
    T = t.shape[0]
    ids = torch.full((T, cfg.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, cfg.k), float("nan"), device="cuda")
    m.moe_gate(t, bias, cfg, ids, w)
    return ids, w


def check(t, l, rng, case, bias):
    T, E, fn, k, G, kept, topn, renorm, scale, _, dtype = case
    m = moe()
    cfg = m.GateCfg(fn, k, G, kept, topn, renorm, scale)
    dev = t.cuda()
    ids, w = run_gate(dev, None if bias is None else torch.from_numpy(bias).cuda(), cfg)
    rid, rw = reference(l, bias, fn, k, G, kept, topn, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), rid)
    err = np.abs(w.cpu().numpy().astype(np.float64) - rw)
    assert (err <= 16 * HALF32 * rw + 2.0 ** -140).all(), (err / np.maximum(rw, 1e-300)).max()
    g = rng.standard_normal((T, k)).astype(np.float32)
    ws = m.new_workspace(T, k, E)
    out = torch.full((T, E), float("nan"), dtype=t.dtype, device="cuda")
    m.moe_gate_backward(dev, ids, torch.from_numpy(g).cuda(), cfg, out, ws)
    m.moe_check_device_status(ws)
    dl, size = gradient(l, rid, g.astype(np.float64), fn, renorm, scale)
    tol = 32 * HALF32 * size + 2.0 ** -120 + (HALF16 * np.abs(dl) * 1.0001 if dtype == "bf16" else 0)
    got = out.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - dl) <= tol).all()
    return ids, w, got, g


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_gate_and_gradient(case):
    T, E, dtype = case[0], case[1], case[10]
    t, l, rng = make(T, E, dtype, 7 * T + E)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if case[9] else None
    check(t, l, rng, case, bias)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_rows(fn, renorm, groups):
    """Masked experts, groups and whole rows; NaN; logits at both ends."""
    def edit(l, rng):
        l[0] = -np.inf
        l[1] = np.nan
        l[2, 3:] = -np.inf                   # fewer unmasked experts than k
        l[3, :16] = -np.inf                  # a group without an unmasked expert
        l[4] = np.finfo(np.float32).min
        l[5] = -90 + 0.01 * l[5]             # sigmoids and their sum near the smallest floats
        l[6] = -300 + 0.01 * l[6]
        l[7, ::2] = np.nan
        l[8] = 0
        l[9, 5] = np.inf
        l[10, :] = -np.inf
        l[10, 63] = 1.0
    case = (24, 64, fn, 6, groups, min(groups, 2), 2, renorm, 1.5, True, "f32")
    t, l, rng = make(24, 64, "f32", 5, edit=edit)
    bias = (0.1 * rng.standard_normal(64)).astype(np.float32)
    check(t, l, rng, case, bias)


def assert_admissible(ids, l, bias, fn, k, G, kept, topn):
    """The choice is one that moe.h allows: scores (and group scores) closer
    than 2^-40 may be taken in either order, exact ties only by id."""
    eps = 2.0 ** -40
    T, E = l.shape
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    c = scores(l, fn) + b
    per = E // G
    gs = np.sort(c.reshape(T, G, per), 2)[:, :, ::-1][:, :, :topn].sum(2)
    ranked = np.sort(gs, 1)[:, ::-1]
    for t in range(T):
        row = ids[t]
        assert len(set(row)) == k
        assert (gs[t, row // per] >= ranked[t, kept - 1] - eps).all()
        assert (np.diff(c[t, row]) <= eps).all()
        sure = np.ones(G, bool) if kept == G else gs[t] > ranked[t, kept] + eps
        rest = np.setdiff1d(np.nonzero(np.repeat(sure, per))[0], row)
        assert (c[t, rest] <= c[t, row].min() + eps).all()
        for a, z in zip(row[:-1], row[1:]):
            if l[t, a] == l[t, z] and b[a] == b[z]:
                assert a < z
        last = row[-1]
        for e in rest:
            if l[t, e] == l[t, last] and b[e] == b[last] and e // per == last // per:
                assert e > last


@pytest.mark.gpu
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
def test_close_scores(fn):
    """Scores closer than fp32 tells apart, and exact ties."""
    T, E = 200, 96
    rng = np.random.default_rng(3)
    l = np.repeat(rng.standard_normal((T, 1)), E, 1).astype(np.float32)
    step = rng.integers(-3, 4, (T, E))
    for _ in range(3):
        l = np.where(step > 0, np.nextafter(l, np.float32(9)), np.where(step < 0, np.nextafter(l, np.float32(-9)), l))
        step -= np.sign(step)
    bias = (rng.integers(-2, 3, E) * 2.0 ** -26).astype(np.float32)
    for b in (None, bias):
        for groups, kept in ((1, 1), (8, 3)):
            cfg = moe().GateCfg(fn, 8, groups, kept, 2, 1, 1.0)
            ids, _ = run_gate(torch.from_numpy(l).cuda(), None if b is None else torch.from_numpy(b).cuda(), cfg)
            assert_admissible(ids.cpu().numpy(), l.astype(np.float64), b, fn, 8, groups, kept, 2)


MANY = [  # sizes that take four lanes a token, and neighbours of them
    (8200, 256, SIGMOID, 8, 8, 4, 2, 1, 2.5, True, "f32"),
    (8192, 256, SIGMOID, 6, 8, 3, 1, 0, 1.0, False, "f32"),
    (8201, 32, SOFTMAX, 4, 1, 1, 1, 0, 1.0, True, "bf16"),
    (8195, 64, SIGMOID, 8, 8, 8, 2, 1, 1.0, True, "f32"),
    (8193, 64, SOFTMAX, 5, 4, 2, 2, 1, 1.0, True, "f32"),
    (8199, 128, SOFTMAX, 8, 4, 1, 2, 0, 2.0, False, "bf16"),
    (8194, 128, SIGMOID, 1, 1, 1, 1, 1, 1.0, True, "bf16"),
    (8197, 256, SOFTMAX, 7, 1, 1, 1, 1, 1.0, True, "f32"),
    (8198, 96, SIGMOID, 4, 1, 1, 1, 1, 1.0, True, "f32"),
    (9000, 256, SIGMOID, 16, 8, 4, 2, 1, 1.0, True, "f32"),
    (8196, 512, SIGMOID, 8, 16, 5, 2, 1, 1.0, True, "f32"),
    (8203, 384, SOFTMAX, 6, 8, 4, 2, 1, 1.0, True, "bf16"),
    (8192, 160, SIGMOID, 8, 4, 3, 1, 1, 1.0, True, "f32"),
    (8192, 512, SOFTMAX, 8, 1, 1, 1, 0, 1.0, True, "bf16"),
    (8192, 320, SIGMOID, 3, 1, 1, 1, 1, 1.0, True, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", MANY)
def test_many_tokens(case):
    """Many tokens: rows of every kind among them, compared with the definition on a sample and with
    the same rows in small calls everywhere."""
    T, E, fn, k, G, kept, topn, renorm, scale, has_bias, dtype = case

    def edit(l, rng):
        l[0] = -np.inf
        l[1] = np.nan
        l[2, 3:] = -np.inf
        l[3, :E // 4] = -np.inf
        l[4] = -90 + 0.01 * l[4]
        l[5] = 0
        l[6, 5] = np.inf
        l[7, ::2] = np.nan
        l[8] = 20 + l[8]
        l[9] *= 30
        l[-1] = l[-2]
    t, l, rng = make(T, E, dtype, T + E, edit=edit)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if has_bias else None
    m = moe()
    cfg = m.GateCfg(fn, k, G, kept, topn, renorm, scale)
    dev, db = t.cuda(), None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = run_gate(dev, db, cfg)
    sample = np.concatenate((np.arange(40), rng.integers(40, T, 200), [T - 2, T - 1]))
    rid, rw = reference(l[sample], bias, fn, k, G, kept, topn, renorm, scale)
    assert np.array_equal(ids.cpu().numpy()[sample], rid)
    err = np.abs(w.cpu().numpy().astype(np.float64)[sample] - rw)
    assert (err <= 16 * HALF32 * rw + 2.0 ** -140).all()
    for lo in range(0, T, 2000):
        i2, w2 = run_gate(dev[lo:lo + 2000], db, cfg)
        assert torch.equal(ids[lo:lo + 2000], i2)
        d = (w[lo:lo + 2000] - w2).abs()
        assert (d <= 32 * HALF32 * w2 + 2.0 ** -140).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
def test_many_tokens_with_large_biases(fn):
    """Scores with biases beyond the range of the fixed-point keys."""
    T, E = 8192, 64
    t, l, rng = make(T, E, "f32", 77)
    bias = (rng.choice([0.0, 3.0, -7.5, 7.8, 9.0, -50.0, 1e30], E)).astype(np.float32)
    for G, kept in ((1, 1), (4, 2)):
        cfg = moe().GateCfg(fn, 6, G, kept, 2 if G > 1 else 1, 1, 1.0)
        db = torch.from_numpy(bias).cuda()
        ids, w = run_gate(t.cuda(), db, cfg)
        i2, w2 = run_gate(t.cuda()[:4000], db, cfg)
        assert torch.equal(ids[:4000], i2)
        assert ((w[:4000] - w2).abs() <= 32 * HALF32 * w2 + 2.0 ** -140).all()
        sample = rng.integers(0, T, 100)
        rid, _ = reference(l[sample], bias, fn, 6, G, kept, 2 if G > 1 else 1, 1, 1.0)
        # (scores under a bias of 1e30 vanish in 64 bits too, and tie by id)
        assert np.array_equal(ids.cpu().numpy()[sample], rid)


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, 1, 2, 3])
def test_many_tokens_groups_with_disabled_experts(first):
    """Group scores that large negative biases enter: one group with a single usable expert, one
    with all experts disabled a little, of which the first has to go."""
    T, E = 8192, 64
    t, l, rng = make(T, E, "f32", 5)
    bias = np.zeros(E, np.float32)
    g = lambda i: slice(16 * ((first + i) % 4), 16 * ((first + i) % 4) + 16)
    bias[g(0)] = -30.0
    bias[g(0).start + 3] = 0.0
    bias[g(1)] = -10.0
    cfg = moe().GateCfg(SIGMOID, 6, 4, 3, 2, 1, 1.0)
    ids, w = run_gate(t.cuda(), torch.from_numpy(bias).cuda(), cfg)
    sample = rng.integers(0, T, 200)
    rid, rw = reference(l[sample], bias, SIGMOID, 6, 4, 3, 2, True, 1.0)
    assert not ((rid // 16) == first).any()
    assert np.array_equal(ids.cpu().numpy()[sample], rid)
    i2, _ = run_gate(t.cuda()[:4096], torch.from_numpy(bias).cuda(), cfg)
    assert torch.equal(ids[:4096], i2)


@pytest.mark.gpu
def test_row_stride_and_bias_order():
    """Rows further apart than their length; a large bias decides the choice, not the weights."""
    m = moe()
    t, l, rng = make(50, 64, "f32", 11)
    wide = torch.zeros(50, 96)
    wide[:, :64] = t
    bias = np.zeros(64, np.float32)
    bias[[9, 3, 60]] = (30.0, 20.0, 1e38)      # the last one is clamped
    cfg = m.GateCfg(SIGMOID, 3, 1, 1, 1, 1, 1.0)
    view = wide.cuda()[:, :64]
    ids, w = run_gate(view, torch.from_numpy(bias).cuda(), cfg)
    assert (ids.cpu().numpy() == [60, 9, 3]).all()
    rw = weights(l, ids.cpu().numpy(), SIGMOID, True, 1.0)
    assert (np.abs(w.cpu().numpy() - rw) <= 16 * HALF32 * rw).all()
    g = torch.ones(50, 3, device="cuda")
    ws = m.new_workspace(50, 3, 64)
    a, b = torch.empty(50, 64, device="cuda"), torch.empty(50, 64, device="cuda")
    m.moe_gate_backward(view, ids, g, cfg, a, ws)
    m.moe_gate_backward(t.cuda(), ids, g, cfg, b, ws)
    assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [0, 1])
def test_gradient_against_differences(fn, renorm):
    case = (6, 12, fn, 3, 1, 1, 1, renorm, 2.0, False, "f32")
    t, l, rng = make(6, 12, "f32", 21)
    ids, _, got, g = check(t, l, rng, case, None)
    ids = ids.cpu().numpy()
    h = 1e-5
    for e in range(12):
        d = np.zeros_like(l)
        d[:, e] = h
        hi, lo = weights(l + d, ids, fn, renorm, 2.0), weights(l - d, ids, fn, renorm, 2.0)
        num = ((hi - lo) / (2 * h) * g).sum(1)
        # differences: h^2 of third derivatives below 2 |g| scale, rounding 1e-16 / h
        assert np.abs(num - got[:, e]).max() <= 4 * np.abs(g).sum(1).max() * (h * h + 1e-11 + 64 * HALF32)


@pytest.mark.gpu
def test_bad_id_is_reported_and_skipped():
    m = moe()
    t = torch.randn(4, 16).cuda()
    ids = torch.tensor([[0, 1], [2, 16], [3, 4], [-1, 5]], dtype=torch.int32, device="cuda")
    cfg = m.GateCfg(SIGMOID, 2, 1, 1, 1, 0, 1.0)
    ws = m.new_workspace(4, 2, 16)
    out = torch.full((4, 16), float("nan"), device="cuda")
    m.moe_gate_backward(t, ids, torch.ones(4, 2, device="cuda"), cfg, out, ws)
    with pytest.raises(m.MoeError) as e:
        m.moe_check_device_status(ws)
    assert e.value.status == 4 and e.value.info in (3, 6)
    got = out.cpu()
    assert torch.isfinite(got).all() and (got[1, 2] != 0) and int((got != 0).sum()) == 6


@pytest.mark.gpu
def test_update_bias_and_graph():
    m = moe()
    rng = np.random.default_rng(0)
    for E in (1, 7, 64, 512):
        n = rng.integers(0, 50, E).astype(np.int32)
        n[0] = 2 ** 31 - 1 if E == 512 else n[0]
        b = rng.standard_normal(E).astype(np.float32)
        t = torch.from_numpy(b).cuda()
        m.moe_gate_update_bias(torch.from_numpy(n).cuda(), t, 0.01, t)
        total = int(n.astype(np.int64).sum())
        sign = np.sign(total - E * n.astype(np.int64)).astype(np.float32)
        assert np.array_equal(t.cpu().numpy(), b + sign * np.float32(0.01))
    # the step as a graph, replayed on new logits
    cfg = m.GateCfg(SIGMOID, 8, 8, 4, 2, 1, 2.5)
    logits = torch.randn(33, 256, device="cuda")
    bias = torch.zeros(256, device="cuda")
    ids = torch.empty(33, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(33, 8, device="cuda")
    m.moe_gate(logits, bias, cfg, ids, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_gate(logits, bias, cfg, ids, w)
    logits.copy_(torch.randn(33, 256, device="cuda"))
    graph.replay()
    i2, w2 = run_gate(logits, bias, cfg)
    assert torch.equal(ids, i2) and torch.equal(w, w2)
