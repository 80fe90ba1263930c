"""The router with a balance bias at the ends of its inputs' range: a bias
that is NaN, scores that vanish in 64 bits, scores far apart.  Ids are equal to the
definition's."""

import numpy as np
import pytest
import torch

from test_gate import SIGMOID, SOFTMAX, check, make, moe, reference, run_gate


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


def ids_of(l, bias, fn, k, G=1, kept=1, topn=1):
    cfg = moe().GateCfg(fn, k, G, kept, topn, 1, 1.0)
    db = None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = run_gate(torch.from_numpy(l).cuda(), db, cfg)
    return ids.cpu().numpy(), w.cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T", [70, 8200])
@pytest.mark.parametrize("G,kept", [(1, 1), (4, 2)])
def test_nan_bias_is_the_lowest(G, kept, T, fn):
    """A bias that is NaN counts as -1e30: its expert is chosen last, and only for want of others."""
    rng = np.random.default_rng(T)
    E = 64
    l = rng.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    bias[[3, 20, 50]] = np.nan
    clean = np.where(np.isnan(bias), np.float32(-1e30), bias)
    ids, w = ids_of(l, bias, fn, 6, G, kept)
    some = np.concatenate((np.arange(64), rng.integers(0, T, 100)))
    rid, _ = reference(l[some], clean, fn, 6, G, kept, 1, True, 1.0)
    assert np.array_equal(ids[some], rid) and np.isfinite(w).all()
    assert not np.isin(ids, (3, 20, 50)).any()


@pytest.mark.gpu
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
def test_vanishing_scores_without_bias_and_groups(fn):
    """Without bias and groups the order is the logits', wherever the scores lie."""
    rng = np.random.default_rng(2)
    T, E, k = 100, 64, 8
    l = np.full((T, E), -900, np.float32)
    step = rng.integers(0, 4, (T, E))
    for i in range(3):                              # within three steps of one another
        l = np.where(step > i, np.nextafter(l, np.float32(0)), l)
    l[50:] *= 1000
    l[::2, 7] = 0
    ids, _ = ids_of(l, None, fn, k)
    assert np.array_equal(ids, np.argsort(-l, 1, kind="stable")[:, :k])


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("n", [9, 12, 16, 60])
def test_vanishing_scores_in_groups(n, fn, bias):
    """Scores that 64 bits hold as zero tie, by id, whether few or many experts are left."""
    rng = np.random.default_rng(n)
    T, E, k, G = 80, 64, 8, 4
    l = np.full((T, E), -np.inf, np.float32)
    for t in range(T):
        on = rng.choice(E, n, replace=False)
        l[t, on] = rng.uniform(-2000, -800, n)
        l[t, on[0]] = 1
    b = np.zeros(E, np.float32) if bias else None
    ids, _ = ids_of(l, b, fn, k, G, G, 2)
    rid, _ = reference(l, b, fn, k, G, G, 2, True, 1.0)
    assert np.array_equal(ids, rid)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [60, 8192])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_of_scores_far_apart(dtype, T):
    """Renormalised sigmoids whose smallest have fewer bits than a float holds, beside larger ones that are
    small themselves: weights and gradients to the last bits all the same (tolerances of test_gate)."""
    def edit(l, rng):
        n = l.shape[0]
        l[:] = -np.inf
        best = rng.choice([3.0, -1.0, -15.0, -30.0, -70.0, -79.0, -85.0], n)
        on = np.argsort(rng.random(l.shape), 1)[:, :9]
        v = best[:, None] - rng.uniform(0, 1, (n, 9)) * rng.choice([10.0, 50.0, 90.0], n)[:, None]
        v[:, 0] = best
        np.put_along_axis(l, on, v.astype(np.float32), 1)
    E = 32
    case = (T, E, SIGMOID, 8, 4, 4, 2, 1, 2.5, True, dtype)
    t, l, rng = make(T, E, dtype, T, edit=edit)
    check(t, l, rng, case, np.zeros(E, np.float32))
