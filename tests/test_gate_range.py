"""The router with a balance bias at the ends of its inputs' range: a bias
that is NaN, and scores that vanish in 64 bits.  Ids are equal to the
definition's."""

import numpy as np
import pytest
import torch

from test_gate import SIGMOID, SOFTMAX, moe, reference, run_gate


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
