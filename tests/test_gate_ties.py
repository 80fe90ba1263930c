"""The router with a balance bias where scores nearly meet and many tokens are
routed at once (from 8192 tokens on a token takes four lanes, each with a part
of the row): the last choice against the first expert left out, both in the
part of one lane or anywhere.

Ids are equal to the definition's: scores that have to be told apart differ by
an fp32 step of a logit of magnitude 0.5 to 4, 2^-25 at least, times a
sigmoid's slope of 0.017 at least or a softmax's score, above 2^-40 of the
score in every case.
"""

import numpy as np
import pytest
import torch

from test_gate import SIGMOID, SOFTMAX, assert_admissible, moe, run_gate

T = 8192


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_ffn_gb300 import build
    build.build()


def rows_with_a_close_ninth(E, rng, home, peak):
    """fp32 rows whose nine best experts lie in `home` (expert numbers): seven
    far apart, then two that are equal or one step apart, the larger one
    before or after the smaller one."""
    l = rng.uniform(-6, -5, (T, E)).astype(np.float32)
    pick = home[np.argsort(rng.random((T, len(home))), 1)[:, :9]]
    put = lambda j, v: np.put_along_axis(l, pick[:, j:j + 1], v.astype(np.float32)[:, None], 1)
    for j in range(7):
        put(j, 1.5 + 0.25 * j + 0.1 * rng.random(T))
    a = rng.uniform(0.5, 1.25, T).astype(np.float32)
    put(7, a)
    put(8, np.where(np.arange(T) % 8 == 0, a, np.nextafter(a, np.float32(9))))
    if peak:
        put(0, np.where(np.arange(T) % 2 == 0, 1.5, 24.0))
    return l


CASES = [  # E, groups, kept, where the nine best lie, bias of that part
    (128, 4, 1, range(64, 96), None),
    (256, 4, 1, range(0, 64), None),
    (256, 4, 2, range(128, 192), None),
    (256, 8, 1, range(32, 64), None),
    (256, 8, 2, range(64, 128), None),          # two groups of one lane
    (512, 16, 1, range(480, 512), None),
    (256, 16, 2, range(16, 48), None),          # two groups of one lane
    (256, 16, 4, range(192, 256), None),        # all four groups of one lane
    (256, 1, 1, range(0, 16), 0.25),
    (64, 1, 1, range(48, 64), 0.25),
    (256, 8, 8, range(0, 256), None),           # anywhere
    (128, 4, 4, range(0, 128), None),
    (256, 1, 1, range(0, 256), 0.25),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fn,peak", [(SIGMOID, False), (SOFTMAX, False), (SOFTMAX, True)])
@pytest.mark.parametrize("case", CASES)
def test_close_ninth(case, fn, peak):
    E, G, kept, home, b = case
    if peak and b is not None:
        pytest.skip("beside a bias of 0.25 such scores are equal to 2^-40 of their sums")
    rng = np.random.default_rng(E + G + kept)
    l = rows_with_a_close_ninth(E, rng, np.array(home), peak)
    bias = None
    if b is not None:
        bias = np.zeros(E, np.float32)
        bias[list(home)] = b
    cfg = moe().GateCfg(fn, 8, G, kept, 2 if G > 1 else 1, 1, 1.0)
    dev, db = torch.from_numpy(l).cuda(), None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = run_gate(dev, db, cfg)
    # the nine best share a bias and lie in kept groups: their order is the logits'
    want = np.argsort(-l, 1, kind="stable")[:, :8]
    wrong = (ids.cpu().numpy() != want).any(1)
    assert not wrong.any(), (int(wrong.sum()), np.nonzero(wrong)[0][:5])
    for lo in (0, 4096):
        i2, _ = run_gate(dev[lo:lo + 4096], db, cfg)
        assert torch.equal(ids[lo:lo + 4096], i2)


def test_row_of_two_close_scores_is_not_a_tie():
    """The first case's premise, on the CPU: in 64 bits the two scores differ."""
    a = np.float32(0.5)
    s = lambda x: 1 / (1 + np.exp(-np.float64(x)))
    assert s(np.nextafter(a, np.float32(9))) - s(a) > 2.0 ** -40


@pytest.mark.gpu
@pytest.mark.parametrize("fn", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("E,G,kept,topn", [(96, 1, 1, 1), (128, 4, 1, 2), (128, 4, 2, 1), (256, 8, 1, 2),
                                           (256, 8, 3, 2), (256, 16, 2, 2)])
@pytest.mark.parametrize("k", [5, 8])
def test_many_close_scores(E, G, kept, topn, k, fn):
    """Rows whose scores all lie within a few fp32 steps, exact ties among them."""
    rng = np.random.default_rng(3 * E + G)
    l = np.repeat(rng.standard_normal((T, 1)), E, 1).astype(np.float32)
    step = rng.integers(-3, 4, (T, E))
    for _ in range(3):
        l = np.where(step > 0, np.nextafter(l, np.float32(9)), np.where(step < 0, np.nextafter(l, np.float32(-9)), l))
        step -= np.sign(step)
    bias = (rng.integers(-2, 3, E) * 2.0 ** -26).astype(np.float32)
    for b in (None, bias):
        if b is None and G == 1:
            b = np.zeros(E, np.float32)
        cfg = moe().GateCfg(fn, k, G, kept, topn, 1, 1.0)
        ids, _ = run_gate(torch.from_numpy(l).cuda(), None if b is None else torch.from_numpy(b).cuda(), cfg)
        some = rng.integers(0, T, 300)
        assert_admissible(ids.cpu().numpy()[some], l[some].astype(np.float64), b, fn, k, G, kept, topn)
