"""Pins of the oracles of the rotary positions, the draft acceptance, the attention mass and the eviction."""
import itertools

import numpy as np
import pytest

from oracle import accept, eviction, rope


def test_rope_identity_norm_and_relative_distance():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 256))
    kw = dict(rotary_dim=128, theta=1e4, sections=(20, 30, 14), deal_axes=True)
    assert np.array_equal(rope.rotate(x, np.zeros((2, 3)), **kw), x)
    y = rope.rotate(x, rng.integers(-1000, 1000, (2, 3)), **kw)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    assert np.array_equal(y[..., 128:], x[..., 128:])
    a, b = x[:1], x[1:]
    dots = [np.sum(rope.rotate(a, [[p + 3, p + 7, p]], **kw) * rope.rotate(b, [[p, p, p - 2]], **kw)) for p in (0, 11, 500)]
    assert np.allclose(dots, dots[0], rtol=1e-10)


def test_rope_pairs_by_hand():
    axis, f = rope.pairs(16, 256.0, (4, 3, 1), True, False)
    assert axis.tolist() == [0, 1, 2, 0, 1, 0, 1, 0] and np.allclose(f, 2.0 ** -np.arange(8))
    axis, f = rope.pairs(16, 16.0, (4, 4), False, True)
    assert axis.tolist() == [0] * 4 + [1] * 4 and np.allclose(f, np.tile(2.0 ** -np.arange(4), 2))
    x = np.zeros((1, 1, 256))
    x[0, 0, 0] = 1.0
    y = rope.rotate(x, [[2]], 16, 1e4, (8,))
    assert y[0, 0, 0] == np.cos(2.0) and y[0, 0, 8] == np.sin(2.0)
    y = rope.rotate(x, [[2]], 16, 1e4, (8,), adjacent=True)
    assert y[0, 0, 0] == np.cos(2.0) and y[0, 0, 1] == np.sin(2.0)


@pytest.mark.parametrize("seed", range(20))
def test_keep_against_brute_force(seed):
    """Every subset of the right size that holds the protected ends: the kept one is the largest by (mass, -position)."""
    rng = np.random.default_rng(seed)
    L = int(rng.integers(1, 9))
    m = rng.integers(0, 3, L).astype(np.float64)
    budget, sink, recent = int(rng.integers(1, 10)), int(rng.integers(0, 3)), int(rng.integers(0, 3))
    got = eviction.keep(m, budget, sink, recent)
    n = min(L, budget)
    assert len(got) == n and np.all(np.diff(got) > 0)
    r = min(recent, n)
    s = min(sink, n - r)
    must = set(range(s)) | set(range(L - r, L))
    assert must <= set(got.tolist())
    best = max((sorted(((m[i], -i) for i in c if i not in must), reverse=True), c) for c in itertools.combinations(range(L), n)
               if must <= set(c))
    assert list(best[1]) == got.tolist()


def test_keep_with_nan_and_infinities():
    m = np.array([np.nan, 1.0, -np.inf, np.inf, np.nan, 0.0, -0.0])
    assert eviction.keep(m, 4, 0, 0).tolist() == [1, 3, 5, 6]
    assert eviction.keep(m, 6, 0, 0).tolist() == [0, 1, 2, 3, 5, 6]


def test_mass_counts_every_row_once():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((3, 8, 256)), rng.standard_normal((50, 256))
    s = eviction.scores(q, k, 47, 8)
    lse = eviction.log_sum_exp(s)
    m = eviction.mass(np.full(50, np.nan), s, lse, 0.0, 47)
    assert np.isclose(m.sum(), 24.0)                # 24 rows of weights that add up to one
    again = eviction.mass(m, s, lse, 0.5, 47)
    assert np.allclose(again[:47], 1.5 * m[:47]) and np.allclose(again[47:], m[47:])
    assert np.all(s[:8, 48:] == -np.inf) and np.all(np.isfinite(s[16:, 49]))


def test_draft_acceptance_follows_the_target():
    """4,000 steps over four tokens: the token after t_0 follows p (five standard deviations: 0.04)."""
    n = 4000
    p, q = np.array([0.5, 0.3, 0.15, 0.05]), np.array([0.1, 0.3, 0.2, 0.4])
    rng = np.random.default_rng(3)
    drafts = rng.choice(4, n, p=q)
    tokens = np.zeros(2 * n, np.int64)
    tokens[1::2] = drafts
    acc, nxt, com, prob, _ = accept.draft_accept(np.tile(np.log(p), (2 * n, 1)), np.tile(q, (2 * n, 1)), 2 * np.arange(n), [2] * n,
                                                 tokens, [10] * n, 1.0, rng.random(2 * n), 17)
    first = np.where(acc == 1, drafts, nxt)
    assert np.all(np.abs(np.bincount(first, minlength=4) / n - p) < 0.04)
    assert np.allclose(prob[0::2], np.minimum(1, p / q)[drafts]) and np.all(np.isnan(prob[1::2]))
    assert np.all(com == 10 - (1 - acc))


def test_draft_acceptance_edges():
    lg = np.full((2, 3), -np.inf)
    lg[1, 2] = 0.0
    q = np.full((2, 3), 1 / 3)
    acc, nxt, com, prob, _ = accept.draft_accept(lg, q, [0], [2], [0, 2], [5], 1.0, [0.0, 0.0], 1)
    assert (acc[0], nxt[0], com[0], prob[0]) == (0, -1, 4, 0.0)      # nothing can follow the first row
    acc, nxt, _, prob, _ = accept.draft_accept(lg[::-1], 0 * q, [0], [2], [0, 2], [5], 1.0, [0.5, 0.0], 1)
    assert (acc[0], nxt[0], prob[0]) == (1, -1, 1.0)                # q = 0 and p > 0: taken
