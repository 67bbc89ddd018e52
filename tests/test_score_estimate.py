"""The score that ranks pages: an estimate of an upper bound of q . k, off from
it by the stated amount and on either side, and how often it chooses the pages
that the bound itself would."""
import numpy as np
import pytest

import ops_reference as R


def _pages(pages, B, D, seed, gain=(), heads=8):
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((pages, 1, B, D)) + rng.standard_normal(D)
    k[..., : len(gain)] *= gain
    summary, ex = np.zeros((pages, 1, 2, D), np.int8), np.zeros((pages, 1), np.int8)
    R.block_summary(k, np.arange(pages * B), summary, ex)
    return k[:, 0], rng.standard_normal((heads, D)), summary[:, 0].astype(np.float64), ex[:, 0].astype(np.int64)


def _scores(k, q, summary, ex):
    """(exact upper bounds, scores, units of the pages, units of the queries)"""
    hi, lo = k.max(1), k.min(1)
    exact = np.stack([np.maximum(x * hi, x * lo).sum(1) for x in q])
    unit = 2.0 ** ex
    form = [R.int8_form(x) for x in q]
    score = np.stack([2.0 ** e * unit * np.maximum(r * summary[:, 0], r * summary[:, 1]).sum(1) for r, e in form])
    return exact, score, unit, np.array([2.0 ** e for _, e in form])


@pytest.mark.parametrize("D", [64, 128])
def test_score_is_within_half_a_unit_a_dim_and_may_be_below(D):
    k, q, summary, ex = _pages(64, 16, D, 3)
    exact, score, unit, qu = _scores(k, q, summary, ex)
    largest = np.abs(k).max(1)
    for i, x in enumerate(q):
        # half a unit of the key for each |q_d|, half a unit of the query for each |k_d|, and their product
        off = 0.5 * unit * np.abs(x).sum() + 0.5 * qu[i] * largest.sum(1) + 0.25 * D * unit * qu[i]
        assert (np.abs(score[i] - exact[i]) <= off * (1 + 1e-12)).all()
    assert 0.2 < (score < exact).mean() < 0.8  # rounded to the nearest: about as often below as above


@pytest.mark.parametrize("gain,least", [((), 0.95), ((15,) * 4, 0.85), ((50,) * 2, 0.75)])
def test_the_choice_by_the_score_against_the_choice_by_the_bound(gain, least):
    k, q, summary, ex = _pages(2048, 16, 128, 11, gain, heads=32)
    exact, score, _, _ = _scores(k, q, summary, ex)
    top = lambda x: set(np.argsort(-x, kind="stable")[:128])  # noqa: E731
    assert np.mean([len(top(a) & top(b)) / 128 for a, b in zip(exact, score)]) > least
