"""The attention's bounds are narrow enough (no GPU): plausible mistakes fall outside them."""
import numpy as np
import pytest

from oracle import kv

from . import kv_cases


def _zeros(s, seen):
    return np.zeros_like(s)


def _mean(s, seen):
    return np.broadcast_to(seen[:, None] / np.maximum(seen.sum(-1), 1)[:, None, None], s.shape)


def _halved(s, seen):
    return kv_cases.softmax_of(s / 2, seen)


def _not_rescaled(s, seen):
    """Sums of the keys up to the last new maximum that count twice, as after a rescaling that was missed in part."""
    w = kv_cases.softmax_of(s, seen)
    last = np.where(seen[:, None], s, -np.inf).argmax(-1)[..., None]
    w = np.where(np.arange(s.shape[-1]) < last, 2 * w, w)
    return w / np.maximum(w.sum(-1, keepdims=True), 1e-300)


@pytest.mark.parametrize("name", kv_cases.CASES)
def test_mistakes_are_outside_the_bound(name):
    """An empty result, the plain mean, halved scores and a missed rescaling, in every sequence of every case."""
    b = kv_cases.CASES[name]()
    for i in range(len(b.seqs)):
        ref, tol = kv_cases.expected(b, i)
        for wrong in (_zeros, _mean, _halved, _not_rescaled):
            if wrong is _not_rescaled and not ("jumps" in name or "rising" in name):
                continue
            off = np.abs(kv_cases.expected(b, i, wrong)[0] - ref)
            assert np.any(off > 2 * tol), (name, i, wrong.__name__, np.max(off / tol))


@pytest.mark.parametrize("name", ["sharp", "rising", "below zero (2, 300, 40)"])
def test_the_cases_formula_is_the_oracles(name):
    b = kv_cases.CASES[name]()
    for i, (n, L) in enumerate(b.seqs[:2]):
        q = b.q[b.starts[i]:b.starts[i] + n].float().numpy().astype(np.float64)
        ref, mag, big = kv.attention(q, *b.kv[i], b.scale, b.window)
        out, tol = kv_cases.expected(b, i)
        np.testing.assert_allclose(out, ref, rtol=1e-9, atol=1e-12)
        np.testing.assert_allclose(tol, kv.tolerance(ref, mag, big, kv_cases.KEYS), rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("n", [1, 3, 80])
def test_small_values_are_not_within_the_bound_of_zero(n):
    """Values of 1e-30: a result flushed to zero is outside."""
    rng = np.random.default_rng(n)
    K, V, q = rng.normal(size=(300, 1, 128)), rng.normal(0.5, 1, size=(300, 1, 128)) * 1e-30, rng.normal(size=(n, 1, 128))
    ref, mag, big = kv.attention(q, K, V, 128 ** -0.5)
    assert np.all(np.any(np.abs(ref) > 2 * kv.tolerance(ref, mag, big), -1))
