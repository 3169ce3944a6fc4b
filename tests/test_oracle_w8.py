"""The 8-bit oracle against closed forms and torch."""
import numpy as np
import pytest
import torch

from oracle import w8


def test_quantize_hand_derived():
    v = np.array([[127.0, -63.5, 0.5, 1.5, -127.0], [0, 0, 0, 0, 0], [np.inf, 0, 0, 0, 0], [1, np.nan, 0, 0, 0],
                  [2.0 ** -101, 0, 0, 0, 0], [254, 1, 3, -1, 5]], np.float32)
    q, s = w8.quantize_rows(v)
    # half to even: 63.5 -> 64, 0.5 -> 0, 1.5 -> 2
    assert q.tolist() == [[127, -64, 0, 2, -127], [0] * 5, [0] * 5, [0] * 5, [0] * 5, [127, 0, 2, 0, 2]]
    assert s[0] == 1 and s[1] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and s[4] == 0 and s[5] == 2


def test_quantize_is_within_half_a_step():
    v = np.random.default_rng(0).normal(size=(40, 333)).astype(np.float32)
    q, s = w8.quantize_rows(v)
    # fp32 products put a code at most 127 * 2^-23 off before it is rounded
    assert np.all(np.abs(q * s[:, None].astype(np.float64) - v) <= s[:, None] * (0.5 + 127 * 2.0 ** -22))
    assert np.all(np.abs(q).max(1) == 127)


def test_norm_matches_torch():
    g = torch.Generator().manual_seed(1)
    x, r, w = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((7, 96), (7, 96), (96,)))
    h, v = w8.rms_norm(x.numpy(), w.numpy(), 1e-5, r.numpy())
    want = torch.nn.functional.rms_norm(x + r, (96,), w, 1e-5)
    assert np.allclose(h, (x + r).numpy(), rtol=0, atol=0) and np.allclose(v, want.numpy(), rtol=1e-12, atol=0)
    h, v = w8.rms_norm(np.full((1, 4), 3.0), np.array([1.0, 2, 0, -1]), 0.0)
    assert v.tolist() == [[1, 2, 0, -1]]


def test_products_are_exact():
    rng = np.random.default_rng(2)
    a, b = rng.integers(-128, 128, (5, 70)), rng.integers(-128, 128, (9, 70))
    assert np.array_equal(w8.sums(a, b), a @ b.T)
    y = w8.linear(a, np.full(5, 0.5), b, np.full(9, 2.0))
    assert y.dtype == np.float32 and np.array_equal(y, a @ b.T)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_matches_torch(kind):
    rng = np.random.default_rng(3)
    x, w, u = rng.integers(-127, 128, (4, 32)), rng.integers(-127, 128, (6, 32)), rng.integers(-127, 128, (6, 32))
    s = [rng.random(n) * 0.02 for n in (4, 6, 6)]
    got = w8.gated(x, s[0], w, s[1], u, s[2], kind)
    X, W, U = (torch.from_numpy(q * t[:, None]) for q, t in ((x, s[0]), (w, s[1]), (u, s[2])))
    f = torch.nn.functional.silu if kind == "silu" else (lambda t: torch.nn.functional.gelu(t, approximate="tanh"))
    assert np.allclose(got, (f(X @ W.T) * (X @ U.T)).numpy(), rtol=1e-9, atol=1e-12)
    assert w8.act(np.array([-1e4, 0.0]), kind).tolist() == [0, 0]
