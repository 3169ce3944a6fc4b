"""Pins for the key/value cache oracle (no GPU): hand-computed bytes, codes and rotations."""
import numpy as np
import pytest

from oracle import kv


def test_codes_and_parameters_by_hand():
    """Values (c - 3) * 0.5 with every code present: lo = -1.5, range 7.5, scale bf16(0.5), offset -1.5, codes c.
    fl32(1/15) * 7.5 = 0.5 + 7.5 * (fl32(1/15) - 1/15) rounds to 0.5 in bf16."""
    c = np.tile(np.arange(16), 4)
    code, par = kv.quantise(((c - 3) * 0.5).astype(np.float32)[None])
    np.testing.assert_array_equal(code[0], c)
    assert par[0].tolist() == [0x3F00, 0xBFC0]


def test_constant_and_tiny_and_non_finite_rows():
    x = np.zeros((5, 64), np.float32)
    x[1] = 2.5
    x[2, 0] = 2.0 ** -130  # range / 15 is below the smallest normal number
    x[3, 5] = np.nan
    x[4, 9] = np.inf
    code, par = kv.quantise(x)
    assert not code[:3].any()
    assert par[0].tolist() == [0, 0] and par[1].tolist() == [0, 0x4020] and par[2].tolist() == [0, 0]
    assert par[3].tolist() == [0x7FC0, 0x7FC0] and par[4].tolist() == [0x7FC0, 0x7FC0]


def test_quantisation_error_is_about_half_a_step():
    """The stored scale and offset are off by at most 2^-9 relative: a value is within
    s/2 + 15 s 2^-8 + |offset| 2^-9 of what is held."""
    rng = np.random.default_rng(3)
    x = rng.normal(0.3, 2, size=(200, 128)).astype(np.float32)
    code, par = kv.quantise(x)
    s, o = (kv.bf16_value(par[:, i:i + 1]).astype(np.float64) for i in (0, 1))
    assert np.all(np.abs(code * s + o - x) <= s * (0.5 + 15 * 2.0 ** -8) + np.abs(o) * 2.0 ** -8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_hand(interleaved):
    """A quarter turn of the first pair, a half turn of the second, and an unrotated rest."""
    x = np.arange(1, 9, dtype=np.float32)[None, None]
    t = np.array([[0, -1, 1, 0]], np.float32)
    want = [-2, 1, -3, -4, 5, 6, 7, 8] if interleaved else [-3, -2, 1, -4, 5, 6, 7, 8]
    np.testing.assert_array_equal(kv.rotate(x, t, interleaved)[0, 0], want)


def test_pool_bytes_and_round_trip():
    """Token 18 of page 1 (pages of 32): block 1, row 2; byte j of its codes holds 2j low and 2j + 1 high."""
    D, P = 64, 32
    pool = np.full((3, 2, P * (D + 8)), 0xEE, np.uint8)
    codes = (np.arange(2 * D).reshape(1, 2, D) * 7 % 16).astype(np.uint8)
    par = np.array([[[0x3F80, 0x4000], [0x3E00, 0xBF80]]], np.uint16)
    kv.pack_rows(pool, P, D, [1 * P + 18], codes, par, codes[:, ::-1], par[:, ::-1])
    blk = pool[1, 0, 16 * (D + 8):]
    assert blk[2 * 32] == codes[0, 0, 0] + 16 * codes[0, 0, 1] and blk[2 * 32 + 31] == codes[0, 0, 62] + 16 * codes[0, 0, 63]
    assert blk[512 + 2 * 32] == codes[0, 1, 0] + 16 * codes[0, 1, 1]
    assert blk[1024 + 8:1024 + 12].tolist() == [0x80, 0x3F, 0x00, 0x40]
    assert blk[1088 + 8:1088 + 12].tolist() == [0x00, 0x3E, 0x80, 0xBF]
    assert (pool != 0xEE).sum() <= 2 * 2 * (32 + 4)
    K, V = kv.unpack_rows(pool, P, D, [1 * P + 18])
    np.testing.assert_array_equal(K[0, 0], codes[0, 0] * 1.0 + 2.0)
    np.testing.assert_array_equal(K[0, 1], codes[0, 1] * 0.125 - 1.0)
    np.testing.assert_array_equal(V[0, 0], codes[0, 1] * 0.125 - 1.0)


def test_attention_by_hand_and_masks():
    """Two keys with scores ln 3 and 0: weights 3/4 and 1/4. A window of one sees the own key alone; a row before
    the first key sees none."""
    K = np.array([[[np.log(3.0), 0.0]], [[0.0, 0.0]]])
    V = np.array([[[4.0, 0.0]], [[8.0, 4.0]]])
    q = np.array([[[1.0, 0.0]]])
    np.testing.assert_allclose(kv.attention(q, K, V, 1.0)[0][0, 0], [5.0, 1.0])
    np.testing.assert_allclose(kv.attention(q, K, V, 1.0, window=1)[0][0, 0], [8.0, 4.0])
    out = kv.attention(np.ones((4, 1, 2)), K, V, 1.0)[0]
    assert not out[:2].any()
    np.testing.assert_allclose(out[2, 0], [4.0, 0.0])


def test_a_planted_mistake_is_outside_the_tolerance():
    """Leaving the newest key out, or seeing one key too many, is far outside the bound for a short cache."""
    rng = np.random.default_rng(4)
    K, V, q = rng.normal(size=(9, 1, 64)), rng.normal(size=(9, 1, 64)), rng.normal(size=(1, 1, 64))
    ref, mag, big = kv.attention(q, K[:8], V[:8], 0.125)
    tol = kv.tolerance(ref, mag, big)
    for L in (7, 9):
        assert np.any(np.abs(kv.attention(q, K[:L], V[:L], 0.125)[0] - ref) > 2 * tol)
