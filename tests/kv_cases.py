"""Cases of the attention whose scores 16 bits hold exactly, so that their bound leaves no room for a wrong softmax.

Keys are (code - 8) or (code + 16) times a power of two and queries small multiples of 1/4: every product and every
operand of a kernel is exact, and a score is off by its fp32 arithmetic alone. (With keys rounded to 2^-9 the bound of a
row grows as exp(2^-8 |score|) and passes the result itself where scores are large.)
"""
import numpy as np
import torch

from oracle import kv

from .test_gpu_kv_attention import Batch

KEYS = 2.0 ** -20  # what fp32 leaves of a score: products and the sum of two terms, the factors, the difference to m


def key_rows(rng, shape, size, centre=-8):
    """fp32 rows (code + centre) * size whose first two channels are the lowest and the highest code: they are held exactly."""
    c = rng.integers(0, 16, shape)
    c[..., 0], c[..., 1] = 0, 15
    return ((c + centre) * size).astype(np.float32)


def query_rows(seed, T, Hq, D, most=8):
    """bf16 multiples of 1/4 up to most / 4."""
    return (torch.randint(-most, most + 1, (T, Hq, D), generator=torch.Generator().manual_seed(seed)) / 4).bfloat16()


def case(seqs, Hq, Hk, D, page, edit, q, window=0, scale=None, seed=0):
    """A Batch with keys (and values) set by edit(i, k, v, rng) and queries q."""
    rng = np.random.default_rng(seed + 1000)
    b = Batch(seqs, Hq, Hk, D, page, seed=seed, edit=lambda i, k, v: edit(i, k, v, rng))
    b.q, b.window, b.scale = q, window, D ** -0.5 if scale is None else scale
    return b


def expected(b, i, softmax=None):
    """(result, bound) of sequence i; `softmax` in place of the oracle's: f(scores [n][Hq][L], seen [n][L]) -> weights."""
    n, L = b.seqs[i]
    q = b.q[b.starts[i]:b.starts[i] + n].float().numpy().astype(np.float64)
    K, V = b.kv[i]
    g = b.Hq // b.Hk
    s = np.einsum("nhgd,jhd->nhgj", q.reshape(n, b.Hk, g, b.D), K).reshape(n, b.Hq, L) * b.scale
    at, j = L - n + np.arange(n)[:, None], np.arange(L)
    seen = (j <= at) & ((j > at - b.window) | (b.window == 0))
    w = softmax_of(s, seen) if softmax is None else softmax(s, seen)
    out = np.einsum("nhgj,jhd->nhgd", w.reshape(n, b.Hk, g, L), V).reshape(n, b.Hq, b.D)
    top = np.repeat(np.abs(V).max(-1), g, axis=1).T  # [Hq][L]
    mag = (w * top).sum(-1)
    ref = np.einsum("nhgd,jhd->nhgj", np.abs(q).reshape(n, b.Hk, g, b.D), np.abs(K)).reshape(n, b.Hq, L) * abs(b.scale)
    ref = np.where(seen[:, None], ref, 0).max(-1, initial=0)
    return out, kv.tolerance(out, mag, ref, KEYS)


def softmax_of(s, seen):
    s = np.where(seen[:, None], s, -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    w = np.where(seen[:, None], np.exp(s - np.where(np.isfinite(top), top, 0)), 0)
    return w / np.maximum(w.sum(-1, keepdims=True), 1e-300)


def check(b, got):
    """got: fp64 [T][Hq][D]."""
    for i, (n, L) in enumerate(b.seqs):
        ref, tol = expected(b, i)
        err = np.abs(got[b.starts[i]:b.starts[i] + n] - ref)
        assert np.all(err <= tol), f"sequence {i} (n {n}, L {L}): off by {np.nanmax(err / np.maximum(tol, 1e-300)):.2f} of the bound"


# ------------------------------------------------------------------ cases that a wrong reference of the softmax fails
def sharp():
    """Scores of some tens to a hundred: the softmax is a few keys."""
    def edit(i, k, v, rng):
        k[:] = key_rows(rng, k.shape, 0.25)
    seqs = [(1, 500), (2, 90), (70, 300)]
    return case(seqs, 4, 2, 128, 16, edit, query_rows(1, 73, 4, 128), scale=0.5)


def rising():
    """Keys that grow along the cache, so that the reference moves again and again."""
    def edit(i, k, v, rng):
        k[:] = key_rows(rng, k.shape, 1.0) * 2.0 ** np.linspace(-6, 0, len(k)).round()[:, None, None]
        v *= 2.0 ** np.linspace(6, -6, len(v))[:, None, None]
    seqs = [(1, 700), (3, 500), (80, 600)]
    return case(seqs, 4, 2, 128, 16, edit, query_rows(2, 84, 4, 128), scale=1 / 32)


def below_zero(n, L, window):
    """All scores between some -300 and -400 in units of log2, behind a window that hides the first tiles."""
    def edit(i, k, v, rng):
        k[:] = key_rows(rng, k.shape, 0.25, centre=16)
    q = query_rows(n, n, 4, 64, most=1) / 2 - 1
    return case([(n, L)], 4, 2, 64, 16, edit, q, window, 5 / 8, seed=n)


def jumps(at, n, L):
    """Keys far above all before them, at the places `at`, each above the last: by 0, 12, 24 .. 48 binades for query heads
    and rows of their own. Their values are small, so that what came before them counts where it was scaled right."""
    def edit(i, k, v, rng):
        k[:] = key_rows(rng, k.shape, 2.0 ** -6)
        k[:, :, 2:18] = 0
        v *= 4
        for x, j in enumerate(at):
            k[j] = 0
            k[j, :, 2:18] = x + 1  # 16 channels: a score of 16 level (x + 1) scale
            v[j] *= 2.0 ** -12
    q = query_rows(3, n, 4, 128)
    q[:, :, 2:18] = (torch.arange(n)[:, None] + 2 * torch.arange(4)).remainder(5)[:, :, None] / 4
    return case([(n, L)], 4, 2, 128, 16, edit, q, scale=2.0, seed=sum(at))


CASES = {"sharp": sharp, "rising": rising}
CASES.update({f"below zero {a}": (lambda a=a: below_zero(*a)) for a in [(1, 300, 0), (2, 300, 40), (100, 400, 60), (200, 200, 0)]})
CASES.update({f"jumps {at} {n}": (lambda at=at, n=n, L=L: jumps(at, n, L))
              for at in ([5], [60], [64], [100], [127, 200], [130, 193, 260], [70, 140, 210, 280])
              for n, L in [(40, 300), (100, 330), (2, 300)]})
