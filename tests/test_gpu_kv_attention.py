"""Attention over the paged 4-bit cache against the fp64 oracle, within the bound that the oracle derives."""
import numpy as np
import pytest
import torch

from oracle import kv
from quantized_linear_error_gb300 import spear

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences of given (new tokens, cached tokens) over a shuffled pool whose unused bytes are 0xFF (codes 15,
    parameters NaN), with keys and values quantised from normal draws."""

    def __init__(self, seqs, Hq, Hk, D, page, seed=0, k_std=1.0, edit=None):
        rng = np.random.default_rng(seed)
        self.seqs, self.Hq, self.Hk, self.D, self.page = seqs, Hq, Hk, D, page
        per = [-(-max(L, 0) // page) for _, L in seqs]
        n_pages = sum(per) + 2
        perm, at = rng.permutation(n_pages), 0
        self.pool = np.full((n_pages, Hk, page * (D + 8)), 0xFF, np.uint8)
        self.table = np.full((len(seqs), max(1, max(per))), -1, np.int32)  # entries past a sequence's pages are not read
        self.kv = []
        for i, (n, L) in enumerate(seqs):
            self.table[i, :per[i]] = perm[at:at + per[i]]
            at += per[i]
            k = (rng.normal(size=(L, Hk, D)) * k_std).astype(np.float32)
            v = rng.normal(0.5, 1, size=(L, Hk, D)).astype(np.float32)
            if edit:
                edit(i, k, v)
            j = np.arange(L)
            slots = self.table[i, j // page].astype(np.int64) * page + j % page
            kv.pack_rows(self.pool, page, D, slots, *kv.quantise(k), *kv.quantise(v))
            self.kv.append(kv.unpack_rows(self.pool, page, D, slots))
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        T = int(self.starts[-1])
        g = torch.Generator().manual_seed(seed)
        self.q = torch.randn(T, Hq, D, generator=g).bfloat16()
        self.max_q = max(n for n, _ in seqs)

    def run(self, window=0, scale=None, ld_q=None, cache=None, max_q=None):
        dev = lambda a: torch.from_numpy(a).cuda()
        self.c = cache or spear.SpearKVCache(self.Hq, self.Hk, self.D, self.page, dev(self.pool))
        T = self.q.shape[0]
        q = torch.zeros(T, (ld_q or self.Hq * self.D), dtype=torch.bfloat16, device="cuda")[:, :self.Hq * self.D].view(T, self.Hq, self.D)
        q.copy_(self.q)
        out = torch.full((T, self.Hq, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.c.attention(q, out, dev(self.table), dev(np.array([L for _, L in self.seqs], np.int32)), dev(self.starts),
                         max_q or self.max_q, scale=scale, window=window)
        return out

    def check(self, out, window=0, scale=None):
        assert self.c.check() == spear.SPEAR_OK
        got = out.float().cpu().numpy().astype(np.float64)
        for i, ((n, L), (K, V)) in enumerate(zip(self.seqs, self.kv)):
            rows = slice(self.starts[i], self.starts[i] + n)
            ref, mag, big = kv.attention(self.q[rows].float().numpy().astype(np.float64), K, V,
                                         self.D ** -0.5 if scale is None else scale, window)
            err, tol = np.abs(got[rows] - ref), kv.tolerance(ref, mag, big)
            assert np.all(err <= tol), f"sequence {i} (n {n}, L {L}): off by {np.nanmax(err / tol):.2f} of the bound"


def _check(seqs, Hq, Hk, D, page, window=0, scale=None, **kw):
    b = Batch(seqs, Hq, Hk, D, page, **kw)
    b.check(b.run(window, scale), window, scale)


@pytest.mark.parametrize("Hq,Hk,D,page", [(8, 2, 128, 16), (4, 4, 64, 32), (32, 1, 128, 48), (7, 1, 64, 16),
                                          (24, 2, 128, 64), (2, 2, 128, 256), (16, 1, 64, 128), (3, 1, 128, 16)])
def test_single_tokens(Hq, Hk, D, page):
    """One new token a sequence; lengths around tile, block and page ends, one and none."""
    _check([(1, L) for L in (1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300)] + [(1, 0)], Hq, Hk, D, page)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 129, 1000])
def test_single_tokens_window(window):
    _check([(1, L) for L in (1, 16, 17, 100, 129, 228, 257, 500)], 8, 2, 128, 32, window=window)


@pytest.mark.parametrize("n,Hq,Hk,D,page,window", [(2, 8, 2, 128, 16, 0), (4, 8, 2, 128, 64, 0), (5, 4, 4, 64, 16, 3),
                                                   (8, 4, 1, 128, 32, 0), (7, 3, 1, 64, 48, 50), (2, 32, 2, 128, 16, 0),
                                                   (3, 10, 1, 128, 16, 140)])
def test_a_few_tokens(n, Hq, Hk, D, page, window):
    """Drafts to verify: each row its own last key, cached lengths down to fewer than the new tokens' number."""
    _check([(n, L) for L in (n, n + 1, 17, 40, 128, 131, 300)] + [(1, 77), (n, 1), (n, 0)], Hq, Hk, D, page, window=window)


@pytest.mark.parametrize("n,L,Hq,Hk,D,page,window", [
    (33, 33, 4, 1, 128, 16, 0), (40, 100, 8, 8, 64, 32, 0), (64, 64, 8, 2, 128, 64, 0), (100, 357, 8, 1, 128, 16, 0),
    (128, 128, 4, 4, 128, 128, 0), (129, 640, 4, 4, 64, 16, 0), (257, 300, 2, 1, 128, 48, 0), (200, 513, 7, 1, 64, 256, 0),
    (300, 1000, 2, 2, 128, 16, 90), (90, 91, 3, 1, 128, 16, 1), (150, 700, 12, 4, 128, 32, 128), (70, 30, 4, 4, 128, 16, 0),
    (200, 0, 4, 2, 64, 16, 0), (300, 170, 2, 1, 64, 64, 40), (513, 513, 1, 1, 128, 16, 0)])
def test_chunks(n, L, Hq, Hk, D, page, window):
    """Prefill chunks: rows and keys around tile ends, GQA rows of one token in several tiles, rows without a key."""
    _check([(n, L)], Hq, Hk, D, page, window=window)


@pytest.mark.parametrize("Hq,Hk,D,window", [(8, 2, 128, 0), (4, 4, 64, 0), (8, 1, 128, 100)])
def test_mixed_batches(Hq, Hk, D, window):
    """Single tokens, drafts and chunks of one step in one call, in any order, empty sequences among them."""
    _check([(1, 200), (60, 260), (0, 50), (1, 1), (4, 64), (129, 129), (1, 0), (0, 0), (34, 500), (2, 350), (1, 400)],
           Hq, Hk, D, 16, window=window)


def test_many_sequences():
    _check([(1, 1 + 7 * i % 90) for i in range(300)], 4, 2, 64, 16)


def test_many_chunks():
    """Many sequences of a few row tiles, and among them one of so many that they are counted in another way; more
    sequences than a warp's lanes."""
    short = [(5 + 7 * i % 60, 70 + 11 * i % 200) for i in range(20)]
    _check(short + [(1400, 1401)], 8, 1, 64, 32)
    _check(short + [(0, 5)] + short + [(700, 720)] + short[:3], 8, 1, 64, 32, window=200)


def test_work_split_over_a_long_cache():
    _check([(1, 20001)], 4, 1, 128, 64, seed=3)
    _check([(3, 9000), (1, 11), (40, 6000)], 4, 1, 64, 128, seed=4)


def test_scale_and_sharp_scores():
    """Scores of some hundreds: the softmax is all but one key; and scale 0 is the plain mean."""
    _check([(1, 500), (2, 90), (70, 300)], 4, 2, 128, 16, k_std=6.0, scale=0.5)
    _check([(1, 500), (70, 300)], 4, 2, 128, 16, scale=0.0)


def test_rising_scores():
    """Keys whose scores climb along the cache, so that the running maximum moves at every tile."""
    def edit(i, k, v):
        k *= np.linspace(0.01, 12, len(k))[:, None, None]
    _check([(1, 700), (3, 500), (80, 600)], 4, 2, 128, 16, edit=edit)


def test_masked_places_do_not_leak():
    """Keys and values that a row must not see are huge or NaN: later tokens of the chunk, keys before the window."""
    for n, L, window, bad in [(4, 300, 0, [298, 299]), (1, 300, 20, [100, 279]), (70, 200, 0, [190, 199]),
                              (100, 400, 30, [3, 200, 270])]:
        for what in (1e30, np.nan, np.inf):
            def edit(i, k, v):
                if i == 0:
                    k[bad], v[bad] = what, what
            b = Batch([(n, L), (1, 50)], 4, 2, 128, 16, seed=5, edit=edit)
            got = b.run(window=window).float().cpu().numpy()
            for r in range(n):
                p = L - n + r
                lo = max(0, p - window + 1) if window else 0
                if any(lo <= j <= p for j in bad):
                    if not np.isfinite(what):
                        assert np.isnan(got[r]).all()
                    continue
                ref, mag, big = kv.attention(b.q[r:r + 1].float().numpy().astype(np.float64), b.kv[0][0][lo:p + 1],
                                             b.kv[0][1][lo:p + 1], 128 ** -0.5)
                assert np.all(np.abs(got[r] - ref[0]) <= kv.tolerance(ref, mag, big)[0]), (n, window, what, r)
            assert np.isfinite(got[n:]).all()


def test_strided_queries_and_output_in_place():
    b = Batch([(1, 100), (40, 90)], 4, 2, 64, 16)
    b.check(b.run(ld_q=4 * 64 + 8))
    dev = lambda a: torch.from_numpy(a).cuda()
    q = b.q.cuda()
    b.c.attention(q, q, dev(b.table), dev(np.array([100, 90], np.int32)), dev(b.starts), 40)
    b.check(q)


def test_repeated_calls_give_the_same_bits():
    """Partial results are joined in a fixed order; counters are left as they were found."""
    b = Batch([(1, 5000), (2, 3000), (64, 2000)], 4, 1, 128, 16)
    first = b.run()
    for _ in range(5):
        assert torch.equal(b.run(cache=b.c), first)
    assert b.c.check() == spear.SPEAR_OK


def test_in_a_graph_and_on_another_stream():
    """Captured once, replayed with longer lengths, on a stream of its own."""
    b = Batch([(1, 600), (1, 60)], 8, 2, 128, 16)
    dev = lambda a: torch.from_numpy(a).cuda()
    c = spear.SpearKVCache(8, 2, 128, 16, dev(b.pool))
    q, table, starts = b.q.cuda(), dev(b.table), dev(b.starts)
    lens = dev(np.array([10, 20], np.int32))
    out = torch.empty_like(q)
    c.attention(q, out, table, lens, starts, 1)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.attention(q, out, table, lens, starts, 1)
    lens.copy_(dev(np.array([600, 60], np.int32)))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    b.c = c
    b.check(out)


def test_indices_out_of_range_are_reported():
    """Page numbers and lengths that the host cannot see: an error status, no fault, other sequences unharmed."""
    for n in (1, 40):
        b = Batch([(n, 100), (n, 90), (n, 33)], 4, 2, 128, 16)
        b.table[0, 3] = len(b.pool)
        b.table[0, 5] = -7
        got = b.run()
        assert b.c.check() == spear.SPEAR_ERR_INVALID_ARG and b.c.check() == spear.SPEAR_OK
        b.seqs, b.kv, b.starts, b.q = b.seqs[1:], b.kv[1:], b.starts[:-1], b.q[n:]
        b.check(got[n:])
        b = Batch([(n, 100), (n, 90)], 4, 2, 128, 16)
        dev = lambda a: torch.from_numpy(a).cuda()
        c = spear.SpearKVCache(4, 2, 128, 16, dev(b.pool))
        q = b.q.cuda()
        out = torch.zeros_like(q)
        c.attention(q, out, dev(b.table), dev(np.array([1 << 30, -5], np.int32)), dev(b.starts), n)
        assert c.check() == spear.SPEAR_ERR_INVALID_ARG


def test_refusals():
    b = Batch([(1, 20)], 4, 2, 64, 16)
    b.run()
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    good = dict(q=q, out=torch.empty_like(q), page_table=i(0, 1).view(1, 2), kv_lens=i(20), q_starts=i(0, 1), max_q=1)
    b.c.attention(**good)
    for bad in [dict(q=q.half()), dict(out=torch.empty(2, 4, 64, dtype=torch.bfloat16, device="cuda")), dict(page_table=i(0, 1)),
                dict(kv_lens=i(20).long()), dict(q_starts=i(0)), dict(q=q[:, :3])]:
        with pytest.raises(ValueError):
            b.c.attention(**{**good, **bad})
    for bad in [dict(max_q=0), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf"))]:
        with pytest.raises(spear.SpearError):
            b.c.attention(**{**good, **bad})
    two = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(spear.SpearError):
        b.c.attention(**{**good, "q": two[:3], "out": two[1:], "q_starts": i(0, 3), "max_q": 3})


def test_scores_that_jump_inside_a_tile():
    """One key far above all before it, at every place in a tile of 128 keys: the reference of the running sums moves
    at the first or the second 64 keys of a tile, once or several times, for some rows and not for others."""
    for at in ([5], [60], [64], [100], [127, 200], [130, 193, 260], [70, 140, 210, 280]):
        def edit(i, k, v):
            k *= 0.05
            for x, j in enumerate(at):
                k[j] *= 400.0 * (x + 1)
        for n, L in [(40, 300), (100, 330), (2, 300)]:
            _check([(n, L)], 4, 2, 128, 16, edit=edit, seed=sum(at))


def test_scores_far_below_zero():
    """All scores at some -400 in units of log2, behind a window that hides the first tiles from most rows."""
    def edit(i, k, v):
        k[:] = np.abs(k) + 5
    for n, L, window in [(1, 300, 0), (100, 400, 60), (200, 200, 0)]:
        b = Batch([(n, L)], 4, 2, 64, 16, edit=edit, seed=n)
        b.q = -b.q.abs() - 1
        b.check(b.run(window=window, scale=1.0), window, 1.0)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e-3, 1e3, 1e6, 1e30])
def test_values_of_any_size(size):
    """Values, keys or both of a size that f16 does not hold, all of them or one token's, beside ordinary ones."""
    for n, L in [(1, 300), (3, 200), (80, 300)]:
        for which in ("v", "one v", "k", "one k"):
            def edit(i, k, v):
                if which == "v":
                    v *= size
                elif which == "one v":
                    v[L // 2] *= size
                elif which == "k":
                    k *= size
                else:
                    k[L // 2] *= min(size, 1e3)
            scale = 128 ** -0.5 / (size if which == "k" else 1)
            _check([(n, L)], 4, 2, 128, 16, edit=edit, scale=scale, seed=n)


@pytest.mark.parametrize("n,L", [(1, 200), (4, 200), (90, 200)])
def test_queries_of_any_size(n, L):
    """Rows of zeros, of subnormal and of huge values beside ordinary ones; a negative scale; rows with NaN or
    infinities are NaN, their neighbours are not."""
    b = Batch([(n, L)], 8, 2, 64, 16, seed=n)
    for h, size in enumerate([0.0, 1e-39, 1e-20, 1e-3, 1.0, 1e3, 30.0]):
        b.q[:, h] *= size
    b.check(b.run(scale=-0.1), scale=-0.1)
    b.q[:, 2] *= 1e30
    b.q[0, 3, 5], b.q[0, 4, 7] = float("nan"), float("inf")
    got = b.run().float()
    assert torch.isnan(got[0, 3:5]).all() and torch.isfinite(got[0, [0, 1, 2, 5, 6, 7]]).all() and torch.isfinite(got[1:]).all()
