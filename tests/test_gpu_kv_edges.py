"""The 4-bit cache and its attention at the edges of their numbers and of their caller's tables and buffers."""
import numpy as np
import pytest
import torch

from oracle import kv
from quantized_linear_error_gb300 import spear

from . import kv_cases
from .test_gpu_kv_attention import Batch

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _leftovers(D, word):
    """Fills the kernels' shared memory with blocks whose parameter pairs are `word`."""
    for n in (1, 100):
        pool = torch.zeros(2, 8, 128 * (D + 8), dtype=torch.uint8, device="cuda").view(torch.int32)
        pool.fill_(word)
        c = spear.SpearKVCache(8, 8, D, 128, pool.view(torch.uint8))
        q = torch.zeros(100 * n, 8, D, dtype=torch.bfloat16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        c.attention(q, torch.empty_like(q), torch.arange(2, **i32).repeat(100, 1), torch.full((100,), 256, **i32),
                    torch.arange(0, 100 * n + 1, n, **i32), n)
        assert c.check() == spear.SPEAR_OK


# ---------------------------------------------------------------------------------- exact scores
@pytest.mark.parametrize("name", kv_cases.CASES)
def test_scores_held_exactly(name):
    """The reference of the running sums, where a score's own rounding leaves the bound no room."""
    b = kv_cases.CASES[name]()
    got = b.run(window=b.window, scale=b.scale)
    assert b.c.check() == spear.SPEAR_OK
    kv_cases.check(b, _f64(got))


# ---------------------------------------------------------------------------------- past the end of a sequence
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 40])
def test_what_lies_past_the_end_changes_no_bit(D, n):
    """Free slots of a sequence's last block, blocks past it that were never copied, and keys before the window: zeros, NaN,
    scales that 16-bit weights take and scales that they do not."""
    for window in (0, 24):
        seqs = [(n, L) for L in (n, n + 1, n + 15, 56, 65, 100, 131)]
        first = None
        for fill, word in ((0x00, 0x3F803F80), (0xFF, 0), (0x3F, 0x7FC07FC0), (0x50, 0x3F803F80), (0x3F, 0x50505050)):
            b = Batch(seqs, 8, 2, D, 16, seed=7)
            blank = np.zeros_like(b.pool)
            for i, (_, L) in enumerate(seqs):
                lo = max(0, L - n - window + 1) if window else 0
                j = np.arange(lo, L)
                slots = b.table[i, j // 16].astype(np.int64) * 16 + j % 16
                ones = np.full((len(j), 2, D), 15, np.uint8)
                kv.pack_rows(blank, 16, D, slots, ones, np.full((len(j), 2, 2), 0xFFFF), ones, np.full((len(j), 2, 2), 0xFFFF))
            b.pool = np.where(blank != 0, b.pool, np.uint8(fill))
            _leftovers(D, word)
            got = b.run(window=window)
            first = got if first is None else first
            assert torch.equal(got, first), (window, hex(fill), hex(word), [
                L for i, (_, L) in enumerate(seqs) if not torch.equal(got[i * n:i * n + n], first[i * n:i * n + n])])


# ---------------------------------------------------------------------------------- small weights
def _shared_cache(b, copies):
    """The one sequence of b, `copies` times over the same pages with the same queries, so that every CTA has whole items."""
    n, L = b.seqs[0]
    c = spear.SpearKVCache(b.Hq, b.Hk, b.D, b.page, _dev(b.pool))
    q = b.q.cuda().repeat(copies, 1, 1)
    out = torch.empty_like(q)
    c.attention(q, out, _dev(b.table).repeat(copies, 1), _dev(np.full(copies, L, np.int32)),
                _dev(np.arange(copies + 1, dtype=np.int32) * n), n, scale=b.scale)
    assert c.check() == spear.SPEAR_OK
    return out.view(copies, n, b.Hq, b.D)


def test_small_weights_of_small_values_few_rows():
    """Keys that hold nearly all of the weight, and whose values are small, before thousands with weights near 2^-17 and
    values of size 0.01 with a channel of one sign: their sum is a third of the result."""
    L, D, Hk = 16384, 128, 8
    def edit(i, k, v, rng):
        k[:] = kv_cases.key_rows(rng, k.shape, 2.0 ** -5)
        k[:, :, 2:18] = 0
        v[:] = rng.normal(size=v.shape)
        v[:, :, 0] = 3
        v *= 0.01
        for j in (0, 33, 70, 100):  # one for each warp's keys of a tile
            k[j], v[j] = 0, v[j] * 0.02
            k[j, :, 2:18] = 1.0
    b = kv_cases.case([(1, L)], Hk, Hk, D, 64, edit, kv_cases.query_rows(5, 1, Hk, D, most=2), scale=0.75)
    b.q[:, :, 2:18] = 1.0
    out = _shared_cache(b, 60)
    for s in (0, 30, 59):
        kv_cases.check(b, _f64(out[s]))


@pytest.mark.parametrize("D,bits", [(64, 21.4), (128, 22.6)])
def test_small_weights_in_a_chunk(D, bits):
    """One key holds nearly all of the weight and its value is 0; thousands behind it have weights of 2^-bits, alike, and
    are all of the result."""
    n, L = 80, 6000
    def edit(i, k, v, rng):
        k[:] = 0
        k[0, :, 2:18], v[0] = 1.0, 0
    q = kv_cases.query_rows(5, n, 2, D, most=2)
    q[:, :, 2:18] = 1.0
    b = kv_cases.case([(n, L)], 2, 1, D, 64, edit, q, scale=bits * np.log(2) / 16)
    out = _shared_cache(b, 200)
    for s in (0, 100, 199):
        kv_cases.check(b, _f64(out[s]))


def test_value_scales_of_every_size_in_one_cache():
    """Blocks of values that grow and shrink by 2^5 to 2^40 from one to the next, and single rows among them."""
    for step in (5, 20, 40, -5, -20, -40):
        def edit(i, k, v, rng):
            k[:] = kv_cases.key_rows(rng, k.shape, 2.0 ** -5)
            e = (np.arange(len(v)) // 32 % 2 if abs(step) > 20 else np.arange(len(v)) // 96 % 4) * step
            e[7::50] = rng.integers(-40, 41, len(e[7::50]))
            v *= 2.0 ** e[:, None, None]
        for n in (1, 4, 60):
            b = kv_cases.case([(n, 700), (n, 90)], 4, 2, 64, 16, edit, kv_cases.query_rows(n, 2 * n, 4, 64), seed=step + 40)
            got = b.run(scale=b.scale)
            assert b.c.check() == spear.SPEAR_OK
            kv_cases.check(b, _f64(got))


@pytest.mark.parametrize("n", [1, 4, 60])
def test_large_constant_values_among_tiny_ones(n):
    """Every second row is one value of 2^60 (scale 0) in a cache whose other values are of size 2^-56: sums stay finite."""
    def edit(i, k, v, rng):
        k[:] = kv_cases.key_rows(rng, k.shape, 2.0 ** -5)
        v *= 2.0 ** -56
        v[1::2] = 2.0 ** 60
    b = kv_cases.case([(n, 9000)], 4, 2, 64, 16, edit, kv_cases.query_rows(n, n, 4, 64))
    got = b.run(scale=b.scale)
    assert b.c.check() == spear.SPEAR_OK
    kv_cases.check(b, _f64(got))


# ---------------------------------------------------------------------------------- released pages
@pytest.mark.parametrize("n,L,window,D,page", [(1, 500, 100, 128, 16), (4, 777, 64, 64, 48), (1, 1000, 1, 128, 32),
                                               (100, 700, 128, 128, 16), (300, 1500, 200, 64, 32), (90, 900, 17, 128, 64)])
def test_pages_before_the_window_may_be_released(n, L, window, D, page):
    """Pages that no query row sees any more stand as -1 in the table, and nothing of them is looked at."""
    _leftovers(D, 0x7FC07FC0)
    seqs = [(n, L), (n, L - 130), (n, L - 5)]
    b = Batch(seqs, 4, 2, D, page, seed=n)
    for i, (_, length) in enumerate(seqs):
        b.table[i, :max(0, length - n - window + 1) // page] = -1
    b.check(b.run(window=window), window)


# ---------------------------------------------------------------------------------- long segments
def test_items_that_take_longer_than_a_wait():
    """Six row tiles a CTA, each over 12 million keys (the same page again and again): a tile takes over 100 ms."""
    D, page, L, n = 64, 4096, 12 << 20, 256
    Hk = 6 * torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator("cuda").manual_seed(1)
    pool = spear.kv_pool(1, Hk, D, page)
    c = spear.SpearKVCache(Hk, Hk, D, page, pool)
    for at in range(0, page, 256):
        k, v = (torch.randn(256, Hk, D, device="cuda", generator=gen).bfloat16() for _ in range(2))
        c.append(None, k, v, None, torch.arange(at, at + 256, device="cuda"))
    q = torch.randn(n, Hk, D, device="cuda", generator=gen).bfloat16()
    out = torch.empty_like(q)
    i32 = dict(dtype=torch.int32, device="cuda")
    c.attention(q, out, torch.zeros(1, L // page, **i32), torch.tensor([L], **i32), torch.tensor([0, n], **i32), n)
    assert c.check() == spear.SPEAR_OK
    host = pool.cpu().numpy()
    for h in (0, 7, Hk - 1):
        K, V = kv.unpack_rows(host[:, h:h + 1], page, D, np.arange(page))
        # the last rows see all but a few of the keys, each page's keys L / page times
        ref, mag, big = kv.attention(_f64(q[-1:, h:h + 1]), K, V, D ** -0.5)
        assert np.all(np.abs(_f64(out[-1:, h:h + 1]) - ref) <= kv.tolerance(ref, mag, big) + 1e-5)


# ---------------------------------------------------------------------------------- queries
@pytest.mark.parametrize("n", [1, 4, 90])
def test_huge_queries_and_tiny_keys(n):
    """Rows of 1e30 to 2e35 whose products with the keys are ordinary numbers, and the other way round."""
    for size in (1e30, 5e34, 1e-30):
        def edit(i, k, v):
            k /= size
        b = Batch([(n, 200)], 8, 2, 128, 16, seed=n, edit=edit)
        b.q = (b.q.float() * size).bfloat16()
        b.check(b.run())


@pytest.mark.parametrize("n", [1, 4, 90])
def test_rows_with_infinities_are_nan(n):
    """Also where every score is minus infinity; a row that sees no key stays zero."""
    def edit(i, k, v):
        np.abs(k, out=k)
    b = Batch([(n, 200), (n, 0)], 4, 2, 64, 16, seed=n, edit=edit)
    b.q[0, 1], b.q[0, 2, 9], b.q[n, 0] = -float("inf"), -float("inf"), float("inf")
    got = b.run().float()
    assert torch.isnan(got[0, 1:3]).all() and torch.isfinite(got[0, [0, 3]]).all() and torch.isfinite(got[1:n]).all()
    assert not got[n:].any()


def test_a_row_of_one_infinity_is_nan_wherever_it_stands():
    """In every element and of either sign, also where no key's code is 0 there, so that all scores are the same infinity."""
    for n in (1, 3, 40):
        def edit(i, k, v):
            k[:] = 1.0 + 15 * (np.arange(64) != i)  # codes 0 in one channel alone, 15 in the others
        seqs = [(n, n + 2)] * 64
        b = Batch(seqs, 2, 1, 64, 16, seed=n, edit=edit)
        for sign in (1, -1):
            for i in range(64):
                b.q[b.starts[i]:b.starts[i + 1], 1] = 0.5
                b.q[b.starts[i]:b.starts[i + 1], 1, (i + 1) % 64] = sign * float("inf")
            got = b.run().float()
            assert torch.isnan(got[:, 1]).all(), (n, sign, (~torch.isnan(got[:, 1])).any(-1).nonzero().flatten().tolist())
            assert torch.isfinite(got[:, 0]).all()


# ---------------------------------------------------------------------------------- arguments
def test_query_and_result_in_one_row_buffer():
    """Neighbouring columns of the same rows do not overlap; columns that do are refused."""
    for n in (1, 40):
        b = Batch([(n, 100), (n, 90)], 4, 2, 64, 16)
        want = b.run()
        rows = torch.zeros(2 * n, 13, 64, dtype=torch.bfloat16, device="cuda")
        for at, to in ((0, 4), (8, 1), (1, 9)):
            q, out = rows[:, at:at + 4], rows[:, to:to + 4]
            q.copy_(b.q)
            args = (_dev(b.table), _dev(np.array([100, 90], np.int32)), _dev(b.starts), n)
            assert torch.equal(b.c.attention(q, out, *args), want)
            for clash in (rows[:, at + 1:at + 5], rows[:, at + 3:at + 7] if at + 7 <= 13 else rows[:, at - 1:at + 3]):
                with pytest.raises(spear.SpearError):
                    b.c.attention(q, clash, *args)


def test_rotated_queries_that_overlap_what_is_read_are_refused():
    """A result that shares elements with q (but is not q), k or v would be a race; neighbouring columns are none."""
    c = spear.SpearKVCache(4, 2, 64, 16, spear.kv_pool(1, 2, 64, 16), spear.rope_table(8, 64))
    for T in (1, 3):
        rows = torch.randn(T, 16, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).bfloat16()
        pos, slots = torch.arange(T, device="cuda"), torch.full((T,), -1, device="cuda")
        q, k, v = rows[:, :4].clone(), rows[:, 4:6].clone(), rows[:, 6:8].clone()
        want = c.append(q, k, v, pos, slots, torch.empty_like(q))
        q, k, v = rows[:, :4], rows[:, 4:6], rows[:, 6:8]
        assert torch.equal(c.append(q, k, v, pos, slots, rows[:, 8:12]), want)
        for at in (1, 2, 3, 4, 5, 7):
            with pytest.raises(spear.SpearError):
                c.append(q, k, v, pos, slots, rows[:, at:at + 4])
        flat = rows.view(-1)
        with pytest.raises(spear.SpearError):  # another stride from the same place
            c.append(q, k, v, pos, slots, flat[64:64 + T * 4 * 64].view(T, 4, 64))
        assert torch.equal(c.append(q, k, v, pos, slots), want)
        with pytest.raises(spear.SpearError):
            c.read(slots, flat[:T * 128].view(T, 2, 64), flat[64:64 + T * 128].view(T, 2, 64))
        with pytest.raises(spear.SpearError):
            c.read(slots, flat[:T * 128].view(T, 2, 64), flat[:T * 128].view(T, 2, 64))
        c.read(slots, flat[:T * 128].view(T, 2, 64), flat[T * 128:T * 256].view(T, 2, 64))
    assert c.check() == spear.SPEAR_OK


def test_strides_of_a_single_token():
    """The stride of one token is of no account, in whatever tensor it stands."""
    b = Batch([(1, 100)], 4, 2, 64, 16)
    want = b.run()
    q = b.q.cuda()
    for stride in (0, 1, 64, 300, 4 * 64 + 3):
        odd = lambda x: torch.as_strided(x, x.shape, (stride, 64, 1), x.storage_offset())
        out = torch.empty_like(q)
        args = (_dev(b.table), _dev(np.array([100], np.int32)), _dev(b.starts), 1)
        b.c.attention(odd(q), odd(out), *args)
        assert torch.equal(out, want)
        k = torch.randn(1, 2, 64, device="cuda").bfloat16()
        b.c.append(odd(q), odd(k), odd(k), None, torch.tensor([-1], device="cuda"), odd(out))
        assert torch.equal(out, q)
    assert b.c.check() == spear.SPEAR_OK


def test_numbers_past_32_bits():
    """A window or a row count that no 32-bit number holds means what it says."""
    b = Batch([(1, 100), (2, 90)], 4, 2, 64, 16)
    want = b.run()
    for big in (1 << 31, (1 << 32) + 5, 1 << 40):
        assert torch.equal(b.run(window=big), want)
        assert torch.equal(b.run(max_q=big), want)
    for low in (-1, -(1 << 31), -(1 << 32) + 7):
        for kw in (dict(window=low), dict(max_q=low)):
            with pytest.raises(spear.SpearError):
                b.run(**kw)


def test_a_new_handle_is_ready_for_any_stream():
    """Its workspace has been cleared when the constructor returns, whatever the stream had to do before."""
    pool, side = spear.kv_pool(1, 2, 64, 16), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a = torch.randn(8192, 8192, device="cuda")
        for _ in range(20):
            a @ a
        c = spear.SpearKVCache(4, 2, 64, 16, pool)
    assert side.query() and c.check() == spear.SPEAR_OK
