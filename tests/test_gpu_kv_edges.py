"""Attention over the 4-bit cache at the edges of its numbers and of its caller's tables."""
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
@pytest.mark.parametrize("n", [1, 4])
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
