"""Append and read-back of the paged 4-bit key/value cache against the oracle, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import kv
from quantized_linear_error_gb300 import spear

from .helpers import bits_of

pytestmark = pytest.mark.gpu


def _f32(t):
    return t.float().cpu().numpy()


def _expect(q, k, v, table, positions, interleaved):
    rows = table.cpu().numpy()[positions] if table is not None else np.zeros((len(positions), 0), np.float32)
    return kv.rotate(_f32(q), rows, interleaved), kv.rotate(_f32(k), rows, interleaved), _f32(v)


def _held(codes, par):
    p = kv.bf16_value(par)
    return kv.bf16_bits((codes.astype(np.float32) * p[..., :1] + p[..., 1:]).astype(np.float32))


def _setup(Hq, Hk, D, page, n_pages, rope, interleaved, seed, fill=0xA5):
    pool = spear.kv_pool(n_pages, Hk, D, page)
    pool.fill_(fill)
    table = spear.rope_table(300, rope) if rope else None
    return spear.SpearKVCache(Hq, Hk, D, page, pool, table, interleaved), pool, table, np.random.default_rng(seed)


@pytest.mark.parametrize("T,Hq,Hk,D,page,rope,interleaved", [
    (1, 32, 8, 128, 16, 128, False), (7, 4, 4, 64, 48, 64, False), (33, 28, 4, 128, 64, 64, False),
    (64, 8, 1, 128, 32, 128, True), (129, 6, 2, 64, 16, 32, True), (5, 3, 3, 128, 256, 0, False),
    (300, 2, 1, 64, 128, 16, False), (2, 64, 2, 128, 16, 112, False), (1100, 8, 8, 128, 16, 128, False)])
def test_append_and_read_bit_exact(T, Hq, Hk, D, page, rope, interleaved):
    """Fused-projection rows (strided slices), random slots: queries, cache bytes and read-back are those of the
    definition; bytes of no slot keep their value."""
    n_pages = T // page + 3
    c, pool, table, rng = _setup(Hq, Hk, D, page, n_pages, rope, interleaved, T)
    qkv = (torch.randn(T, Hq + 2 * Hk, D, device="cuda", generator=torch.Generator("cuda").manual_seed(T)) * 2).bfloat16()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[T // 2] = -1
    pos = rng.integers(0, 300, T).astype(np.int64)
    eq, ek, ev = _expect(q, k, v, table, pos, interleaved)
    want = pool.cpu().numpy().copy()
    kc, vc = kv.quantise(ek), kv.quantise(ev)
    kv.pack_rows(want, page, D, slots, *kc, *vc)
    q_out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    ds, dp = torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda()
    c.append(q, k, v, dp, ds, q_out)
    k_out, v_out = torch.empty(T, Hk, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hk, D, dtype=torch.bfloat16, device="cuda")
    c.read(ds, k_out, v_out)
    assert c.check() == spear.SPEAR_OK
    np.testing.assert_array_equal(bits_of(q_out), kv.bf16_bits(eq))
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    on = slots >= 0
    np.testing.assert_array_equal(bits_of(k_out)[on], _held(*kc)[on])
    np.testing.assert_array_equal(bits_of(v_out)[on], _held(*vc)[on])
    assert not bits_of(k_out)[~on].any() and not bits_of(v_out)[~on].any()


def test_queries_in_place_and_left_out():
    c, pool, table, rng = _setup(4, 2, 128, 16, 4, 128, False, 9)
    q, k, v = (torch.randn(5, h, 128, device="cuda").bfloat16() for h in (4, 2, 2))
    pos = torch.arange(5, device="cuda")
    slots = torch.arange(20, 25, device="cuda")
    want = kv.bf16_bits(_expect(q, k, v, table, pos.cpu().numpy(), False)[0])
    c.append(None, k, v, pos, slots)
    first = pool.clone()
    c.append(q, k, v, pos, slots)
    np.testing.assert_array_equal(bits_of(q), want)
    assert torch.equal(pool, first)
    assert c.append(q[:0], k[:0], v[:0], pos[:0], slots[:0]).shape[0] == 0


def test_constant_tiny_and_non_finite_rows():
    """Rows of one value, of subnormal range, with NaN or infinities, of the largest finite values: the parameter
    words of the definition, and no code outside 0..15 of the neighbours."""
    c, pool, table, rng = _setup(2, 1, 64, 16, 1, 0, False, 1)
    x = torch.randn(8, 1, 64, device="cuda")
    x[0], x[1] = 0.0, -3.25
    x[2] = 0.0
    x[2, 0, 0] = 2.0 ** -130
    x[3, 0, 7], x[4, 0, 63], x[5, 0, 0] = float("nan"), float("inf"), float("-inf")
    x[6, 0, :2] = torch.tensor([3.0e38, -3.0e38])
    v = x.bfloat16()
    k = torch.flip(v, [0])
    slots = torch.arange(8, device="cuda")
    want = pool.cpu().numpy().copy()
    kc, vc = kv.quantise(_f32(k)), kv.quantise(_f32(v))
    kv.pack_rows(want, 16, 64, range(8), *kc, *vc)
    c.append(None, k, v, None, slots)
    got = pool.cpu().numpy()
    finite = [0, 1, 2, 7]
    for t in range(8):
        assert np.array_equal(got[0, 0, 1088 + 4 * t:1092 + 4 * t], want[0, 0, 1088 + 4 * t:1092 + 4 * t]), t
        if t in finite:
            assert np.array_equal(got[0, 0, 512 + 32 * t:544 + 32 * t], want[0, 0, 512 + 32 * t:544 + 32 * t]), t
    k_out, v_out = (torch.empty(8, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.read(slots, k_out, v_out)
    assert torch.isnan(v_out[3:7].float()).all() and torch.isfinite(v_out[finite].float()).all()


def test_indices_out_of_range_are_skipped_and_reported():
    """Slots and positions that the host cannot see: nothing is written for them, the rest is, and check says so once."""
    c, pool, table, rng = _setup(2, 1, 128, 16, 2, 128, False, 2)
    q, k, v = (torch.randn(6, h, 128, device="cuda").bfloat16() for h in (2, 1, 1))
    slots = torch.tensor([0, 32, 5, -2, 1 << 40, 7], device="cuda")
    pos = torch.tensor([0, 1, 300, 2, 3, -1], device="cuda")
    q_out = torch.full_like(q, 7.0)
    want = pool.cpu().numpy().copy()
    e = _expect(q, k, v, table, np.zeros(6, np.int64), False)
    kc, vc = kv.quantise(e[1]), kv.quantise(e[2])
    kv.pack_rows(want, 16, 128, [0, -1, -1, -1, -1, -1], *kc, *vc)
    c.append(q, k, v, pos, slots, q_out)
    assert c.check() == spear.SPEAR_ERR_INVALID_ARG and c.check() == spear.SPEAR_OK
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    assert (q_out[1:] == 7.0).all()
    out = torch.empty(2, 1, 128, dtype=torch.bfloat16, device="cuda")
    c.read(torch.tensor([31, 32], device="cuda"), out, torch.empty_like(out))
    assert not out[1].any() and c.check() == spear.SPEAR_ERR_INVALID_ARG


def test_offsets_past_32_bits():
    """A pool of 5 GB: the last page's tokens land where they belong."""
    Hk, D, page = 8, 128, 256
    n_pages = (5 << 30) // spear.kv_page_bytes(Hk, D, page)
    pool = torch.empty(n_pages, Hk, spear.kv_page_bytes(1, D, page), dtype=torch.uint8, device="cuda")
    pool[-1].zero_()
    c = spear.SpearKVCache(Hk, Hk, D, page, pool)
    k, v = (torch.randn(3, Hk, D, device="cuda").bfloat16() for _ in range(2))
    last = n_pages * page
    slots = np.array([last - 1, last - 2, last - 100])
    want = np.zeros((1, Hk, page * (D + 8)), np.uint8)
    kv.pack_rows(want, page, D, slots - (last - page), *kv.quantise(_f32(k)), *kv.quantise(_f32(v)))
    c.append(None, k, v, None, torch.from_numpy(slots).cuda())
    assert c.check() == spear.SPEAR_OK
    np.testing.assert_array_equal(pool[-1:].cpu().numpy(), want)


def test_refusals():
    """Wrong types, shapes, strides and alignments are errors of the call, before anything is launched."""
    pool = spear.kv_pool(2, 2, 64, 16)
    c = spear.SpearKVCache(4, 2, 64, 16, pool, spear.rope_table(8, 64))
    q, k, v = (torch.zeros(3, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    i = torch.zeros(3, dtype=torch.int64, device="cuda")
    for bad in [dict(q=q.float()), dict(q=q[:2]), dict(k=k[:, :1]), dict(v=v.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(positions=None), dict(positions=i.int()), dict(slots=i[:2]), dict(q_out=q[:2]), dict(slots=i.cpu()), dict(k=k.cpu()),
                dict(positions=torch.zeros(6, dtype=torch.int64, device="cuda")[::2])]:
        a = dict(q=q, k=k, v=v, positions=i, slots=i, q_out=None)
        a.update(bad)
        with pytest.raises(ValueError):
            c.append(**a)
    odd = torch.zeros(3 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 2, 64)
    with pytest.raises(spear.SpearError):
        c.append(q, odd, v, i, i)
    with pytest.raises(ValueError):
        spear.SpearKVCache(4, 2, 64, 16, pool[:, :, :-1])
    with pytest.raises(ValueError):
        spear.SpearKVCache(4, 2, 64, 16, pool, spear.rope_table(8, 64).double())
    assert not pool.any()
