"""Refusals of the key/value cache calls that need no GPU: every bad descriptor and argument is turned down before
the device is touched."""
import ctypes

import pytest

from quantized_linear_error_gb300 import build, spear


@pytest.fixture(scope="module")
def L():
    build.build()
    return spear.load()


def _desc(**kw):
    d = dict(n_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=4, pool=4096, rope_dim=128,
             rope_interleaved=0, n_positions=64, rope_table=4096)
    d.update(kw)
    return spear.spear_kv_desc_t(*[d[f] for f, _ in spear.spear_kv_desc_t._fields_])


@pytest.mark.parametrize("bad", [dict(n_heads=0), dict(n_heads=7), dict(n_kv_heads=0), dict(n_heads=66), dict(n_heads=8192, n_kv_heads=1024), dict(head_dim=96),
                                 dict(n_heads=1, n_kv_heads=2), dict(n_heads=-8, n_kv_heads=-2),
                                 dict(head_dim=256), dict(page_size=0), dict(page_size=24), dict(page_size=65552),
                                 dict(n_pages=0), dict(pool=None), dict(pool=4104), dict(rope_dim=8), dict(rope_dim=144),
                                 dict(rope_dim=-16), dict(rope_table=None), dict(rope_table=4104), dict(n_positions=0),
                                 dict(head_dim=64)])
def test_create_rejects_bad_descriptor(L, bad):
    h = ctypes.c_void_p(1234)
    assert L.spear_kv_create(ctypes.byref(_desc(**bad)), None, ctypes.byref(h)) == spear.SPEAR_ERR_INVALID_ARG
    assert h.value is None


def test_null_arguments(L):
    h = ctypes.c_void_p()
    assert L.spear_kv_create(None, None, ctypes.byref(h)) == spear.SPEAR_ERR_INVALID_ARG
    assert L.spear_kv_create(ctypes.byref(_desc()), None, None) == spear.SPEAR_ERR_INVALID_ARG
    assert L.spear_kv_append(None, 16, 8, 16, 8, 16, 8, 16, 16, 1, 16, 8, None) == spear.SPEAR_ERR_INVALID_ARG
    assert L.spear_kv_read(None, 16, 1, 16, 16, None) == spear.SPEAR_ERR_INVALID_ARG
    assert L.spear_kv_attention(None, 16, 8, 16, 8, 16, 1, 16, 16, 1, 1, 1, 1.0, 0, None) == spear.SPEAR_ERR_INVALID_ARG
    assert L.spear_kv_check(None, None) == spear.SPEAR_ERR_INVALID_ARG
    assert L.spear_kv_destroy(None) == spear.SPEAR_OK


def test_page_bytes():
    assert spear.kv_page_bytes(8, 128, 64) == 8 * 64 * 136
    assert spear.kv_page_bytes(1, 64, 16) == 16 * 72
