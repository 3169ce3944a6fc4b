"""Refusals of the 8-bit calls that need no GPU: every bad descriptor and argument is turned down before the device is
touched."""
import ctypes

import pytest

from quantized_linear_error_gb300 import build, spear

BAD, UNSUPPORTED = spear.SPEAR_ERR_INVALID_ARG, spear.SPEAR_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build()
    return spear.load()


def _desc(**kw):
    d = dict(K=64, N=8, qweight=4096, scales=4096, qweight_up=None, scales_up=None, activation=0, max_tokens=4, workspace=None, workspace_bytes=0)
    d.update(kw)
    return spear.spear_w8_desc_t(*[d[f] for f, _ in spear.spear_w8_desc_t._fields_])


@pytest.mark.parametrize("bad", [dict(K=0), dict(K=8), dict(K=72), dict(K=-64), dict(N=0), dict(N=-8), dict(qweight=None),
                                 dict(qweight=4104), dict(scales=None), dict(scales=4098), dict(max_tokens=0),
                                 dict(qweight_up=4096), dict(scales_up=4096), dict(qweight_up=4100, scales_up=4096),
                                 dict(qweight_up=4096, scales_up=4098),
                                 dict(qweight_up=4096, scales_up=4096, activation=2),
                                 dict(qweight_up=4096, scales_up=4096, activation=-1),
                                 dict(workspace=4096 + 64, workspace_bytes=1 << 30), dict(workspace=4096, workspace_bytes=-1)])
def test_create_rejects_bad_descriptor(L, bad):
    h = ctypes.c_void_p(1234)
    assert L.spear_w8_create(ctypes.byref(_desc(**bad)), None, ctypes.byref(h)) == BAD
    assert h.value is None


@pytest.mark.parametrize("big", [dict(K=(1 << 20) + 16), dict(N=(1 << 22) + 1), dict(max_tokens=(1 << 20) + 1),
                                 dict(K=1 << 20, N=1 << 22)])
def test_create_rejects_sizes_past_the_kernels(L, big):
    h = ctypes.c_void_p(1234)
    assert L.spear_w8_create(ctypes.byref(_desc(**big)), None, ctypes.byref(h)) == UNSUPPORTED
    assert h.value is None


def test_null_arguments(L):
    h = ctypes.c_void_p()
    assert L.spear_w8_create(None, None, ctypes.byref(h)) == BAD
    assert L.spear_w8_create(ctypes.byref(_desc()), None, None) == BAD
    assert L.spear_w8_workspace(None, ctypes.byref(ctypes.c_int64())) == BAD
    assert L.spear_w8_workspace(ctypes.byref(_desc()), None) == BAD
    assert L.spear_w8_workspace(ctypes.byref(_desc(K=8)), ctypes.byref(ctypes.c_int64())) == BAD
    assert L.spear_w8_forward(None, 16, 64, 16, 16, 8, 0, 1, None) == BAD
    assert L.spear_w8_check(None, None) == BAD
    assert L.spear_w8_destroy(None) == spear.SPEAR_OK


M, K = 4, 64
NORM = dict(x=1 << 20, ld_x=K, type=0, res=None, ld_res=0, res_out=None, ld_res_out=0, res_type=0, weight=2 << 20,
            weight_type=0, eps=1e-5, M=M, K=K, y=3 << 20, ld_y=K, q=4 << 20, ld_q=K, scales=5 << 20)
RES = dict(res=6 << 20, ld_res=K, res_out=7 << 20, ld_res_out=K)


def _norm(L, **kw):
    return L.spear_rms_norm(*{**NORM, **kw}.values(), None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=(1 << 20) + 1), dict(ld_x=K - 1), dict(type=3), dict(type=-1), dict(weight=None),
    dict(weight=(2 << 20) + 1), dict(weight_type=1), dict(weight_type=3), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(M=-1), dict(K=0), dict(y=None, q=None), dict(y=(3 << 20) + 1), dict(ld_y=K - 1),
    dict(ld_q=K - 1), dict(scales=None), dict(scales=(5 << 20) + 2),
    {**RES, "res_out": None}, {**RES, "ld_res": K - 1}, {**RES, "ld_res_out": 0}, {**RES, "res_type": 1},
    {**RES, "res": (6 << 20) + 1},
    # results that overlap what is read, each other, the weight or the scales
    dict(y=(1 << 20) + 2 * K), dict(q=1 << 20), dict(q=(3 << 20) + 8), dict(y=2 << 20), dict(scales=(4 << 20) + 16),
    dict(scales=1 << 20), dict(scales=2 << 20), {**RES, "scales": 6 << 20}, {**RES, "res_out": (6 << 20) + 2 * K}, {**RES, "res_out": 3 << 20}, {**RES, "y": 6 << 20, "ld_y": K + 8},
    {**RES, "res_type": 2, "res_out": 1 << 20}, {**RES, "q": 6 << 20}])
def test_norm_rejects_bad_arguments(L, bad):
    assert _norm(L, **bad) == BAD


def test_norm_rejects_rows_past_the_registers(L):
    assert _norm(L, K=32769, ld_x=32769, ld_y=32769, ld_q=32769) == UNSUPPORTED


def test_no_rows_is_a_no_op(L):
    assert _norm(L, M=0, x=None, y=None, q=None, scales=None) == spear.SPEAR_OK
    assert L.spear_quantize_rows(None, K, 0, 0, K, None, K, None, None) == spear.SPEAR_OK
    assert L.spear_dequantize_rows(None, K, None, 0, K, None, K, 0, None) == spear.SPEAR_OK


@pytest.mark.parametrize("bad", [dict(x=None), dict(ld_x=K - 1), dict(x=(1 << 20) + 1), dict(type=3), dict(M=-1), dict(K=0),
                                 dict(q=None), dict(ld_q=K - 1), dict(scales=None), dict(scales=(5 << 20) + 1),
                                 dict(q=(1 << 20) + 64), dict(scales=1 << 20), dict(scales=4 << 20)])
def test_quantize_rejects_bad_arguments(L, bad):
    a = dict(x=1 << 20, ld_x=K, type=0, M=M, K=K, q=4 << 20, ld_q=K, scales=5 << 20)
    a.update(bad)
    assert L.spear_quantize_rows(*a.values(), None) == BAD


@pytest.mark.parametrize("bad", [dict(q=None), dict(ld_q=K - 1), dict(scales=None), dict(scales=(5 << 20) + 1), dict(M=-1),
                                 dict(K=0), dict(out=None), dict(out=(1 << 20) + 1), dict(ld_out=K - 1), dict(type=3),
                                 dict(out=4 << 20), dict(out=5 << 20)])
def test_dequantize_rejects_bad_arguments(L, bad):
    a = dict(q=4 << 20, ld_q=K, scales=5 << 20, M=M, K=K, out=1 << 20, ld_out=K, type=0)
    a.update(bad)
    assert L.spear_dequantize_rows(*a.values(), None) == BAD


def test_arguments_in_a_struct_mean_the_same(L):
    """Each field is where the library looks for it: spoilt one by one, only the one that the call then refuses changes."""
    r = spear._rows()
    ok, unsupported = spear.SPEAR_OK, UNSUPPORTED
    norm = dict(x=1 << 20, ld_x=K, res=6 << 20, ld_res=K, res_out=7 << 20, ld_res_out=K, weight=2 << 20, y=3 << 20, ld_y=K,
                q=4 << 20, ld_q=K, scales=5 << 20, stream=0, type=0, res_type=0, weight_type=0, M=0, K=K, eps=1e-5)
    call = lambda **kw: L.spear_rms_norm_args(r.norm_args(*{**norm, **kw}.values()))
    assert call() == ok and call(K=32769) == unsupported
    assert call(eps=-1.0) == BAD and call(type=3) == BAD and call(weight_type=1) == BAD and call(weight=0) == BAD
    for bad in (dict(x=0), dict(ld_x=K - 1), dict(ld_res=K - 1), dict(res_out=0), dict(ld_res_out=0), dict(res=1 + (6 << 20)),
                dict(ld_y=K - 1), dict(y=1 + (3 << 20)), dict(ld_q=K - 1), dict(scales=2 + (5 << 20)), dict(q=3 << 20),
                dict(res_type=1)):
        assert call(M=4, **bad) == BAD, bad
    quant = dict(x=1 << 20, ld_x=K, q=4 << 20, ld_q=K, scales=5 << 20, stream=0, type=0, M=0, K=K)
    call = lambda **kw: L.spear_quantize_rows_args(r.quantize_args(*{**quant, **kw}.values()))
    assert call() == ok and call(K=32769) == unsupported and call(type=3) == BAD
    for bad in (dict(x=0), dict(ld_x=K - 1), dict(q=0), dict(ld_q=K - 1), dict(scales=1 + (5 << 20))):
        assert call(M=4, **bad) == BAD, bad
    back = dict(q=4 << 20, ld_q=K, scales=5 << 20, out=1 << 20, ld_out=K, stream=0, type=0, M=0, K=K)
    call = lambda **kw: L.spear_dequantize_rows_args(r.dequantize_args(*{**back, **kw}.values()))
    assert call() == ok and call(K=0) == BAD and call(type=3) == BAD
    for bad in (dict(q=0), dict(ld_q=K - 1), dict(scales=1 + (5 << 20)), dict(out=0), dict(ld_out=K - 1)):
        assert call(M=4, **bad) == BAD, bad
    assert L.spear_w8_forward_args(r.forward_args(0, 16, 64, 16, 16, 8, 0, 0, 1)) == BAD
    for name in ("rms_norm", "quantize_rows", "dequantize_rows", "w8_forward"):
        assert getattr(L, f"spear_{name}_args")(None) == BAD


def test_debug_set_needs_a_handle(L):
    assert L.spear_w8_debug_set(None, 0, 0) == BAD


@pytest.mark.parametrize("ld", [0, -5, 1])
def test_the_distance_of_a_single_row_is_of_no_account(L, ld):
    """Past the checks of the arguments comes that of the width, which stops these calls before the device."""
    W = 32769
    lds = dict(ld_x=ld, ld_res=ld, ld_res_out=ld, ld_y=ld, ld_q=ld)
    assert _norm(L, **{**RES, **lds, "M": 1, "K": W}) == UNSUPPORTED
    assert _norm(L, **{**RES, **lds, "M": 2, "K": W}) == BAD
    quant = lambda M: L.spear_quantize_rows(1 << 20, ld, 0, M, W, 4 << 20, ld, 5 << 20, None)
    assert quant(1) == UNSUPPORTED and quant(2) == BAD
    # what overlaps is found whatever the distance says
    assert _norm(L, M=1, ld_x=ld, ld_y=ld, ld_q=ld, y=(1 << 20) + 2) == BAD
    assert L.spear_quantize_rows(1 << 20, ld, 0, 1, K, (1 << 20) + 2, ld, 5 << 20, None) == BAD
    assert L.spear_dequantize_rows(4 << 20, ld, 5 << 20, 1, K, (4 << 20) + 16, ld, 0, None) == BAD
