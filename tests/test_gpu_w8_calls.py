"""Calls of the 8-bit operators that their documentation allows and the other tests leave out: results in place of what is
read, surroundings that are not finite, weights that start anywhere, and the largest sizes."""
import numpy as np
import pytest
import torch

from oracle import w8
from quantized_linear_error_gb300 import spear

from .test_gpu_rows import _codes_near, _near, _np, _rand
from .test_gpu_w8 import _dev

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _outs(M, K, dtype):
    return (torch.empty(M, K, dtype=dtype, device="cuda"), torch.empty(M, K, dtype=torch.int8, device="cuda"),
            torch.empty(M, device="cuda"))


@pytest.mark.parametrize("M,K", [(3, 520), (2000, 520), (3, 4096), (1300, 4096), (1300, 4097), (400, 12289)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_results_in_place_of_what_is_read(M, K, dtype):
    x, r, w = _rand(1, M, K, dtype=dtype), _rand(2, M, K, dtype=dtype), _rand(3, K, dtype=dtype)
    y, ro = torch.empty_like(x), torch.empty_like(r)
    spear.rms_norm(x, w, 1e-5, r, ro, y)
    a = x.clone()
    spear.rms_norm(a, w, 1e-5, r.clone(), a, y2 := torch.empty_like(x))  # the sum over x
    assert torch.equal(a, ro) and torch.equal(y2, y)
    a, b = x.clone(), r.clone()
    spear.rms_norm(a, w, 1e-5, b, b, a)  # the sum over the residual, the result over x
    assert torch.equal(a, y) and torch.equal(b, ro)
    twice = torch.empty_like(x)
    spear.rms_norm(x, w, 1e-5, x, twice, y2)  # x is its own residual
    assert torch.equal(twice, x + x)
    a = x.clone()
    spear.rms_norm(a, w, 1e-5, a, y=b)
    assert torch.equal(a, twice) and torch.equal(b, y2)


@pytest.mark.parametrize("M,K", [(3, 1), (5, 127), (3, 1000), (2000, 255), (2000, 1000), (5, 4100), (1300, 4095), (400, 12290),
                                 (160, 20487)])
@pytest.mark.parametrize("x,res", [(BF16, F32), (F16, F16), (F32, F32)])
def test_surroundings_that_are_not_finite(M, K, x, res):
    """What lies beside the rows, the weight and the scales is read in part, and used nowhere."""
    def inside(lead, rows, cols, dtype, seed):
        ld = cols + 3
        buf = torch.full((lead + rows * ld + 40,), float("nan"), dtype=dtype, device="cuda")
        view = buf[lead:].as_strided((rows, cols), (ld, 1))
        view.copy_(_rand(seed, rows, cols, dtype=dtype))
        return view
    X, R, W = inside(1, M, K, x, 1), inside(5, M, K, res, 2), inside(3, 1, K, x, 3)[0]
    y, q, s = _outs(M, K, x)
    ro = torch.empty(M, K, dtype=res, device="cuda")
    spear.rms_norm(X, W, 1e-5, R, ro, y, q, s)
    h = X.float() + R.float()
    assert torch.equal(ro, h.to(res))
    v = w8.rms_norm(_np(h), _np(W), 1e-5)[1]
    _near(y, v, x)
    _codes_near(q, s, v)
    spear.quantize_rows(X, q, s)
    qr, sr = w8.quantize_rows(_np(X))
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)


@pytest.mark.parametrize("M,K", [(3, 256), (3000, 256), (3000, 1024), (3, 8192), (1300, 4096), (400, 16384)])
@pytest.mark.parametrize("wdtype", [BF16, F32])
def test_a_weight_that_starts_anywhere(M, K, wdtype):
    x, buf = _rand(1, M, K, dtype=BF16), _rand(2, K + 16, dtype=wdtype)
    for lead in (1, 2, 7):
        w = buf[lead:lead + K]
        y, q, s = _outs(M, K, BF16)
        spear.rms_norm(x, w, 1e-5, y=y, q=q, scales=s)
        v = w8.rms_norm(_np(x), _np(w), 1e-5)[1]
        _near(y, v, BF16)
        _codes_near(q, s, v)


def _linear_of(N, K, M, max_tokens, dtype, top):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    code = lambda rows: torch.randint(-top, top + 1, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    w, sw = code(N), torch.rand(N, generator=g, device="cuda") + 0.5
    layer = spear.SpearW8Linear(w, sw, max_tokens=max_tokens)
    for m in M:
        x, sx = code(m), torch.rand(m, generator=g, device="cuda") + 0.5
        y = torch.full((m, N), 7.0, dtype=dtype, device="cuda")
        layer.forward(x, sx, y)
        assert layer.check() == spear.SPEAR_OK
        # sums of at most 2^24: exact in fp64, then two roundings to fp32 and one to the result's type
        rows, cols = torch.arange(0, m, max(1, m // 4000), device="cuda"), torch.arange(0, N, max(1, N // 3000), device="cuda")
        rows[-1], cols[-1] = m - 1, N - 1
        p = x[rows].double() @ w[cols].double().t()
        assert float(p.abs().max()) < 2 ** 24
        assert torch.equal(y[rows][:, cols], (p.float() * sx[rows, None] * sw[cols]).to(dtype))
    layer.close()


def test_the_most_tokens():
    _linear_of(24, 64, [1 << 20, (1 << 20) - 1], 1 << 20, BF16, 127)


def test_the_most_outputs():
    _linear_of(1 << 22, 16, [1, 9, 33], 33, BF16, 127)


def test_the_most_channels():
    _linear_of(20, 1 << 20, [1, 20, 40], 40, F32, 1)


@pytest.mark.parametrize("K", [16, 17])
def test_millions_of_rows(K):
    M = 3_000_001
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    q, s = spear.quantize_rows(x)
    a = x.float().abs().amax(1)
    i = torch.randint(0, M, (20000,), generator=g, device="cuda")
    i[0], i[1] = M - 1, 0
    qr, sr = w8.quantize_rows(_np(x[i]))
    assert np.array_equal(q[i].cpu().numpy(), qr) and np.array_equal(s[i].cpu().numpy(), sr)
    # a code is within half a step of its value, and the products of fp32 off by 127 half steps of it at most, three times
    assert bool(((q.float() * s[:, None] - x.float()).abs() <= s[:, None] * (0.5 + 2.0 ** -14)).all())
    assert torch.equal(s, torch.from_numpy((a.cpu().numpy() / np.float32(127))).cuda())
    y = spear.dequantize_rows(q, s, torch.empty_like(x))
    assert torch.equal(y, (q.float() * s[:, None]).bfloat16())
