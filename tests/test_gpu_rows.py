"""The norm, the 8-bit quantisation of rows and the read-back against the oracle."""
import numpy as np
import pytest
import torch

from oracle import w8
from quantized_linear_error_gb300 import spear

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# Statistics: a sum of K squares, at most 32 in a row a thread and ten levels of pairs, off by 42 half steps of fp32;
# half of that in the root, and eight more roundings (mean, eps, root, products): below 32 half steps.
NORM_REL = 32 * 2.0 ** -24


def _rand(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def _np(t):
    return t.detach().float().cpu().numpy()


def _near(got, want, dtype):
    """got of `dtype` is the rounding of a value within NORM_REL of want (f16: or half its smallest step)."""
    half = torch.finfo(dtype).eps / 2
    tol = np.abs(want) * (NORM_REL + half * (1 + NORM_REL)) + (2.0 ** -25 if dtype is F16 else 2.0 ** -140)
    assert np.all(np.abs(_np(got).astype(np.float64) - want) <= tol)


def _codes_near(q, s, v):
    """Codes and scales of rows whose values lie within NORM_REL of v."""
    q, s = q.cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64)
    a = np.abs(v).max(1)
    assert np.all(np.abs(s - a / 127) <= a / 127 * (NORM_REL + 2.0 ** -23))
    assert np.all(np.abs(q * s[:, None] - v) <= s[:, None] * (0.5 + 127 * 4 * NORM_REL))


# widths: a warp a row (1 to 4 groups), a block a row (1 to 4 groups), ragged ones that no wide access fits
WIDTHS = [1, 7, 8, 64, 250, 256, 257, 512, 1000, 1024, 1032, 4096, 4100, 8192, 11008, 12345, 16384, 20000, 28672, 32768]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("K", WIDTHS)
def test_quantize_bit_exact(K, dtype):
    x = _rand(K, 5, K, dtype=dtype)
    x[1] = 0
    x[2] *= 2.0 ** -10
    if K > 8:
        x[3, K - 1] = float("nan")
        x[4, 3] = float("-inf")
    q, s = spear.quantize_rows(x)
    qr, sr = w8.quantize_rows(_np(x))
    assert np.array_equal(q.cpu().numpy(), qr)
    assert np.array_equal(s.cpu().numpy(), sr, equal_nan=True)
    for out in (BF16, F16, F32):
        got = spear.dequantize_rows(q, s, torch.empty(5, K, dtype=out, device="cuda"))
        want = (torch.from_numpy(qr).float() * torch.from_numpy(sr)[:, None]).to(out)
        assert torch.equal(got.cpu().nan_to_num(77.0), want.nan_to_num(77.0))


@pytest.mark.parametrize("M", [1, 2, 9, 160, 500])
def test_quantize_row_counts(M):
    for K in (96, 4096):
        x = _rand(M, M, K, dtype=BF16)
        q, s = spear.quantize_rows(x)
        qr, sr = w8.quantize_rows(_np(x))
        assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -101, 2.0 ** -99, 2.0 ** 100, 2.0 ** 125])
def test_quantize_of_any_size(scale):
    x = _rand(3, 4, 300) * 0.5 * scale
    q, s = spear.quantize_rows(x)
    qr, sr = w8.quantize_rows(_np(x))
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)


@pytest.mark.parametrize("dtype,res", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32), (BF16, None),
                                       (F32, None)])
@pytest.mark.parametrize("K", WIDTHS)
def test_norm(K, dtype, res):
    M = 3
    x, w = _rand(K, M, K, dtype=dtype), _rand(K + 1, K, dtype=dtype) + 1
    r = None if res is None else _rand(K + 2, M, K, dtype=res, scale=3.0)
    ro = None if res is None else torch.empty_like(r)
    y, q, s = torch.empty_like(x), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    spear.rms_norm(x, w, 1e-5, r, ro, y, q, s)
    h, v = w8.rms_norm(_np(x), _np(w), 1e-5, None if r is None else _np(r))
    if r is not None:  # one fp32 sum, one rounding
        assert torch.equal(ro.cpu(), (x.float() + r.float()).to(res).cpu())
    # the fp32 sum of x and the residual is a rounding of its own
    _near(y, v, dtype) if r is None else _near_sum(y, h, v, dtype, _np(w))
    if r is None:
        _codes_near(q, s, v)


def _near_sum(got, h, v, dtype, w):
    h32 = h.astype(np.float32).astype(np.float64)  # what the kernel works on: x + residual rounded to fp32
    want = h32 / np.sqrt((h32 * h32).mean(1, keepdims=True) + 1e-5) * w
    _near(got, want, dtype)


@pytest.mark.parametrize("only", ["y", "q"])
@pytest.mark.parametrize("wdtype", [BF16, F32])
def test_norm_outputs_one_by_one_are_the_same(only, wdtype):
    M, K = 6, 1536
    x, w, r = _rand(1, M, K, dtype=BF16), _rand(2, K, dtype=wdtype) + 1, _rand(3, M, K, dtype=BF16)
    new = lambda: (torch.empty_like(x), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"))
    y, q, s = new()
    ro = torch.empty_like(r)
    spear.rms_norm(x, w, 1e-6, r, ro, y, q, s)
    y1, q1, s1 = new()
    if only == "y":
        assert spear.rms_norm(x, w, 1e-6, r.clone(), y=y1) is y1
        assert torch.equal(y1, y)
    else:
        spear.rms_norm(x, w, 1e-6, r.clone(), q=q1, scales=s1)
        assert torch.equal(q1, q) and torch.equal(s1, s)
    _codes_near(q, s, w8.rms_norm(_np(ro * 0), _np(w), 1e-6, (_np(x) + _np(r)))[1])


# rows enough that warps and blocks go through several of their own, of each width class and pair of types
@pytest.mark.parametrize("x,res,weight", [(BF16, BF16, BF16), (BF16, F32, BF16), (F16, F16, F32), (F16, F32, F32),
                                          (F32, F32, F32), (BF16, None, F32), (F32, None, F32)])
@pytest.mark.parametrize("M,K", [(11000, 128), (11000, 264), (5300, 520), (5300, 1016), (1500, 1032), (1300, 4096),
                                 (700, 8200), (650, 12296), (330, 16384), (170, 20488)])
def test_many_rows(M, K, x, res, weight):
    X, W = _rand(K, M, K, dtype=x), _rand(K + 1, K, dtype=weight) + 1
    R = None if res is None else _rand(K + 2, M, K, dtype=res, scale=3.0)
    if M > 1000:
        X[7, 3], X[M - 1, K - 1] = float("nan"), float("inf")
    ro = None if res is None else torch.empty_like(R)
    y, q, s = torch.empty_like(X), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    spear.rms_norm(X, W, 1e-5, R, ro, y, q, s)
    # the same rows a few at a time: the kernel that takes a row and ends
    for i in list(range(0, M, M // 3)) + [M - 5]:
        part = slice(i, i + 5)
        n = X[part].shape[0]
        y1, q1, s1 = torch.empty_like(X[part]), torch.empty(n, K, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        ro1 = None if res is None else torch.empty_like(R[part])
        spear.rms_norm(X[part], W, 1e-5, None if R is None else R[part], ro1, y1, q1, s1)
        if R is not None:
            assert torch.equal(ro[part].nan_to_num(9.0), ro1.nan_to_num(9.0))
    h = X.double() if R is None else (X.float() + R.float()).double()
    if R is not None:
        assert torch.equal(ro.nan_to_num(9.0), (X.float() + R.float()).to(res).nan_to_num(9.0))
    v = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * W.double()
    bad = ~h.isfinite().all(1)
    assert torch.equal(y.isnan().all(1), bad) and torch.equal(s.isnan(), bad) and not q[bad].any()
    ok = ~bad
    half, floor = torch.finfo(x).eps / 2, 2.0 ** -25 if x is F16 else 2.0 ** -140
    tol = v[ok].abs() * (NORM_REL + half * (1 + NORM_REL)) + floor
    assert bool(((y[ok].double() - v[ok]).abs() <= tol).all())
    a, sd = v[ok].abs().amax(1), s[ok].double()
    assert bool(((sd - a / 127).abs() <= a / 127 * (NORM_REL + 2.0 ** -23)).all())
    assert bool(((q[ok].double() * sd[:, None] - v[ok]).abs() <= sd[:, None] * (0.5 + 127 * 4 * NORM_REL)).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,K", [(11000, 128), (5300, 520), (2600, 1024), (1500, 1032), (1300, 4096), (700, 11008),
                                 (330, 16384), (170, 28672)])
def test_quantize_many_rows(M, K, dtype):
    x = _rand(M, M, K + 16, dtype=dtype)[:, 8:8 + K]
    q, s = spear.quantize_rows(x)
    qr, sr = w8.quantize_rows(_np(x))
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)
    out = spear.dequantize_rows(q, s, torch.empty(M, K, dtype=dtype, device="cuda"))
    assert torch.equal(out, (q.float() * s[:, None]).to(dtype))


def test_many_rows_in_place():
    M, K = 2000, 2048
    x, w, r = _rand(1, M, K, dtype=BF16), _rand(2, K, dtype=BF16), _rand(3, M, K, dtype=F32)
    y, ro = torch.empty_like(x), torch.empty_like(r)
    spear.rms_norm(x, w, 1e-5, r, ro, y)
    spear.rms_norm(x, w, 1e-5, r, r, x)
    assert torch.equal(x, y) and torch.equal(r, ro)


def test_norm_in_place_and_strided():
    M, K = 70, 1000
    wide = _rand(5, M, 3 * 1008, dtype=BF16)
    x, r = wide[:, :K], wide[:, 1008:1008 + K]
    w = _rand(6, K, dtype=BF16)
    q, s = torch.full((M, K + 24), 99, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    want_y, want_r = torch.empty(M, K, dtype=BF16, device="cuda"), torch.empty(M, K, dtype=BF16, device="cuda")
    want_q, want_s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    spear.rms_norm(x.contiguous(), w, 1e-5, r.contiguous(), want_r, want_y, want_q, want_s)
    keep = wide.clone()
    spear.rms_norm(x, w, 1e-5, r, y=x, q=q[:, 16:16 + K], scales=s)  # y over x, the residual in place
    assert torch.equal(x, want_y) and torch.equal(r, want_r) and torch.equal(q[:, 16:16 + K], want_q)
    assert torch.equal(s, want_s) and torch.all(q[:, :16] == 99) and torch.all(q[:, 16 + K:] == 99)
    assert torch.equal(wide[:, K:1008], keep[:, K:1008]) and torch.equal(wide[:, 1008 + K:], keep[:, 1008 + K:])
    odd = _rand(7, M, 1001, dtype=BF16)[:, 1:]  # neither base nor rows are aligned
    y = torch.empty(M, 1003, dtype=BF16, device="cuda")[:, 2:1002]
    spear.rms_norm(odd, w, 1e-5, y=y)
    _near(y, w8.rms_norm(_np(odd), _np(w), 1e-5)[1], BF16)


def test_rows_far_apart():
    """Offsets past 32 bits, for few rows and for many."""
    for M, ld in ((5, 1 << 30), (1300, 1 << 22)):
        K = 2056
        big = torch.empty((M - 1) * ld + K, dtype=BF16, device="cuda")
        x = big.as_strided((M, K), (ld, 1))
        x.copy_(_rand(M, M, K))
        q = torch.empty((M - 1) * ld + K, dtype=torch.int8, device="cuda").as_strided((M, K), (ld, 1))
        s = torch.empty(M, device="cuda")
        spear.quantize_rows(x, q, s)
        qr, sr = w8.quantize_rows(_np(x))
        assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)
        y, w = torch.empty(M, K, dtype=BF16, device="cuda"), _rand(1, K, dtype=BF16)
        spear.rms_norm(x, w, y=y)
        assert torch.equal(spear.dequantize_rows(q, s, x), spear.dequantize_rows(q, s, torch.empty_like(y)))
        near = spear.rms_norm(_rand(M, M, K).bfloat16(), w, y=torch.empty_like(y))
        assert torch.equal(y, near)
        del big, x, q


def test_norm_rows_that_are_not_finite():
    x, w = _rand(1, 6, 2048, dtype=BF16), _rand(2, 2048, dtype=BF16) + 1
    x[1, 5], x[3, 2047], x[4, 0] = float("nan"), float("inf"), float("-inf")
    y, q, s = torch.empty_like(x), torch.empty(6, 2048, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    spear.rms_norm(x, w, y=y, q=q, scales=s)
    for i in range(6):
        bad = i in (1, 3, 4)
        assert bool(y[i].isnan().all()) == bad and bool(y[i].isnan().any()) == bad and bool(s[i].isnan()) == bad
        assert not bad or bool((q[i] == 0).all())


@pytest.mark.parametrize("scale,eps", [(1e18, 1e-5), (1e37, 1e-5), (1e-25, 0.0), (2.0 ** -120, 0.0), (1e-15, 1e-30),
                                       (1e-12, 1e-5), (1e10, 0.0)])
def test_norm_of_any_size(scale, eps):
    """Squares beyond fp32 on either side."""
    for K in (200, 3000):
        x, w = _rand(9, 4, K) * scale, _rand(8, K) + 1
        y, q, s = torch.empty_like(x), torch.empty(4, K, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
        spear.rms_norm(x, w, eps, y=y, q=q, scales=s)
        eps32 = float(np.float32(eps))
        v = w8.rms_norm(_np(x), _np(w), eps32)[1]
        _near(y, v, F32)
        _codes_near(q, s, v)


def test_norm_zero_rows():
    x, w = torch.zeros(2, 4096, dtype=BF16, device="cuda"), torch.ones(4096, dtype=BF16, device="cuda")
    y, q, s = torch.ones_like(x), torch.ones(2, 4096, dtype=torch.int8, device="cuda"), torch.ones(2, device="cuda")
    spear.rms_norm(x, w, 1e-5, y=y, q=q, scales=s)
    assert not y.any() and not q.any() and not s.any()


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    spear.rms_norm(x, w, y=torch.empty_like(x))
    q, s = spear.quantize_rows(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    spear.dequantize_rows(q, s, torch.empty_like(x))


def test_refusals_of_the_binding():
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    y, q, s = torch.empty_like(x), torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    for bad in (dict(y=None), dict(y=y, q=q), dict(y=y, scales=s), dict(y=y.float()), dict(y=y[:, :32]), dict(y=y.cpu()),
                dict(y=y, residual_out=y.clone()), dict(y=y, residual=x.half()), dict(y=y, residual=x[:2]),
                dict(q=q, scales=s.half()), dict(q=q.to(torch.uint8), scales=s), dict(q=q, scales=s[:2])):
        with pytest.raises(ValueError):
            spear.rms_norm(x, w, **bad)
    for weight in (w.half(), w[:32], w.cpu(), torch.ones(128, dtype=BF16, device="cuda")[::2]):
        with pytest.raises(ValueError):
            spear.rms_norm(x, weight, y=y)
    with pytest.raises(ValueError):
        spear.rms_norm(x.t(), w, y=y.t())
    with pytest.raises(ValueError):
        spear.quantize_rows(x.int())
    with pytest.raises(spear.SpearError):
        spear.quantize_rows(torch.zeros(1, 32769, device="cuda"))
    with pytest.raises(spear.SpearError):
        spear.rms_norm(x, w, y=x.view(-1)[:256].view(4, 64)[:, :], residual=x)  # residual_out over y
    with pytest.raises(ValueError):
        spear.dequantize_rows(q, s, torch.empty(4, 63, device="cuda"))


def test_captured_on_another_stream():
    x, w, r = _rand(1, 33, 4096, dtype=BF16), _rand(2, 4096, dtype=BF16), _rand(3, 33, 4096, dtype=BF16)
    ro, q, s = torch.empty_like(r), torch.empty(33, 4096, dtype=torch.int8, device="cuda"), torch.empty(33, device="cuda")
    v = torch.empty_like(x)
    spear.rms_norm(x, w, 1e-5, r, ro, q=q, scales=s)
    spear.dequantize_rows(q, s, v)
    want = [t.clone() for t in (ro, q, s, v)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        spear.rms_norm(x, w, 1e-5, r, ro, q=q, scales=s)
        spear.dequantize_rows(q, s, v)
    for t in (ro, q, s, v):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((ro, q, s, v), want))


def _guarded(M, K, lead, ld, dtype, seed=None):
    """Rows that start `lead` elements behind an aligned address, `ld` apart, with the buffer that holds them."""
    n = lead + M * ld + 64
    buf = torch.full((n,), 77, dtype=dtype, device="cuda") if seed is None else _rand(seed, n, dtype=dtype)
    return buf, buf[lead:].as_strided((M, K), (ld, 1))


# Rows that no wide access fits, in number enough that warps and blocks go through several: odd widths, starts and
# distances, each a different one for every array.
@pytest.mark.parametrize("x,res", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32), (BF16, None), (F32, None)])
@pytest.mark.parametrize("M,K", [(11000, 1), (11000, 127), (11000, 256), (5300, 257), (5300, 511), (3000, 517), (2600, 1023),
                                 (1500, 1025), (1300, 4097), (700, 8191), (400, 12289), (200, 16383), (170, 20487)])
def test_many_rows_of_any_width(M, K, x, res):
    xb, X = _guarded(M, K, 3, K + 2, x, 11)
    rb, R = (None, None) if res is None else _guarded(M, K, 5, K + 1, res, 12)
    w = _rand(13, K, dtype=x) + 1
    yb, y = _guarded(M, K, 7, K + 3, x)
    ob, ro = (None, None) if res is None else _guarded(M, K, 1, K + 5, res)
    qb, q = _guarded(M, K, 9, K + 7, torch.int8)
    s = torch.empty(M, device="cuda")
    spear.rms_norm(X, w, 1e-5, R, ro, y, q, s)
    h = X.double() if R is None else (X.float() + R.float()).double()
    v = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    half, floor = torch.finfo(x).eps / 2, 2.0 ** -25 if x is F16 else 2.0 ** -140
    assert bool(((y.double() - v).abs() <= v.abs() * (NORM_REL + half * (1 + NORM_REL)) + floor).all())
    a, sd = v.abs().amax(1), s.double()
    assert bool(((sd - a / 127).abs() <= a / 127 * (NORM_REL + 2.0 ** -23) + floor).all())
    assert bool(((q.double() * sd[:, None] - v).abs() <= sd[:, None] * (0.5 + 127 * 4 * NORM_REL) + floor).all())
    if R is not None:
        assert torch.equal(ro, (X.float() + R.float()).to(res))
    keep = [(yb, y), (qb, q)] + ([] if ob is None else [(ob, ro)])
    for buf, rows in keep:  # nothing beside the rows
        rows.fill_(77)
        assert bool((buf == 77).all())
    # quantised, and in place over x and the residual: the same bits
    q2b, q2 = _guarded(M, K, 2, K + 1, torch.int8)
    spear.quantize_rows(X, q2, s)
    qr, sr = w8.quantize_rows(_np(X))
    assert np.array_equal(q2.cpu().numpy(), qr) and np.array_equal(s.cpu().numpy(), sr)
    q2.fill_(77)
    assert bool((q2b == 77).all())
    want_y, want_r = torch.empty(M, K, dtype=x, device="cuda"), None if R is None else torch.empty(M, K, dtype=res, device="cuda")
    spear.rms_norm(X, w, 1e-5, R, want_r, want_y)
    spear.rms_norm(X, w, 1e-5, R, R, X)
    assert torch.equal(X, want_y) and (R is None or torch.equal(R, want_r))


@pytest.mark.parametrize("out", [BF16, F16, F32])
@pytest.mark.parametrize("M,K", [(1, 1), (5, 15), (1, 16), (3, 16), (7, 17), (33, 31), (2, 33), (700, 4097), (129, 12289), (4, 16383)])
def test_read_back_of_any_width(M, K, out):
    """Rows one after the other, in a buffer that goes on, and rows apart."""
    codes = torch.randint(-127, 128, (M, K), generator=torch.Generator().manual_seed(K)).to(torch.int8).cuda()
    s = _rand(M, M).abs() + 0.1
    want = (codes.float() * s[:, None]).to(out)
    for lead, ld in ((0, K), (16, K), (1, K), (0, K + 1), (3, K + 8)):
        _, q = _guarded(M, K, lead, ld, torch.int8)
        q.copy_(codes)
        buf, got = _guarded(M, K, lead, ld, out)
        spear.dequantize_rows(q, s, got)
        assert torch.equal(got, want)
        got.fill_(77)
        assert bool((buf == 77).all())


@pytest.mark.parametrize("M,K", [((1 << 32) + 3, 16), ((1 << 31) + 1, 16), (3, (1 << 32) + 16), (1, (1 << 31))])
def test_sizes_past_32_bits_mean_what_they_say(M, K):
    """They are refused, not cut to their lower half. (Views of few elements: nothing is read.)"""
    def view(dtype, *shape):
        return torch.empty(1, dtype=dtype, device="cuda").as_strided(shape, (0,) * (len(shape) - 1) + (1,)) if shape[-1] == 1 \
            else torch.empty(64, dtype=dtype, device="cuda")[:1].expand(shape)
    x, q, s, w = view(BF16, M, K), view(torch.int8, M, K), view(F32, M), view(BF16, K)
    with pytest.raises(ValueError):
        spear.rms_norm(x, w, 1e-5, q=q, scales=s)
    with pytest.raises(ValueError):
        spear.quantize_rows(x, q, s)
    with pytest.raises(ValueError):
        spear.dequantize_rows(q, s, x)


def test_rows_and_results_on_one_device():
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    for call in (lambda: spear.rms_norm(x, w.cpu(), y=x), lambda: spear.rms_norm(x.cpu(), w, y=x.cpu()),
                 lambda: spear.rms_norm(x, w, residual=x.cpu(), y=x), lambda: spear.rms_norm(x, w, q=q, scales=s.cpu()),
                 lambda: spear.rms_norm(x, w, y=x.cpu()), lambda: spear.quantize_rows(x, q.cpu(), s),
                 lambda: spear.quantize_rows(x.cpu(), q.cpu(), s.cpu()), lambda: spear.dequantize_rows(q, s, x.cpu()),
                 lambda: spear.dequantize_rows(q, s.cpu(), x)):
        with pytest.raises(ValueError):
            call()


def test_read_back_of_the_widest_row():
    K = (1 << 31) - 1
    q = torch.zeros(K, dtype=torch.int8, device="cuda")
    q[-40:] = torch.arange(40, dtype=torch.int8, device="cuda")
    out = torch.full((K + 16,), 7, dtype=BF16, device="cuda")
    s = torch.full((1,), 2.0, device="cuda")
    spear.dequantize_rows(q.view(1, K), s, out[:K].view(1, K))
    assert torch.equal(out[K - 40:K], 2 * torch.arange(40, device="cuda").to(BF16)) and not out[:K - 39].any()
    assert bool((out[K:] == 7).all())


def test_results_belong_to_the_stream_that_makes_them():
    """Memory that the current stream freed and may still use is not given to rows quantised on another one."""
    x = _rand(1, 2000, 4096, dtype=BF16)
    want, ws = spear.quantize_rows(x)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (other, other.cuda_stream):
        used = torch.empty(2000, 4096, dtype=torch.int8, device="cuda")
        for _ in range(50):
            used.fill_(1)
        del used  # its block goes to the next of this size on the current stream
        q, s = spear.quantize_rows(x, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(q, want) and torch.equal(s, ws)
