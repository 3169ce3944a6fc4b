"""The 8-bit integer linears against exact integer products."""
import numpy as np
import pytest
import torch

from oracle import w8
from quantized_linear_error_gb300 import spear

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _codes(seed, rows, K, top=127):
    """Codes as a quantiser leaves them (normal, some at the ends) and scales."""
    rng = np.random.default_rng(seed)
    q = np.clip(np.rint(rng.normal(0, top / 4, (rows, K))), -top, top).astype(np.int8)
    q[:, rng.integers(0, K, 2)] = (-top, top)
    return q, (rng.random(rows) * 0.01 + 0.001).astype(np.float32)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _layer(w, u=None, max_tokens=4096, activation="silu"):
    up = {} if u is None else dict(up=_dev(u[0]), up_scales=_dev(u[1]), activation=activation)
    return spear.SpearW8Linear(_dev(w[0]), _dev(w[1]), max_tokens=max_tokens, **up)


def _forward(layer, x, dtype=BF16):
    y = torch.full((x[0].shape[0], layer.N), 7.0, dtype=dtype, device="cuda")
    layer.forward(_dev(x[0]), _dev(x[1]), y)
    assert layer.check() == spear.SPEAR_OK
    return y


def _equal(y, want):
    """y is the rounding of the fp32 values `want`, bit for bit."""
    assert torch.equal(y.cpu(), torch.from_numpy(np.ascontiguousarray(want)).to(y.dtype))


# (N, K): strips and blocks that are not whole, one and many row groups a CTA, work split between CTAs
SHAPES = [(1, 16), (8, 64), (17, 80), (128, 256), (300, 1040), (1000, 4096), (4096, 512), (136, 11008), (5000, 144), (72, 70016)]
TOKENS = [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 61, 64, 100, 128, 129, 200, 257]


@pytest.mark.parametrize("N,K", SHAPES)
def test_linear_bit_exact(N, K):
    w = _codes(N + K, N, K)
    layer = _layer(w)
    for M in TOKENS:
        x = _codes(M, M, K)
        _equal(_forward(layer, x), w8.linear(*x, *w))
    layer.close()


@pytest.mark.parametrize("dtype", [F16, F32])
def test_linear_types(dtype):
    w = _codes(1, 200, 320)
    layer = _layer(w)
    for M in (1, 20, 90, 300):
        x = _codes(M, M, 320)
        _equal(_forward(layer, x, dtype), w8.linear(*x, *w))
    layer.close()


@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("N,K", [(1, 16), (8, 64), (15, 96), (129, 272), (1000, 1040), (2048, 4096)])
def test_gated(N, K, activation):
    w, u = _codes(N, N, K), _codes(N + 1, N, K)
    layer = _layer(w, u, activation=activation)
    for M in (1, 5, 16, 32, 33, 70, 130, 260):
        x = _codes(M, M, K)
        want = w8.gated(*x, *w, *u, activation)
        for dtype in (BF16, F32):
            y = _forward(layer, x, dtype).float().cpu().numpy().astype(np.float64)
            # A relative error d of z is an error d |z| of exp(-z), and |z| < 88 where the result is not below 2^-120.
            # Half steps of fp32 (2^-24): SiLU's z = g carries 2 (two scales), 88 * 2 = 176; GELU's z carries 3 * 2
            # from g's cube and 4 of its own products and sum, 88 * 10 = 880. Beside them the second projection (2),
            # exp (4), the sum, the quotient (4) and the product: 13. So 189 < 2^8 and 893 < 2^10 half steps.
            # 16-bit results take a faster exponential: 88 for the rounding of z log2(e), 8 of its own.
            # 285 < 2^9 and 989 < 2^10.
            rel = 2.0 ** ((-16 if dtype is F32 else -15) if activation == "silu" else -14)
            tol = np.abs(want) * (rel + torch.finfo(dtype).eps / 2) + 2.0 ** -120
            assert np.all(np.abs(y - want) <= tol)
    layer.close()


def test_codes_over_the_whole_range_and_large_sums():
    """Codes -128 .. 127, and sums past 2^24, which are rounded to fp32."""
    N, K = 40, 4096
    rng = np.random.default_rng(0)
    w = np.full((N, K), -128, np.int8), np.ones(N, np.float32)
    w[0][1::2] = 127
    w[0][2] = rng.integers(-128, 128, K)
    for M in (3, 30, 150):
        x = np.full((M, K), -128, np.int8), np.ones(M, np.float32)
        x[0][2:] = rng.integers(-128, 128, (M - 2, K))
        y = _forward(_layer(w), x, F32).cpu().numpy().astype(np.float64)
        size = w8.sums(np.abs(x[0].astype(np.int32)), np.abs(w[0].astype(np.int32)))
        # a step of 16 products at a time: K / 16 sums, and 64 more that join them, each a step of fp32 off at most
        assert np.all(np.abs(y - w8.sums(x[0], w[0])) <= size * (K / 16 + 64) * 2.0 ** -23)


def test_the_same_bits_whatever_the_batch():
    """Sums are exact, so a token's result does not depend on what runs beside it."""
    N, K = 700, 2048
    w, u, x = _codes(1, N, K), _codes(2, N, K), _codes(3, 300, K)
    for layer in (_layer(w), _layer(w, u)):
        for dtype in (BF16, F32):
            whole = _forward(layer, x, dtype)
            for a, b in ((0, 1), (1, 9), (9, 25), (25, 57), (57, 90), (90, 218)):
                assert torch.equal(_forward(layer, (x[0][a:b], x[1][a:b]), dtype), whole[a:b])


def test_many_tiles_and_splits():
    """Token counts around a tile's, weights of which 17 tokens go to the tensor cores, tiles split over pairs."""
    for N, K in ((11008, 4096), (2304, 8192), (256 * 76, 512), (20000, 2048)):
        w = _codes(N, N, K)
        layer = _layer(w, max_tokens=700)
        wd, sw = _dev(w[0]).double(), _dev(w[1])
        for M in (17, 32, 63, 150, 192, 193, 385, 500, 577, 700):
            x = _codes(M, M, K)
            y = _forward(layer, x, F32)
            p = _dev(x[0]).double() @ wd.t()  # integers below 2^24: exact
            assert float(p.abs().max()) < 2 ** 24
            assert torch.equal(y, p.float() * _dev(x[1])[:, None] * sw)
        layer.close()


def test_strides_and_untouched_elements():
    N, K = 72, 160
    w = _codes(1, N, K)
    layer = _layer(w)
    for M in (1, 5, 40, 150):
        x = _codes(M, M, K)
        for ld_x, ld_y, off, dtype in ((K + 16, N + 5, 3, BF16), (K + 48, N + 8, 8, F16), (K, N + 1, 1, F32)):
            big_x = torch.full((M, ld_x), 99, dtype=torch.int8, device="cuda")
            big_x[:, :K] = _dev(x[0])
            big_y = torch.full((M + 2, ld_y), 7.0, dtype=dtype, device="cuda")
            y = big_y[1:M + 1, off - 1:off - 1 + N]
            layer.forward(big_x[:, :K], _dev(x[1]), y)
            _equal(y.contiguous(), w8.linear(*x, *w))
            rest = big_y.clone()
            rest[1:M + 1, off - 1:off - 1 + N] = 7.0
            assert torch.all(rest == 7.0)
    layer.close()


def test_scales_that_are_zero_or_not_finite():
    N, K = 40, 128
    w = _codes(1, N, K)
    w[1][3], w[1][7] = 0, np.nan
    layer = _layer(w)
    for M in (6, 40):
        x = _codes(2, M, K)
        x[1][1], x[1][2] = 0, np.nan
        y = _forward(layer, x).float().cpu().numpy()
        nan = np.zeros((M, N), bool)
        nan[2], nan[:, 7] = True, True
        assert np.array_equal(np.isnan(y), nan)
        assert not y[1][~nan[1]].any() and not y[:, 3][~nan[:, 3]].any()


def test_repeated_and_captured_calls_give_the_same_bits():
    """Two handles, several token counts, one graph; replayed with other inputs."""
    N, K = 1500, 8192
    w, u = _codes(1, N, K), _codes(2, N, K)
    a, b = _layer(w), _layer(w, u)
    x = {M: _codes(M, M, K) for M in (1, 20, 64, 150)}
    q, s = {M: _dev(v[0]) for M, v in x.items()}, {M: _dev(v[1]) for M, v in x.items()}
    y = {M: [torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(2)] for M in x}

    def step():
        for M in x:
            a.forward(q[M], s[M], y[M][0])
            b.forward(q[M], s[M], y[M][1])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(2):
        for M in x:
            new = _codes(100 * seed + M, M, K)
            x[M] = new
            q[M].copy_(_dev(new[0])), s[M].copy_(_dev(new[1]))
        graph.replay()
        torch.cuda.synchronize()
        for M in x:
            _equal(y[M][0], w8.linear(*x[M], *w))
            eager = torch.empty_like(y[M][1])
            b.forward(q[M], s[M], eager)
            assert torch.equal(eager, y[M][1])
    assert a.check() == spear.SPEAR_OK and b.check() == spear.SPEAR_OK


def test_two_streams_at_once():
    """Layers with workspaces of their own, on two streams without an order between them."""
    K = 2048
    w, u = [_codes(i, 1400, K) for i in range(2)], [_codes(10 + i, 1400, K) for i in range(2)]
    layers = [_layer(w[0], max_tokens=300), _layer(w[1], u[1], max_tokens=300)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = []
    for n, M in enumerate((300, 40, 8, 170, 25, 260)):
        for i, layer in enumerate(layers):
            x = _codes(n, M, K)
            q, s = _dev(x[0]), _dev(x[1])
            want = torch.empty(M, 1400, dtype=BF16, device="cuda")
            layer.forward(q, s, want)
            calls.append((i, q, s, want, torch.empty_like(want)))
    torch.cuda.synchronize()
    for _ in range(10):
        for i, q, s, _, y in calls:
            layers[i].forward(q, s, y, stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for _, _, _, want, y in calls)
    assert all(layer.check() == spear.SPEAR_OK for layer in layers)


def test_many_tokens_of_a_narrow_layer():
    w = _codes(1, 520, 144)
    layer = _layer(w, max_tokens=20011)
    x = _codes(2, 20011, 144)
    _equal(_forward(layer, x), w8.linear(*x, *w))
    layer.close()


def test_offsets_past_32_bits():
    """Rows so far apart that elements and bytes from the first one on do not fit 32 bits, and weights of 2.7 GB."""
    N, K, ld = 72, 160, 1 << 27
    w = _codes(1, N, K)
    layer = _layer(w)
    for M in (20, 40):
        x = _codes(M, M, K)
        q = torch.empty((M - 1) * ld + K, dtype=torch.int8, device="cuda").as_strided((M, K), (ld, 1))
        q.copy_(_dev(x[0]))
        y = torch.empty((M - 1) * (ld // 2) + N, dtype=BF16, device="cuda").as_strided((M, N), (ld // 2, 1))
        layer.forward(q, _dev(x[1]), y)
        _equal(y.contiguous(), w8.linear(*x, *w))
        del q, y
    N, K = 131072, 20480
    g = torch.Generator(device="cuda").manual_seed(0)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand(N, generator=g, device="cuda")
    layer = spear.SpearW8Linear(wq, sw, max_tokens=64)
    rows = [0, 1, 65535, 104857, 104858, 131070, 131071]  # 104858 * 20480 is past 2^31
    for M in (3, 50):
        x = _codes(M, M, K)
        y = torch.empty(M, N, dtype=F32, device="cuda")
        layer.forward(_dev(x[0]), _dev(x[1]), y)
        p = _dev(x[0]).double() @ wq[rows].double().t()
        assert float(p.abs().max()) < 2 ** 24
        assert torch.equal(y[:, rows], p.float() * _dev(x[1])[:, None] * sw[rows])
    assert layer.check() == spear.SPEAR_OK
    layer.close()


def test_layers_share_a_workspace():
    """Layers of several shapes and token counts on one workspace, in one graph, give what they give alone."""
    shapes = [(700, 1024, False, 200), (256, 4096, False, 16), (2000, 2048, True, 300), (300, 512, False, 40)]
    ws = torch.full((max(spear.w8_workspace_bytes(n, k, m, g) for n, k, g, m in shapes),), 255, dtype=torch.uint8, device="cuda")
    layers = []
    for i, (N, K, gated, most) in enumerate(shapes):
        w, u = _codes(i, N, K), _codes(10 + i, N, K) if gated else None
        up = dict(up=_dev(u[0]), up_scales=_dev(u[1])) if gated else {}
        layers.append((spear.SpearW8Linear(_dev(w[0]), _dev(w[1]), max_tokens=most, workspace=ws, **up), _layer(w, u, most), K, N, most))
    calls = []
    for n, (shared, alone, K, N, most) in enumerate(layers * 2):
        x = _codes(n, most if n < len(layers) else (most + 1) // 2, K)
        q, s = _dev(x[0]), _dev(x[1])
        y = [torch.empty(q.shape[0], N, dtype=BF16, device="cuda") for _ in range(2)]
        alone.forward(q, s, y[1])
        calls.append((shared, q, s, y))
    for shared, q, s, y in calls:
        shared.forward(q, s, y[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for shared, q, s, y in calls:
            shared.forward(q, s, y[0])
    for _, _, _, y in calls:
        assert torch.equal(y[0], y[1])
        y[0].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for shared, _, _, y in calls:
        assert torch.equal(y[0], y[1]) and shared.check() == spear.SPEAR_OK
    with pytest.raises(spear.SpearError):  # too small
        spear.SpearW8Linear(_dev(_codes(0, 64, 64)[0]), _dev(_codes(0, 64, 64)[1]), max_tokens=100, workspace=ws[:1 << 20])


def test_refusals():
    w = _codes(1, 24, 64)
    layer = _layer(w, max_tokens=8)
    q, s = torch.zeros(8, 64, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    y = torch.empty(8, 24, dtype=BF16, device="cuda")
    layer.forward(q, s, y)
    layer.forward(q[:0], s[:0], y[:0])
    for bad in ((q[:, :48], s, y), (q.float(), s, y), (q, s[:4], y), (q, s.half(), y), (q, s, y[:, :16]), (q, s, y.double()),
                (q.cpu(), s, y), (q, s, y.cpu()), (q, s, y.t().contiguous().t())):
        with pytest.raises(ValueError):
            layer.forward(*bad)
    big = torch.zeros(16, 80, dtype=torch.int8, device="cuda")
    for bad in ((big[:9, :64], torch.ones(9, device="cuda"), torch.empty(9, 24, dtype=BF16, device="cuda")),  # max_tokens
                (big[:8, 8:72], s, y),                                                                     # base
                (torch.zeros(8, 72, dtype=torch.int8, device="cuda")[:, :64], s, y),                         # ld
                (q, s, q.view(BF16)[:, :24])):                                                               # over x
        with pytest.raises(spear.SpearError):
            layer.forward(*bad)
    with pytest.raises(ValueError):
        spear.SpearW8Linear(_dev(w[0]), _dev(w[1]), up=_dev(w[0]))
    with pytest.raises(ValueError):
        spear.SpearW8Linear(_dev(w[0]), _dev(w[1]), up=_dev(w[0][:8]), up_scales=_dev(w[1][:8]))
    with pytest.raises(ValueError):
        spear.SpearW8Linear(_dev(w[0]), _dev(w[1]), activation="relu")
    with pytest.raises(ValueError):
        spear.SpearW8Linear(_dev(w[0])[:, :32], _dev(w[1]))
    with pytest.raises(spear.SpearError):
        spear.SpearW8Linear(_dev(w[0])[:, :40].contiguous(), _dev(w[1]))
    layer.close()


def test_rows_to_product_and_back():
    """Norm with the residual, both projections and the activation, quantisation, down projection: as a block runs them."""
    M, K, F = 45, 512, 768
    g = torch.Generator().manual_seed(0)
    x, r = (torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(2))
    weight = (1 + 0.1 * torch.randn(K, generator=g)).bfloat16().cuda()
    W, U = (torch.randn(F, K, generator=g).cuda() * K ** -0.5 for _ in range(2))
    D = torch.randn(K, F, generator=g).cuda() * F ** -0.5
    qw, qu, qd = (spear.quantize_rows(t) for t in (W, U, D))
    pair = spear.SpearW8Linear(*qw, max_tokens=64, up=qu[0], up_scales=qu[1])
    down = spear.SpearW8Linear(*qd, max_tokens=64)
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    h, y = torch.empty(M, F, dtype=BF16, device="cuda"), torch.empty(M, K, dtype=BF16, device="cuda")
    before = r.clone()
    spear.rms_norm(x, weight, 1e-5, residual=r, q=q, scales=s)
    pair.forward(q, s, h)
    down.forward(*spear.quantize_rows(h), y)
    # each stage against the oracle on the stage's own inputs
    n = lambda t: t.float().cpu().numpy()
    v = w8.rms_norm(n(x), n(weight), 1e-5, n(before))[1]
    assert np.all(np.abs(n(q) * n(s)[:, None] - v) <= n(s)[:, None] * 0.51)
    arr = lambda p: (p[0].cpu().numpy(), p[1].cpu().numpy())
    want = w8.gated(*arr((q, s)), *arr(qw), *arr(qu))
    assert np.all(np.abs(n(h) - want) <= np.abs(want) * (2.0 ** -16 + 2.0 ** -8) + 1e-30)
    _equal(y, w8.linear(*w8.quantize_rows(n(h)), *arr(qd)))
    # and the whole near the block in full precision: three roundings to 8 bits, of half a step of max / 127 each
    hn = torch.nn.functional.rms_norm((x + before).double(), (K,), weight.double(), 1e-5)
    full = (torch.nn.functional.silu(hn @ W.double().t()) * (hn @ U.double().t())) @ D.double().t()
    assert (y.double() - full).norm() / full.norm() < 0.05
    pair.close(), down.close()


def test_sizes_past_32_bits_and_other_devices_are_refused():
    w = torch.zeros(32, 64, dtype=torch.int8, device="cuda")
    s = torch.ones(32, device="cuda")
    for n in ((1 << 32) + 8, 1 << 31):
        with pytest.raises(ValueError):
            spear.SpearW8Linear(w, s, max_tokens=n)
        with pytest.raises(ValueError):
            spear.w8_workspace_bytes(32, 64, n)
        with pytest.raises(ValueError):
            spear.w8_workspace_bytes(n, 64, 8)
    with pytest.raises(ValueError):
        spear.SpearW8Linear(w, s.cpu())
    layer = spear.SpearW8Linear(w, s, max_tokens=8)
    x, xs, y = torch.zeros(2, 64, dtype=torch.int8, device="cuda"), torch.ones(2, device="cuda"), torch.empty(2, 32, device="cuda")
    for args in ((x.cpu(), xs, y), (x, xs.cpu(), y), (x, xs, y.cpu())):
        with pytest.raises(ValueError):
            layer.forward(*args)
    M = (1 << 32) + 2  # views of few elements: nothing is read
    with pytest.raises(ValueError):
        layer.forward(x[:1].expand(M, 64), xs[:1].expand(M), y[:1].expand(M, 32))
    layer.forward(x, xs, y)
    assert not y.any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N", [1, 15, 17, 31, 48, 100, 257, 1026])
def test_results_of_any_alignment(N, gated, dtype):
    """Starts and distances of results that fit wide stores, and those that do not: the same bits, and nothing beside them."""
    K = 208
    w, u = _codes(N, N, K), _codes(N + 1, N, K)
    layer = _layer(w, u if gated else None, max_tokens=300)
    for M in (3, 20, 40, 209):
        x = _codes(M, M, K)
        xd = _dev(x[0]), _dev(x[1])
        want = torch.empty(M, N, dtype=dtype, device="cuda")
        layer.forward(*xd, want)
        if not gated:
            _equal(want, w8.linear(*x, *w))
        for lead, more in ((0, 0), (1, 0), (0, 1), (8, 8 - N % 8), (4, 4 - N % 4), (2, 2 + N % 2)):
            buf = torch.full((lead + M * (N + more) + 40,), 7.0, dtype=dtype, device="cuda")
            y = buf[lead:].as_strided((M, N), (N + more, 1))
            layer.forward(*xd, y)
            assert torch.equal(y, want)
            y.fill_(7.0)
            assert bool((buf == 7.0).all())
    assert layer.check() == spear.SPEAR_OK
    layer.close()
