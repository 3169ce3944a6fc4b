"""8-bit rows and linears at the C entry points and at edges that the other tests leave out."""
import numpy as np
import pytest
import torch

from oracle import w8
from quantized_linear_error_gb300 import spear

from .test_gpu_rows import _codes_near, _near, _np, _rand
from .test_gpu_w8 import _codes, _dev, _equal, _layer

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("ld", [0, -7, 1 << 40])
def test_a_single_row_of_any_distance(ld):
    L, stream = spear.load(), torch.cuda.current_stream().cuda_stream
    K, N = 208, 40
    x, w, r = _rand(1, 1, K, dtype=BF16), _rand(2, K, dtype=BF16), _rand(3, 1, K, dtype=BF16)
    ro, y = torch.empty_like(r), torch.empty_like(x)
    q, s = torch.empty(1, K, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    p = lambda t: t.data_ptr()
    assert L.spear_rms_norm(p(x), ld, 0, p(r), ld, p(ro), ld, 0, p(w), 0, 1e-5, 1, K, p(y), ld, p(q), ld, p(s), stream) == 0
    want = torch.empty_like(x)
    spear.rms_norm(x, w, 1e-5, r.clone(), y=want)
    assert torch.equal(y, want) and torch.equal(ro, (x.float() + r.float()).bfloat16())
    assert L.spear_quantize_rows(p(x), ld, 0, 1, K, p(q), ld, p(s), stream) == 0
    assert all(torch.equal(a, b) for a, b in zip((q, s), spear.quantize_rows(x)))
    assert L.spear_dequantize_rows(p(q), ld, p(s), 1, K, p(y), ld, 0, stream) == 0
    assert torch.equal(y, spear.dequantize_rows(q, s, torch.empty_like(y)))
    weights = _codes(1, N, K)
    layer = _layer(weights)
    out = torch.empty(1, N, dtype=F32, device="cuda")
    assert L.spear_w8_forward(layer.h, p(q), ld, p(s), p(out), ld, spear.SPEAR_F32, 1, stream) == 0
    _equal(out, w8.linear(q.cpu().numpy(), s.cpu().numpy(), *weights))
    layer.close()


def _gate_of(g):
    """A gated layer whose results for a token of codes (1, 0, 0 ...) are act(g) times one."""
    N = len(g)
    w, one = np.zeros((N, 16), np.int8), np.zeros((N, 16), np.int8)
    w[:, 0], one[:, 0] = 1, 1
    return (w, g), (one, np.ones(N, np.float32))


@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 20, 40])
def test_fp32_activation_is_off_by_its_roundings_alone(activation, M):
    """g and the second projection are exact here, so that only the activation's own operations round. In half steps of
    fp32 (2^-24 of a value), with t = exp(-|z|): expf 2 of t (one step), the divisor 1 + t carries t / (1 + t) of that and
    rounds once, the quotient rounds once.
      SiLU, g > 0: 2 t / (1 + t) + 1 + 1 <= 3. g < 0: g t rounds once more and t's own error stays in part, 2 / (1 + t), so
      2 + 1 + 1 + 1 = 5.
      GELU: z's constants, products and sum are 7 at most, which exp turns into 7 |z| of t, so 7 |z| t / (1 + t) <= 2
      more for g > 0 and 7 |z| for g < 0.
    Second orders are below 2^-10 of these."""
    rng = np.random.default_rng(M)
    top = 80 if activation == "silu" else 9
    g = np.concatenate([rng.uniform(-top, top, 20000), rng.uniform(-3, 3, 40000), rng.normal(0, 1, 5000)]).astype(np.float32)
    w, u = _gate_of(g)
    layer = _layer(w, u, max_tokens=64, activation=activation)
    x = np.zeros((M, 16), np.int8)
    x[:, 0] = 1
    y = torch.empty(M, len(g), dtype=F32, device="cuda")
    layer.forward(_dev(x), _dev(np.ones(M, np.float32)), y)
    y = y.cpu().numpy().astype(np.float64)
    assert np.array_equal(y, np.broadcast_to(y[:1], y.shape))
    want = w8.act(g, activation)
    z = np.abs(g.astype(np.float64))
    if activation == "gelu":
        z = 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    steps = np.where(g > 0, 3.0, 5.0)
    if activation == "gelu":
        steps += np.where(g > 0, 2.0, 7 * z)
    off = np.abs(y[0] - want) / np.abs(want) * 2.0 ** 24
    print(activation, M, "half steps off: g > 0", off[g > 0].max(), "g < 0", off[g < 0].max(), "mean", off.mean())
    assert np.all(off <= steps * (1 + 2.0 ** -10))
    layer.close()


@pytest.mark.parametrize("M", [1, 40])
def test_fp32_activation_of_the_ends(M):
    g = np.array([0.0, -0.0, np.inf, np.nan, 3e38, -3e38, 1e30, -1e30, 200.0, -200.0, 2.0 ** -140, -2.0 ** -140, 2.0 ** -149],
                 np.float32)
    w, u = _gate_of(g)
    for activation in ("silu", "gelu"):
        layer = _layer(w, u, max_tokens=64, activation=activation)
        x = np.zeros((M, 16), np.int8)
        x[:, 0] = 1
        y = torch.empty(M, len(g), dtype=F32, device="cuda")
        layer.forward(_dev(x), _dev(np.ones(M, np.float32)), y)
        y = y.cpu().numpy()
        for row in y:
            assert row[0] == 0 and row[1] == 0 and row[2] == np.inf and np.isnan(row[3])
            assert np.array_equal(row[[4, 6, 8]], g[[4, 6, 8]]) and not row[[5, 7, 9]].any()
            # half of g, of the denormal numbers too
            assert np.all(np.abs(row[10:].astype(np.float64) - g[10:].astype(np.float64) / 2) <= 2.0 ** -149)
        layer.close()


@pytest.mark.parametrize("M", [1, 20, 40])
def test_fp32_quotient_rounds_once(M):
    """SiLU's bound of the test above, element by element, where exp's part fades: for g > 0 2 t / (1 + t) half steps come
    of t, one of the divisor's rounding and one of the quotient's; for g < 0 2 / (1 + t), and one more of g t. A quotient
    of two steps' error is beyond it."""
    rng = np.random.default_rng(100 + M)
    g = np.concatenate([rng.uniform(2, 12, 100000), -rng.uniform(0, 1, 20000)]).astype(np.float32)
    w, u = _gate_of(g)
    layer = _layer(w, u, max_tokens=64)
    x = np.zeros((M, 16), np.int8)
    x[:, 0] = 1
    y = torch.empty(M, len(g), dtype=F32, device="cuda")
    layer.forward(_dev(x), _dev(np.ones(M, np.float32)), y)
    want, t = w8.act(g, "silu"), np.exp(-np.abs(g.astype(np.float64)))
    bound = np.where(g > 0, 2 * t / (1 + t) + 2, 2 / (1 + t) + 3)
    off = np.abs(y[0].cpu().numpy().astype(np.float64) - want) / np.abs(want) * 2.0 ** 24
    print(M, "largest share of the bound", (off / bound)[g > 0].max(), (off / bound)[g < 0].max())
    assert np.all(off <= bound * (1 + 2.0 ** -10))
    layer.close()


@pytest.mark.parametrize("activation", ["silu", "gelu"])
@pytest.mark.parametrize("N,K", [(8, 64), (15, 96), (129, 272), (1000, 1040), (2048, 4096)])
def test_gated_f16_results(N, K, activation):
    """The bound of bf16 results (the fast exponential: 2^-15 of SiLU, 2^-14 of GELU), with f16's rounding and, below its
    normal numbers, half its smallest step."""
    w, u = _codes(N, N, K), _codes(N + 1, N, K)
    layer = _layer(w, u, max_tokens=300, activation=activation)
    rel, half = 2.0 ** (-15 if activation == "silu" else -14), 2.0 ** -11
    for M in (1, 7, 16, 30, 33, 130, 260):
        x = _codes(M, M, K)
        want = w8.gated(*x, *w, *u, activation)
        assert np.abs(want).max() < 60000
        y = torch.full((M, N), 7.0, dtype=F16, device="cuda")
        layer.forward(_dev(x[0]), _dev(x[1]), y)
        y = y.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(y - want) <= np.abs(want) * (rel + half * (1 + rel)) + 2.0 ** -25)
    assert layer.check() == spear.SPEAR_OK
    layer.close()


PAIRS = [(BF16, BF16, BF16), (BF16, F32, BF16), (F16, F16, F32), (F16, F32, F16), (F32, F32, F32), (BF16, BF16, F32)]
ROWS = [1, 7, 250, 256, 257, 512, 517, 1000, 1016, 1024, 1032, 4096, 4100, 8200, 11008, 12296, 16384, 20488, 28671, 32768]


@pytest.mark.parametrize("i,K", list(enumerate(ROWS)))
@pytest.mark.parametrize("M", [4, 150])
def test_norm_with_a_residual_in_all_outputs(i, K, M):
    """Few rows: the kernels that take a row and end, on what the residual's addition leaves in fp32."""
    for x, res, weight in (PAIRS[i % 6], PAIRS[(i + 3) % 6]):
        X, W, R = _rand(K, M, K, dtype=x), _rand(K + 1, K, dtype=weight) + 1, _rand(K + 2, M, K, dtype=res, scale=3.0)
        ro, y = torch.empty_like(R), torch.empty_like(X)
        q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        spear.rms_norm(X, W, 1e-5, R, ro, y, q, s)
        h = X.float() + R.float()
        assert torch.equal(ro, h.to(res))
        v = w8.rms_norm(_np(h), _np(W), 1e-5)[1]
        _near(y, v, x)
        _codes_near(q, s, v)
        y1, q1, s1 = torch.empty_like(y), torch.empty_like(q), torch.empty_like(s)
        spear.rms_norm(X, W, 1e-5, R.clone(), y=y1)
        spear.rms_norm(X, W, 1e-5, R, q=q1, scales=s1)  # in place
        assert torch.equal(y1, y) and torch.equal(q1, q) and torch.equal(s1, s) and torch.equal(R, ro)


@pytest.mark.parametrize("N,K", [(8, 16), (4096, 4096), (8192, 28672), (64, 1 << 20)])
@pytest.mark.parametrize("gated", [False, True])
def test_the_workspace_is_what_the_header_says(N, K, gated):
    """1.2 MB, or 16.2 MB + K (512 + 2.25 max_tokens) bytes: within 2% (the figures are rounded)."""
    wide = (K + 127) // 128 * 128
    weights = wide * ((N * (2 if gated else 1) + 127) // 128 * 128)
    for tokens in (1, 16, 17, 32, 33, 64, 1000, 100000):
        many = tokens > 32 or (tokens > 16 and weights > 36 << 20)
        want = 16.2e6 + wide * (512 + 2.25 * tokens) if many else 1.2e6
        got = spear.w8_workspace_bytes(N, K, tokens, gated)
        assert abs(got - want) <= 0.02 * want + (wide * 2 if many else 0.04 * want), (tokens, got, want)
