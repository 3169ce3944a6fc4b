"""Waits of the 8-bit linears that run out: what the handle says, and that it is right again afterwards. A kernel whose
wait runs out gives up and returns, so nothing hangs."""
import numpy as np
import pytest
import torch

from oracle import w8
from quantized_linear_error_gb300 import spear

from .test_gpu_w8 import _codes, _dev, _equal, _layer

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
LIMIT = 2_000_000  # ns


def _run(layer, x):
    y = torch.full((x[0].shape[0], layer.N), 7.0, dtype=BF16, device="cuda")
    return layer.forward(_dev(x[0]), _dev(x[1]), y)


def _right(layer, x, w, u=None):
    y = _run(layer, x)
    assert layer.check() == spear.SPEAR_OK
    if u is None:
        _equal(y, w8.linear(*x, *w))
    else:  # |error| of the fast exponential and of the rounding to bf16
        want = w8.gated(*x, *w, *u)
        assert np.all(np.abs(y.float().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -15 + 2.0 ** -8) + 2.0 ** -120)


# (N, K, M): few tokens with whole row groups a CTA and with groups that CTAs share; many tokens with whole tiles (too few
# channels to split) and with tiles split along K
@pytest.mark.parametrize("N,K,M", [(128, 256, 3), (300, 8192, 9), (4864, 512, 20), (600, 256, 100), (2304, 8192, 150),
                                   (700, 4096, 40)])
@pytest.mark.parametrize("gated", [False, True])
def test_a_wait_that_runs_out_is_reported_and_recovered(N, K, M, gated):
    w, u = _codes(1, N, K), _codes(2, N, K) if gated else None
    layer, x = _layer(w, u, max_tokens=200), _codes(3, M, K)
    _right(layer, x, w, u)
    layer.debug_set(wait_ns=LIMIT, skip_arrive=True)
    _run(layer, x)
    assert layer.check() == spear.SPEAR_ERR_TIMEOUT
    layer.debug_set()
    for _ in range(2):  # counters and sums are zeros again
        _right(layer, x, w, u)
    layer.close()
