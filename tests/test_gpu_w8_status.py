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


def _pair_on_one_workspace(N=2304, K=8192, most=200):
    """Two layers on one workspace, whose tiles are split along K for 150 tokens, and their weights."""
    ws = torch.zeros(spear.w8_workspace_bytes(N, K, most), dtype=torch.uint8, device="cuda")
    w = [_codes(i, N, K) for i in range(2)]
    return [spear.SpearW8Linear(_dev(a[0]), _dev(a[1]), max_tokens=most, workspace=ws) for a in w], w, _codes(5, 150, K)


def _give_up(layer, x):
    layer.debug_set(wait_ns=LIMIT, skip_arrive=True)
    _run(layer, x)
    layer.debug_set()


@pytest.mark.parametrize("checked_first", ["the other", "the failed", "none"])
def test_a_failed_call_does_not_spoil_others_on_the_workspace_unseen(checked_first):
    """What a call that gave up leaves in a shared workspace: a layer that meets it says so, until a check."""
    (a, b), w, x = _pair_on_one_workspace()
    _right(a, x, w[0]), _right(b, x, w[1])
    _give_up(a, x)
    assert b.check() == spear.SPEAR_OK  # nothing of b's has run since
    if checked_first == "the other":  # b runs on what a has left
        y = _run(b, x)
        assert b.check() == spear.SPEAR_ERR_TIMEOUT or torch.equal(y.cpu(), torch.from_numpy(w8.linear(*x, *w[1])).to(BF16))
        _right(b, x, w[1])
        assert a.check() == spear.SPEAR_ERR_TIMEOUT  # a's own result is still wrong
    elif checked_first == "the failed":
        assert a.check() == spear.SPEAR_ERR_TIMEOUT
        _right(b, x, w[1])
    else:  # a goes without a check
        a.close()
        y = _run(b, x)
        assert b.check() == spear.SPEAR_ERR_TIMEOUT or torch.equal(y.cpu(), torch.from_numpy(w8.linear(*x, *w[1])).to(BF16))
        _right(b, x, w[1])
        return
    for _ in range(2):
        _right(a, x, w[0]), _right(b, x, w[1])
    a.close(), b.close()


def test_few_tokens_and_whole_tiles_do_not_depend_on_a_failed_call():
    (a, b), w, x = _pair_on_one_workspace()
    few = x[0][:9], x[1][:9]
    narrow = _codes(9, 260, 256)  # few channels: no tile is split
    c = spear.SpearW8Linear(_dev(narrow[0]), _dev(narrow[1]), max_tokens=200, workspace=b.workspace)
    _give_up(a, x)
    _right(b, few, w[1])
    xc = _codes(6, 100, 256)
    _right(c, xc, narrow)
    # and one that gives up itself without split tiles leaves the others alone
    assert a.check() == spear.SPEAR_ERR_TIMEOUT
    _give_up(c, xc)
    _right(b, x, w[1])
    assert c.check() == spear.SPEAR_ERR_TIMEOUT
    for layer in (a, b, c):
        layer.close()
