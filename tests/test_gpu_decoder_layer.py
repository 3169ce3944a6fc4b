"""The decoder of the example: a chunk, then decode steps from a graph. Every stage around the attention block (which has
its own test) is compared with its definition on what the stage before handed on."""
import numpy as np
import pytest
import torch

from examples import decoder_layer as dl
from oracle import w8

pytestmark = pytest.mark.gpu


def _n(t):
    return t.float().cpu().numpy()


def _pair(p):
    return p[0].cpu().numpy(), p[1].cpu().numpy()


def _near(got, want):
    """bf16 results of values within 2^-15 of `want`."""
    assert np.all(np.abs(_n(got) - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -15) + 1e-30)


def _follow(d, x, y):
    """After a step of a one-layer decoder over the rows x."""
    T, ff = x.shape[0], d.ffs[0]
    _near(d.h[:T], w8.rms_norm(_n(x), _n(d.norms[0]), d.eps)[1])
    mid = (x.float() + d.attn[:T].float()).bfloat16()  # the residual that the final norm adds to
    h, v = w8.rms_norm(_n(x) + _n(d.attn[:T]), _n(d.norms[1]), d.eps)
    s = _n(d.scales[:T])
    assert np.all(np.abs(_n(d.q[:T]) * s[:, None] - v) <= s[:, None] * 0.51)
    q, sc = _pair((d.q[:T], d.scales[:T]))
    _near(ff.g[:T], w8.gated(q, sc, *_pair(ff.gate), *_pair(ff.up)))
    fq, fs = w8.quantize_rows(_n(ff.g[:T]))
    assert np.array_equal(ff.q[:T].cpu().numpy(), fq) and np.array_equal(_n(ff.scales[:T]), fs)
    want = torch.from_numpy(w8.linear(fq, fs, *_pair(ff.down_weight))).bfloat16()
    assert torch.equal(d.delta[:T].cpu(), want)
    total = mid.float() + d.delta[:T].float()
    assert torch.equal(d.residual[:T], total.bfloat16())
    _near(y, w8.rms_norm(_n(total), _n(d.norms[2]), d.eps)[1])


def test_chunk_and_graph_decode_stage_by_stage():
    d = dl.Decoder(1, hidden=512, width=768, n_heads=8, n_kv_heads=2, page_size=16, n_pages=32, max_tokens=128,
                   max_positions=512, rank=32)
    torch.manual_seed(5)
    seqs = dl.Sequences(d, 2, 160)
    for s, T in ((0, 90), (1, 17), (0, 33)):
        x = torch.randn(T, 512, device="cuda").bfloat16()
        y = torch.empty_like(x)
        seqs.prefill(s, x, y)
        _follow(d, x, y)
    x = torch.randn(2, 512, device="cuda").bfloat16()
    y = torch.empty_like(x)
    graph = seqs.decode_graph(x, y)
    for _ in range(3):
        x.copy_(torch.randn(2, 512, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        _follow(d, x, y)
    assert seqs.lens.tolist() == [126, 20] and d.check()
    d.close()


def test_the_example_runs(capsys):
    dl.main(["--steps", "3", "--prompt", "70", "--layers", "2"])
    out = capsys.readouterr().out
    assert "lengths [73, 39]" in out and "status ok" in out
