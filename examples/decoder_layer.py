"""A small decoder served with 4-bit attention and an 8-bit feed-forward block.

Each layer: norm, the attention block of ``attention_block.py`` (W4 + compensator linears, 4-bit cache), then

    residual += attention;  q, s = norm(residual) in 8 bits;  g = silu(q G^T) * (q U^T);  g in 8 bits;  delta = g D^T

and the next layer's norm adds delta to the residual. Layers share the workspace of their 8-bit linears. Two prompts go in
as chunks, then both sequences decode token by token from one CUDA graph. Weights and inputs are random.

    python examples/decoder_layer.py [--steps 64] [--prompt 1000] [--layers 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.attention_block import AttentionBlock, Sequences  # noqa: E402
from quantized_linear_error_gb300 import spear  # noqa: E402


class FeedForward:
    """Gate, up and down projections in 8 bits, quantised from random weights."""

    def __init__(self, hidden, width, max_tokens, workspace, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return spear.quantize_rows(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)

        self.gate, self.up, self.down_weight = weight(width, hidden), weight(width, hidden), weight(hidden, width)
        self.pair = spear.SpearW8Linear(*self.gate, max_tokens=max_tokens, up=self.up[0], up_scales=self.up[1],
                                        workspace=workspace)
        self.down = spear.SpearW8Linear(*self.down_weight, max_tokens=max_tokens, workspace=workspace)
        self.g = torch.empty(max_tokens, width, dtype=torch.bfloat16, device="cuda")
        self.q = torch.empty(max_tokens, width, dtype=torch.int8, device="cuda")
        self.scales = torch.empty(max_tokens, device="cuda")

    def forward(self, q, scales, y):
        """y bf16 [T][hidden] of the 8-bit rows q, scales."""
        T = q.shape[0]
        self.pair.forward(q, scales, self.g[:T])
        spear.quantize_rows(self.g[:T], self.q[:T], self.scales[:T])
        return self.down.forward(self.q[:T], self.scales[:T], y)


class Decoder:
    """``forward`` has the arguments of AttentionBlock.forward, so that Sequences drives it; all layers' caches have the
    same pages in use."""

    def __init__(self, n_layers=2, hidden=4096, width=14336, n_heads=32, n_kv_heads=8, page_size=64, n_pages=256,
                 max_tokens=2048, max_positions=32768, rank=64, eps=1e-5, seed=0):
        self.eps, self.page_size = eps, page_size
        room = max(spear.w8_workspace_bytes(width, hidden, max_tokens, gated=True),
                   spear.w8_workspace_bytes(hidden, width, max_tokens))
        self.workspace = torch.empty(room, dtype=torch.uint8, device="cuda")
        self.blocks = [AttentionBlock(hidden, n_heads, n_kv_heads, page_size, n_pages, max_tokens, max_positions, rank,
                                      seed + i) for i in range(n_layers)]
        self.ffs = [FeedForward(hidden, width, max_tokens, self.workspace, seed + i) for i in range(n_layers)]
        g = torch.Generator(device="cuda").manual_seed(seed + 1000)
        self.norms = [(1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).bfloat16() for _ in range(2 * n_layers + 1)]
        self.pool = self.blocks[0].pool  # its size is what Sequences asks for
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.residual, self.h, self.attn, self.delta = (torch.empty(max_tokens, hidden, **bf16) for _ in range(4))
        self.q = torch.empty(max_tokens, hidden, dtype=torch.int8, device="cuda")
        self.scales = torch.empty(max_tokens, device="cuda")

    def forward(self, x, y, *where):
        """y bf16 [T][hidden]: the final norm of the residual stream that starts as x."""
        T = x.shape[0]
        residual, h, attn, delta, q, scales = (t[:T] for t in (self.residual, self.h, self.attn, self.delta, self.q, self.scales))
        residual.copy_(x)
        for i, (block, ff) in enumerate(zip(self.blocks, self.ffs)):
            if i == 0:
                spear.rms_norm(residual, self.norms[0], self.eps, y=h)
            else:
                spear.rms_norm(delta, self.norms[2 * i], self.eps, residual, y=h)
            block.forward(h, attn, *where)
            spear.rms_norm(attn, self.norms[2 * i + 1], self.eps, residual, q=q, scales=scales)
            ff.forward(q, scales, delta)
        spear.rms_norm(delta, self.norms[-1], self.eps, residual, y=y)
        return y

    def check(self) -> bool:
        # each of them: a check also makes its handle fit again
        return all([b.check() for b in self.blocks] + [x.check() == spear.SPEAR_OK for f in self.ffs for x in (f.pair, f.down)])

    def close(self):
        for b in self.blocks:
            b.close()
        for f in self.ffs:
            f.pair.close(), f.down.close()


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    decoder = Decoder(a.layers, max_tokens=max(32, a.prompt))
    seqs = Sequences(decoder, 2, a.prompt + a.steps + 1)
    hidden = decoder.residual.shape[1]
    x = torch.randn(a.prompt, hidden, device="cuda").bfloat16()
    y = torch.empty_like(x)
    for s, n in enumerate((a.prompt, a.prompt // 2 + 1)):
        seqs.prefill(s, x[:n], y[:n])
    xd = torch.randn(2, hidden, device="cuda").bfloat16()
    yd = torch.empty_like(xd)
    graph = seqs.decode_graph(xd, yd)
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    for _ in range(a.steps):
        graph.replay()  # a server writes the next tokens' embeddings to xd between replays
    t1.record()
    torch.cuda.synchronize()
    print(f"lengths {seqs.lens.tolist()}, {t0.elapsed_time(t1) / a.steps * 1e3:.1f} us a decode step of {a.layers} layers, "
          f"status {'ok' if decoder.check() else 'error'}")
    decoder.close()


if __name__ == "__main__":
    main()
