"""An attention block of a decoder layer, served from quantised weights and a quantised cache.

W4 + compensator linears (q/k/v as one grouped handle, o), the paged 4-bit key/value cache and the attention over it:

    qkv = W_qkv x;  rotate q and k, append k and v;  a = attention(q);  y = W_o a

Two prompts go in as chunks, then both sequences decode token by token; the decode step is captured once in a CUDA
graph, in which positions, slots and lengths advance on the device. Weights and inputs are random.

    python examples/attention_block.py [--steps 64] [--prompt 1000]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_linear_error_gb300 import spear  # noqa: E402
from quantized_linear_error_gb300 import workload as wl  # noqa: E402


class AttentionBlock:
    """One block's weights and cache. ``tokens`` x, lengths and tables come from the caller, as a server has them."""

    def __init__(self, hidden=4096, n_heads=32, n_kv_heads=8, page_size=64, n_pages=256, max_tokens=2048,
                 max_positions=32768, rank=64, seed=0):
        self.n_heads, self.n_kv_heads, self.D = n_heads, n_kv_heads, hidden // n_heads
        self.page_size, self.max_tokens = page_size, max_tokens
        kv = n_kv_heads * self.D
        specs = [wl.LinearSpec(n, hidden, N, 128, rank) for n, N in (("q", hidden), ("k", kv), ("v", kv))]
        self.weights = [wl.make_weights(s, seed, "block/") for s in specs]
        self.o_weights = wl.make_weights(wl.LinearSpec("o", hidden, hidden, 128, rank), seed, "block/")
        self.qkv = spear.grouped_from_weights(self.weights, max_tokens=max_tokens)
        self.o = spear.from_weights(self.o_weights, max_tokens=max_tokens)
        self.pool = spear.kv_pool(n_pages, n_kv_heads, self.D, page_size)
        self.cache = spear.SpearKVCache(n_heads, n_kv_heads, self.D, page_size, self.pool,
                                        spear.rope_table(max_positions, self.D))
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.qkv_out = torch.empty(max_tokens, hidden + 2 * kv, **bf16)
        self.attn_out = torch.empty(max_tokens, n_heads, self.D, **bf16)

    def forward(self, x, y, positions, slots, page_table, kv_lens, q_starts, max_q):
        """x, y bf16 [T][hidden]; the index tensors as SpearKVCache.append and .attention take them."""
        T, H, G = x.shape[0], self.n_heads, self.n_kv_heads
        rows = self.qkv_out[:T]
        self.qkv.forward(x, rows)
        heads = rows.view(T, H + 2 * G, self.D)
        q = self.cache.append(heads[:, :H], heads[:, H:H + G], heads[:, H + G:], positions, slots)  # q rotated in place
        a = self.cache.attention(q, self.attn_out[:T], page_table, kv_lens, q_starts, max_q)
        return self.o.forward(a.view(T, -1), y)

    def check(self) -> bool:
        return all(x.check() == spear.SPEAR_OK for x in (self.qkv, self.cache, self.o))

    def close(self):
        for x in (self.qkv, self.cache, self.o):
            x.close()


class Sequences:
    """Page tables and lengths of a few sequences on the device: what a scheduler keeps."""

    def __init__(self, block, n_seqs, max_len):
        self.block, self.n = block, n_seqs
        cols = -(-max_len // block.page_size)
        pages = torch.randperm(block.pool.shape[0])[:n_seqs * cols]
        self.table = pages.view(n_seqs, cols).to(torch.int32).cuda()
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        # read by the captured step, so kept as long as the object
        self.starts = torch.arange(n_seqs + 1, dtype=torch.int32, device="cuda")
        self.which = torch.arange(n_seqs, device="cuda")

    def slots_of(self, seq, positions):
        """Slot numbers of positions (int64, on the device) of sequences seq (a number or int64 tensor)."""
        p = self.block.page_size
        return self.table.long()[seq, positions // p] * p + positions % p

    def prefill(self, seq, x, y):
        """The next tokens of one sequence, as one chunk."""
        T, start = x.shape[0], int(self.lens[seq])
        positions = torch.arange(start, start + T, device="cuda")
        self.lens[seq] += T
        self.block.forward(x, y, positions, self.slots_of(seq, positions), self.table[seq:seq + 1],
                           self.lens[seq:seq + 1], torch.tensor([0, T], dtype=torch.int32, device="cuda"), T)

    def decode_graph(self, x, y):
        """A graph of one decode step of all sequences (one token each): x [n_seqs][hidden] in, y out. Whoever replays
        it keeps this object, the block, x and y."""

        def step():
            positions = self.lens.long()
            slots = self.slots_of(self.which, positions)
            self.lens += 1
            self.block.forward(x, y, positions, slots, self.table, self.lens, self.starts, 1)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # a first step outside the graph; its length and slot are used again
            step()
            self.lens -= 1
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        return graph


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=1000)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    block = AttentionBlock(max_tokens=max(32, a.prompt))
    seqs = Sequences(block, 2, a.prompt + a.steps + 1)
    hidden = block.n_heads * block.D
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
        graph.replay()  # a server writes the next tokens' activations to xd between replays
    t1.record()
    torch.cuda.synchronize()
    print(f"lengths {seqs.lens.tolist()}, {t0.elapsed_time(t1) / a.steps * 1e3:.1f} us a decode step, "
          f"status {'ok' if block.check() else 'error'}")
    block.close()


if __name__ == "__main__":
    main()
