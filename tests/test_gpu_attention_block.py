"""The quantised attention block of the example: chunks, then decode steps from a graph. Every stage is compared with
its own definition on what the stage before handed on: the linears with the layer's oracle and its tolerance, the
cache's bytes bit for bit, attention within the bound that its oracle derives."""
import numpy as np
import pytest
import torch

from examples import attention_block as ab
from oracle import kv, ref

from .helpers import bits_of, rel_err

pytestmark = pytest.mark.gpu
TOL = 1e-2  # of the linears


class Follower:
    """Keeps the bytes that the pool should hold, and checks one step of the block at a time."""

    def __init__(self, block, seqs):
        self.b, self.s = block, seqs
        self.pool = block.pool.cpu().numpy().copy()

    def step(self, x, y, seq_of, positions):
        """After a step over the rows x: row i is the token at positions[i] of sequence seq_of[i]."""
        b = self.b
        H, G, D, T = b.n_heads, b.n_kv_heads, b.D, len(positions)
        xb = bits_of(x)
        rows = torch.empty(T, (H + 2 * G) * D, dtype=torch.bfloat16, device="cuda")
        b.qkv.forward(x, rows)
        got = rows.float().cpu().numpy()
        at = 0
        for w in b.weights:
            assert rel_err(got[:, at:at + w.spec.N].astype(np.float64), ref.forward_w(w, xb)) <= TOL
            at += w.spec.N
        heads = got.reshape(T, H + 2 * G, D)
        turn = b.cache.rope_table.cpu().numpy()[positions]
        q, k = (kv.rotate(t, turn, False) for t in (heads[:, :H], heads[:, H:H + G]))
        slots = np.array([int(self.s.slots_of(int(s), torch.tensor([p], device="cuda"))) for s, p in zip(seq_of, positions)])
        kv.pack_rows(self.pool, b.page_size, D, slots, *kv.quantise(k), *kv.quantise(heads[:, H + G:]))
        np.testing.assert_array_equal(b.pool.cpu().numpy(), self.pool)
        q = kv.bf16_value(kv.bf16_bits(q)).astype(np.float64)
        attn = b.attn_out[:T].float().cpu().numpy().astype(np.float64)
        for s in sorted(set(seq_of)):
            mine = [i for i in range(T) if seq_of[i] == s]
            L = positions[mine[-1]] + 1
            K, V = kv.unpack_rows(self.pool, b.page_size, D, self.s.slots_of(int(s), torch.arange(L, device="cuda")).cpu().numpy())
            want, mag, big = kv.attention(q[mine], K, V, D ** -0.5)
            assert np.all(np.abs(attn[mine] - want) <= kv.tolerance(want, mag, big)), f"sequence {s}, length {L}"
        want = ref.forward_w(b.o_weights, bits_of(b.attn_out[:T]).reshape(T, -1))
        assert rel_err(y.float().cpu().numpy().astype(np.float64), want) <= TOL


def test_chunks_and_graph_decode_stage_by_stage():
    """Both sequences' prompts (one in two chunks), then four decode steps by graph replay."""
    block = ab.AttentionBlock(hidden=512, n_heads=8, n_kv_heads=2, page_size=16, n_pages=32, max_tokens=128,
                              max_positions=512, rank=32)
    torch.manual_seed(3)
    seqs = ab.Sequences(block, 2, 160)
    follower = Follower(block, seqs)
    at = [0, 0]
    for s, T in ((0, 90), (1, 37), (0, 33)):
        x = torch.randn(T, 512, device="cuda").bfloat16()
        y = torch.empty_like(x)
        seqs.prefill(s, x, y)
        follower.step(x, y, [s] * T, np.arange(at[s], at[s] + T))
        at[s] += T
    x = torch.zeros(2, 512, device="cuda").bfloat16()
    y = torch.empty_like(x)
    graph = seqs.decode_graph(x, y)
    assert seqs.lens.tolist() == at
    for _ in range(4):
        x.copy_(torch.randn(2, 512, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        follower.step(x, y, [0, 1], np.array(at))
        at = [n + 1 for n in at]
    assert seqs.lens.tolist() == at and block.check()
    block.close()


def test_the_example_runs(capsys):
    ab.main(["--steps", "3", "--prompt", "70"])
    out = capsys.readouterr().out
    assert "lengths [73, 39]" in out and "status ok" in out  # prompts of 70 and 36 tokens
