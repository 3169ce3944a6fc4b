"""check() of the examples asks every handle, whatever those before it say: a check also makes its handle fit again."""
import pytest

from examples.attention_block import AttentionBlock
from examples.decoder_layer import Decoder
from quantized_linear_error_gb300 import spear


class Handle:
    def __init__(self, status):
        self.status, self.asked = status, 0

    def check(self):
        self.asked += 1
        status, self.status = self.status, spear.SPEAR_OK
        return status


class Block:
    def __init__(self, ok):
        self.ok, self.asked = ok, 0

    def check(self):
        self.asked += 1
        return self.ok


@pytest.mark.parametrize("bad", [(), (0,), (1,), (0, 2), (0, 1, 2)])
def test_attention_block(bad):
    block = AttentionBlock.__new__(AttentionBlock)
    handles = [Handle(spear.SPEAR_ERR_TIMEOUT if i in bad else spear.SPEAR_OK) for i in range(3)]
    block.qkv, block.cache, block.o = handles
    assert block.check() == (not bad)
    assert [h.asked for h in handles] == [1, 1, 1]
    assert block.check()


@pytest.mark.parametrize("bad_blocks", [(), (0,), (1,)])
@pytest.mark.parametrize("bad", [(), (0,), (1, 2), (3,)])
def test_decoder(bad, bad_blocks):
    d = Decoder.__new__(Decoder)
    d.blocks = [Block(i not in bad_blocks) for i in range(2)]
    handles = [Handle(spear.SPEAR_ERR_TIMEOUT if i in bad else spear.SPEAR_OK) for i in range(4)]

    class FF:
        def __init__(self, pair, down):
            self.pair, self.down = pair, down

    d.ffs = [FF(*handles[:2]), FF(*handles[2:])]
    assert d.check() == (not bad and not bad_blocks)
    assert [b.asked for b in d.blocks] == [1, 1] and [h.asked for h in handles] == [1] * 4
