"""What Decoder looks up for a token that is none (-1): no index leaves the embedding, on a stand-in for the block."""
import pytest

torch = pytest.importorskip("torch")

HIDDEN, VOCAB = 64, 10


class Block:
    def step(self, x, n_new, tree=None):
        return torch.zeros_like(x, dtype=torch.float32), "maps"

    def _product(self, W, x):
        return x.float()


def decoder(vocab=VOCAB, rows=VOCAB, **kw):
    from weight_quantized_decode_gb300.decode_block import Decoder
    embedding = torch.arange(vocab * HIDDEN).reshape(vocab, HIDDEN).half()
    return Decoder(Block(), embedding, torch.zeros(rows, HIDDEN // 32 * 18, dtype=torch.uint8)), embedding


def test_no_token_is_looked_up_as_the_first():
    d, embedding = decoder()
    tokens = torch.tensor([3, -1, 9, 0, -1], dtype=torch.int32)
    rows, maps = d.logits(tokens, None)
    assert torch.equal(rows, embedding[[3, 0, 9, 0, 0]].float()) and maps == "maps"
    assert tokens.tolist() == [3, -1, 9, 0, -1]


def test_a_head_with_more_tokens_than_the_embedding():
    """Its tokens would be looked up past the embedding's end."""
    decoder(VOCAB, VOCAB - 1)
    decoder(VOCAB + 1, VOCAB)
    with pytest.raises(ValueError):
        decoder(VOCAB, VOCAB + 1)
