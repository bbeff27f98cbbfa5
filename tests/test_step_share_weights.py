"""Steps that share weights have to agree on every size that the weights fix: their outputs are written into the new step's
buffers (no GPU: a step that does not fit is refused before anything is allocated)."""
import pytest

from nvfp4_w4a4_decode_gemv_gb300.decode_step import DecodeStep
from nvfp4_w4a4_decode_gemv_gb300.serving_step import ServingStep

SHAPES = [("qkv", 512, 1024), ("o", 512, 512), ("gate_up", 512, 256), ("down", 128, 512)]


class Step:
    """What another step says of its weights."""

    def __init__(self, **other):
        self.layers, self.hidden, self.vocab, self.n_qkv, self.k_o, self.n_gu, self.k_d = 2, 512, 1000, 1024, 512, 256, 128
        self.experts, self.weights, self.rowmajor, self.routers, self.lm_head = 0, [], [], [], None
        self.__dict__.update(other)


@pytest.mark.parametrize("what", ["layers", "hidden", "vocab", "n_qkv", "k_o", "n_gu", "k_d", "experts"])
def test_dense_steps(what):
    other = Step()
    setattr(other, what, getattr(other, what) + 64)
    with pytest.raises(ValueError, match=what):
        DecodeStep(1, 2, shapes=SHAPES, vocab=1000, share_weights=other)


@pytest.mark.parametrize("there,here", [(0, 12), (12, 0), (16, 12), (8, 12)])
def test_numbers_of_experts(there, here):
    with pytest.raises(ValueError, match="experts"):
        ServingStep(1, 2, 4, 2, 128, 16, 40, max_len=200, shapes=SHAPES, vocab=1000, experts=here, router={"top_k": 3},
                    share_weights=Step(experts=there))
