"""What the layer of experts refuses, decided before anything touches a GPU."""
import pytest
import torch

from w8a8_int8_quantized_norm_b200 import moe


@pytest.mark.parametrize("shape", [(6, 4), (4, 4), (5, 3), (5, 5), (5,)])
def test_layer_refuses_logits_of_other_tokens_or_experts(shape):
    """More rows than tokens would become rows of zeros, fewer would drop tokens."""
    layer = moe.MoELayer(torch.zeros(4, 64, 32), torch.zeros(4, 32, 32), 2)
    layer.gate_up_q = layer.gate_up_scale = layer.down_q = layer.down_scale = None  # not reached
    with pytest.raises(ValueError, match=r"logits must be \[T, E\] = \[5, 4\]"):
        layer.forward(torch.zeros((5, 32), dtype=torch.int8), torch.zeros(5), torch.zeros(shape))
