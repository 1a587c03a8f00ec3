"""What the packed-weight bindings refuse before anything reaches the GPU."""
import pytest
import torch

import post_bit_weight_awq_amd as awq
import w4_plain as P

CALLS = {
    "awq_w4a16_linear": lambda x, l: awq.awq_w4a16_linear(x, *l),
    "awq_w4a16_gated": lambda x, l: awq.awq_w4a16_gated(x, *l),
    "awq_w4a16_input_grad": lambda x, l: awq.awq_w4a16_input_grad(x, *l),
    "awq_w4a16_gated_backward": lambda x, l: awq.awq_w4a16_gated_backward(x, x, *l),
    "awq_w4a16_param_grad": lambda x, l: awq.awq_w4a16_param_grad(x, x, *l),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_that_requires_a_gradient(name):
    """Refused while gradients are recorded; elsewhere the call goes on (here to the refusal of CPU tensors)."""
    layer = P.make_layer(8, 256, 64, 0)
    x = torch.zeros(2, 256, dtype=torch.float16, requires_grad=True)
    with pytest.raises(RuntimeError, match="requires a gradient"):
        CALLS[name](x, layer)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        CALLS[name](x, layer)
