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


def test_gelu_is_the_tanh_form_by_either_name():
    assert awq._w4_act("gelu") == awq._w4_act("gelu_tanh") != awq._w4_act("silu")
    for name in ("gelu_erf", "tanh", "relu", ""):
        with pytest.raises(ValueError, match="act must be one of"):
            awq._w4_act(name)
    assert "not the erf one" in awq.awq_w4a16_gated.__doc__
    # the plain form the tests hold the kernels to is torch's tanh form
    g = torch.linspace(-6, 6, 201, dtype=torch.float64)
    assert torch.allclose(P.act(g, "gelu")[0], torch.nn.functional.gelu(g, approximate="tanh"), rtol=0, atol=1e-14)


def test_a_stream_of_another_device_is_refused():
    class Stream:
        cuda_stream = 5

        def __init__(self, device_index):
            self.device_index = device_index

    assert awq._w4_stream(Stream(0), 0) == 5
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        awq._w4_stream(Stream(1), 0)
