"""Packed-weight operators on the GPU against their definition in binary64, and their gradients against differences."""
import sys

import pytest

torch = pytest.importorskip("torch")

import w4_exact as E
import w4_plain as P

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def awq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import post_bit_weight_awq_amd as m
    m.load()
    return m


CHAINS = [(1, 128, 5, 32, BF16, "silu"), (40, 256, 48, 64, F16, "silu"), (7, 384, 31, 32, BF16, "gelu"),
          (130, 128, 80, 128, BF16, "silu"), (300, 512, 161, 32, F16, "gelu")]


@pytest.mark.parametrize("n,k,f,group,t,act", CHAINS, ids=str)
def test_chain_of_gradients(awq, n, k, f, group, t, act):
    """gated, its backward pass and the parameters' gradients, chained as a training step chains them."""
    _say("chain", n, k, f, group, t, act)
    layer, x, dh = E.a_chain(n, k, f, group, t, act, 5, "cuda")
    _, pre = awq.awq_w4a16_gated(x, *layer, act=act, keep_pre=True)
    dx, dpre = awq.awq_w4a16_gated_backward(dh, pre, *layer, act=act)
    ds, dz = awq.awq_w4a16_param_grad(dpre, x, *layer)
    torch.cuda.synchronize()
    chain = E.Chain(x, dh, layer, act)
    for name, got in (("x", dx), ("step", ds), ("zero", dz)):
        assert chain.agrees(name, got), name
