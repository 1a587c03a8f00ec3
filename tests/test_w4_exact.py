"""The checks of w4_exact.py themselves, without a GPU: right gradients pass, mistaken ones do not."""
import pytest
import torch

import w4_exact as E
import w4_plain as P

CHAINS = [(40, 256, 48, 64, torch.float16, "silu"), (7, 384, 31, 32, torch.bfloat16, "gelu"),
          (130, 128, 80, 128, torch.bfloat16, "silu")]


def plain_gradients(layer, x, dh, act):
    """The run's gradients from the definition, rounded where the operators round."""
    t = x.dtype
    w = E.weights(*layer)
    pre = (x.to(P.F64) @ w.T).to(t)
    dpre = P.gated_grad(dh, pre, act)[0].to(t).to(P.F64)
    dx = (dpre @ w.to(torch.float16).to(P.F64)).to(t)
    o, ng = layer[1].shape
    d = (dpre.T @ x.to(P.F64)).view(o, ng, -1)
    ds = (d * E.differences(layer[0], layer[2]).view(d.shape)).sum(-1)
    return {"x": dx.to(P.F64), "step": ds, "zero": -layer[1].to(P.F64) * d.sum(-1)}, dpre, d


@pytest.mark.parametrize("n,k,f,group,t,act", CHAINS, ids=str)
def test_the_directional_check_bites(n, k, f, group, t, act):
    layer, x, dh = E.a_chain(n, k, f, group, t, act, 5)
    chain = E.Chain(x, dh, layer, act)
    right, dpre, d = plain_gradients(layer, x, dh, act)
    swapped = torch.cat([dpre[:, f:], dpre[:, :f]], 1)
    w = E.weights(*layer)
    mistakes = {
        "x": [swapped @ w, dpre[:, :f] @ w[:f], dpre @ w.roll(8, 1)],
        "step": [(d * P.codes(layer[0]).view(d.shape)).sum(-1), right["step"].roll(1, 0)],
        "zero": [right["zero"] / layer[1].to(P.F64), right["zero"].roll(1, 1)],
    }
    for name, got in right.items():
        assert chain.agrees(name, got), name
        for bad in [0 * got, -got, 1.05 * got, 0.95 * got] + mistakes[name]:
            if not torch.equal(bad, got):
                assert not chain.agrees(name, bad), name


def rnd(n, m, t, seed, scale=1.0):
    """test_w4_ops_gpu.py's inputs, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn(n, m, generator=g)
    x[:, torch.rand(m, generator=g) < 0.02] *= 16
    return x.to(t)


TYPES = (torch.float16, torch.bfloat16)


@pytest.mark.parametrize("n,k,o", E.ROUNDED_PARAM_GRAD, ids=str)
@pytest.mark.parametrize("t", TYPES, ids=str)
def test_rounded_reference_of_param_grad(n, k, o, t):
    """The definition's own value, rounded once to binary32, is out of the named cases' bounds."""
    for group in E.ROUNDED_PARAM_GRAD[n, k, o]:
        layer = P.make_layer(o, k, group, n + k + o, zeros="any")
        dy, x = rnd(n, o, t, n + 5, 0.01), rnd(n, k, t, n + 6)
        want, e, _, _ = P.param_grad(dy, x, *layer)
        d = (dy.to(P.F64).T @ x.to(P.F64)).view(o, k // group, group)
        right = (d * E.differences(layer[0], layer[2]).view(d.shape)).sum(-1).float().to(P.F64)
        assert bool(((right - want).abs() > P.rounded(want, e, torch.float32)).any()), group


@pytest.mark.parametrize("n", E.ROUNDED_LINEAR_ZEROS)
@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("group", E.ALL)
def test_rounded_reference_of_linear_zeros(n, t, group):
    layer = P.make_layer(200, 512, group, 5, zeros="any")
    x = rnd(n, 512, t, 9)
    want, e = P.linear(x, P.weights(*layer))
    right = (x.to(P.F64) @ E.weights(*layer).T).float().to(P.F64)
    assert bool(((right - want).abs() > P.rounded(want, e, torch.float32)).any())
