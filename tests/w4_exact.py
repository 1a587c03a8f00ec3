"""Packed-weight operators from their definition in binary64, the zeros unrounded, and the directional check of a
chain of gradients (torch, any device, no library code)."""
import torch

import w4_plain as P


def differences(qweight, zero):
    q = P.codes(qweight)
    return q - P.spread(zero, q.shape[1])


def weights(qweight, step, zero):
    d = differences(qweight, zero)
    return d * P.spread(step, d.shape[1])


class Chain:
    """L(X, step, zero) = sum(dH * act(G) * U) with [G | U] = X W^T, the loss that a gated block's backward pass from
    dH is the gradient of."""

    #: displacement along a unit vector: the loss is smooth over many times that, and binary64 holds its difference to
    #: 1e-8 or better
    H = {"x": 1e-3, "step": 1e-6, "zero": 1e-3}

    def __init__(self, x, dh, layer, act):
        self.args = {"x": x.to(P.F64), "step": layer[1].to(P.F64), "zero": layer[2].to(P.F64)}
        self.q, self.dh, self.act = P.codes(layer[0]), dh.to(P.F64), act

    def loss(self, x, step, zero):
        k = x.shape[1]
        h = x @ ((self.q - P.spread(zero, k)) * P.spread(step, k)).T
        f = self.dh.shape[1]
        return float((self.dh * P.act(h[:, :f], self.act)[0] * h[:, f:]).sum())

    def along(self, name, v):
        """The central difference of the loss along v."""
        h = self.H[name]
        hi, lo = dict(self.args), dict(self.args)
        hi[name], lo[name] = hi[name] + h * v, lo[name] - h * v
        return (self.loss(**hi) - self.loss(**lo)) / (2 * h)

    def agrees(self, name, got):
        """Whether `got` is the gradient in `name`, by central differences along got itself, where a right gradient's
        terms do not cancel and the derivative is its length |got|, and along 24 single coordinates, which also see
        what is missing at right angles to got.  A term of a gradient carries at most five roundings to 16 bits (pre
        moves act' and U, then dpre, the weight, the result): 5 * 2^-8 of itself in bf16.  The terms' errors, of either
        sign, add as the root of their squares, and so do the terms in |got|: a thirtieth of the length holds them,
        and a twentieth off is off; the 24 coordinates are off by a tenth of their own length at most."""
        got = got.to(P.F64)
        size = float(got.norm())
        if not size > 0 or abs(self.along(name, got / size) - size) > size / 30:
            return False
        g = torch.Generator().manual_seed(got.numel())
        off = want = 0.0
        for i in torch.randperm(got.numel(), generator=g)[:24].tolist():
            e = torch.zeros_like(got)
            e.view(-1)[i] = 1
            d = self.along(name, e)
            off, want = off + (d - float(got.view(-1)[i])) ** 2, want + d * d
        return off <= want / 100


def a_chain(n, k, f, group, t, act, seed, dev="cpu"):
    g = torch.Generator().manual_seed(seed)
    layer = P.make_layer(2 * f, k, group, seed, dev, "any")
    x = torch.randn(n, k, generator=g).to(t).to(dev)
    dh = (0.1 * torch.randn(n, f, generator=g)).to(t).to(dev)
    return layer, x, dh


#: Cases of test_w4_ops_gpu.py whose reference value is not the definition's: w4_plain.differences rounds q - zero to
#: 11 bits, which takes a result with fractional zeros further off than the case's own bound (it counts binary32's
#: roundings alone).  An operator that holds zeros whole fails them; test_w4_exact.py shows it for each.
ALL = (128, 64, 32)
ROUNDED_PARAM_GRAD = {(1, 128, 1): (64,), (1, 512, 512): ALL, (1, 1152, 333): ALL, (3, 640, 17): ALL, (5, 384, 96): ALL,
                      (17, 256, 65): ALL, (33, 640, 130): ALL, (65, 128, 257): (64, 32), (129, 1280, 193): (64, 32)}
ROUNDED_LINEAR_ZEROS = (7, 40, 200, 600)


def holds_rounded_zeros(test, p):
    """Whether the case `p` (its parameters) of a test is one of them."""
    if test == "test_linear_zeros":
        return p["zeros"] == "any" and p["n"] in ROUNDED_LINEAR_ZEROS
    return test == "test_param_grad" and p["group"] in ROUNDED_PARAM_GRAD.get((p["n"], p["k"], p["o"]), ())
