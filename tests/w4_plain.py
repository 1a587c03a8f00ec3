"""Plain binary64 forms of the packed-weight operators and the error bounds
their tests hold the kernels to (torch, any device, no library code)."""
import math

import torch

F64 = torch.float64
U32 = 2.0 ** -24          # half a step of binary32


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half the spacing of the smallest subnormals."""
    f = torch.finfo(t)
    return f.smallest_normal * f.eps / 2


def make_layer(o, k, group, seed, dev="cpu", zeros="packed"):
    """qweight, step, zero with every code value; zeros: integers in 0..15 as
    packing leaves them, "far" integers up to 2000 in magnitude, or "any"
    fp16 values."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (o, k), generator=g, dtype=torch.int32)
    ng = k // group
    step = (0.002 + 0.01 * torch.rand(o, ng, generator=g)).to(torch.float16)
    if zeros == "packed":
        zero = torch.randint(0, 16, (o, ng), generator=g).to(torch.float16)
    elif zeros == "far":
        zero = torch.randint(-2000, 2001, (o, ng), generator=g).to(torch.float16)
    else:
        zero = (8 + 4 * torch.randn(o, ng, generator=g)).to(torch.float16)
    sh = torch.arange(0, 32, 4, dtype=torch.int64)
    words = (q.view(o, k // 8, 8).to(torch.int64) << sh).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    return words.to(dev), step.to(dev), zero.to(dev)


def codes(qweight):
    sh = torch.arange(0, 32, 4, dtype=torch.int32, device=qweight.device)
    return ((qweight[:, :, None] >> sh) & 15).flatten(1).to(F64)


def spread(p, k):
    return p.to(F64).repeat_interleave(k // p.shape[1], 1)


def differences(qweight, zero):
    """q - zero as the operators take it: in fp16 and units of 2^-9, so with 11
    bits or to a multiple of 2^-15, the zero first (where it is below 2^-5)
    and then the difference."""
    q = codes(qweight)
    z = (zero.to(F64) / 512).to(torch.float16).to(F64)
    return (q / 512 - spread(z, q.shape[1])).to(torch.float16).to(F64) * 512


def weights(qweight, step, zero):
    d = differences(qweight, zero)
    return d * spread(step, d.shape[1])


def act(g, name):
    if name == "silu":
        y, dy = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        y, dy = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)
    p = torch.sigmoid(y)
    return g * p, p + g * dy * p * torch.sigmoid(-y)


def linear(x, w):
    """(Y, bound of the binary32 sum): any order of k + 64 additions, each off
    by at most a step (twice half a step: a sum inside the matrix unit may be
    cut rather than rounded)."""
    x = x.to(F64)
    return x @ w.T, 2 * (w.shape[1] + 64) * U32 * (x.abs() @ w.abs().T)


def rounded(y, bound, t):
    """Bound of a value within `bound` of y after rounding once to t."""
    return bound + half_step(t) * (y.abs() + bound) + tiny(t)


def gated(x, w, name):
    """H, pre and their bounds before the last rounding.  |act'| <= 1.13 for
    both gates; the gate's value is off by 16 binary32 half steps of |g| (the
    exponential, a sum, a quotient, products; its argument's own rounding is
    scaled by |y| e^-|y| < 0.37)."""
    f = w.shape[0] // 2
    pre, e = linear(x, w)
    g, u, eg, eu = pre[:, :f], pre[:, f:], e[:, :f], e[:, f:]
    a = act(g, name)[0]
    ea = 1.13 * eg + 16 * U32 * g.abs()
    return a * u, (a.abs() + ea) * eu + ea * u.abs() + 2 * U32 * (a * u).abs(), pre, e


def input_grad(dy, w, t):
    """dX and its bound: the sum's and each weight's rounding to fp16."""
    dy = dy.to(F64)
    y, s = dy @ w, dy.abs() @ w.abs()
    b = (2 * (w.shape[0] + 64) * U32 + half_step(torch.float16)) * s
    return y, b + tiny(torch.float16) * dy.abs().sum(1, keepdim=True)


def gated_grad(dh, pre, name):
    """dpre and its bound before rounding: 32 half steps of each product of
    magnitudes (|slope| is at most |p| + |g y' p q|, whose terms may cancel)."""
    f = dh.shape[1]
    dh, g, u = dh.to(F64), pre[:, :f].to(F64), pre[:, f:].to(F64)
    a, s = act(g, name)
    e = 32 * U32 * torch.cat([(dh * u).abs() * (1 + g.abs()), (dh * g).abs()], 1)
    return torch.cat([dh * u * s, dh * a], 1), e


def param_grad(dy, x, qweight, step, zero):
    dy, x = dy.to(F64), x.to(F64)
    o, ng = step.shape
    d, da = (dy.T @ x).view(o, ng, -1), (dy.abs().T @ x.abs()).view(o, ng, -1)
    q = differences(qweight, zero).view(d.shape)
    n = 2 * (dy.shape[0] + d.shape[2] + 64) * U32
    s = step.to(F64)
    return (d * q).sum(-1), n * (da * q.abs()).sum(-1), -s * d.sum(-1), n * s * da.sum(-1)
