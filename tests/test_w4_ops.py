"""Packed-weight operators without a GPU: the refusals of the C calls and of
the binding, and the plain binary64 forms against differences and brute force."""
import ctypes

import pytest
import torch

import w4_plain as P
from post_bit_weight_awq_amd import _lib

BAD, UNS, WS = _lib.AWQ_ERR_INVALID_ARG, _lib.AWQ_ERR_UNSUPPORTED, _lib.AWQ_ERR_WORKSPACE
OPS = ("linear", "gated", "input_grad", "gated_backward", "param_grad")
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def ptr(i):
    return ctypes.c_void_p((i + 1) << 44)  # far apart, never dereferenced


def call(lib, op, n=4, k=256, o=32, group=128, dtype=0, act=0, y=None, p=None, size=BIG):
    p = [ptr(i) for i in range(8)] if p is None else p
    q, s, z = p[5], p[6], p[7]
    if op == "linear":
        a = (p[0], dtype, n, k, o, group, q, s, z, p[1], dtype if y is None else y, p[2], size, None)
    elif op == "gated":
        a = (p[0], dtype, n, k, o, group, act, q, s, z, p[1], p[3], p[2], size, None)
    elif op == "input_grad":
        a = (p[0], dtype, n, k, o, group, q, s, z, p[1], p[2], size, None)
    elif op == "gated_backward":
        a = (p[0], p[4], dtype, n, k, o, group, act, q, s, z, p[3], p[1], p[2], size, None)
    else:
        a = (p[0], p[4], dtype, n, k, o, group, q, s, z, p[1], p[3], p[2], size, None)
    return getattr(lib, "awq_w4a16_" + op)(*a)


#: which of the eight pointers each call takes (2 is the workspace)
USED = {"linear": (0, 1, 5, 6, 7), "gated": (0, 1, 5, 6, 7), "input_grad": (0, 1, 5, 6, 7),
        "gated_backward": (0, 1, 3, 4, 5, 6, 7), "param_grad": (0, 1, 3, 4, 5, 6, 7)}


@pytest.mark.parametrize("op", OPS)
def test_refuses_sizes_and_types(lib, op):
    for kw in (dict(n=0), dict(n=-1), dict(n=(1 << 20) + 1), dict(k=0), dict(k=200), dict(k=64),
               dict(k=1 << 21), dict(o=0), dict(o=-3), dict(o=1 << 21), dict(k=1 << 20, o=1 << 19)):
        assert call(lib, op, **kw) == BAD, kw
        assert lib.awq_last_error()
        size = getattr(lib, f"awq_w4a16_{op}_workspace_size")
        d = dict(n=4, k=256, o=32, **{}) | kw
        assert size(d["n"], d["k"], d["o"], 128, 0) == ctypes.c_size_t(-1).value
    for kw in (dict(group=16), dict(group=256), dict(group=0), dict(dtype=2), dict(dtype=-1)):
        assert call(lib, op, **kw) == UNS, kw
        size = getattr(lib, f"awq_w4a16_{op}_workspace_size")
        assert size(4, 256, 32, kw.get("group", 128), kw.get("dtype", 0)) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("op", OPS)
def test_refuses_pointers(lib, op):
    for i in USED[op]:
        for bad in (None, ctypes.c_void_p(((i + 1) << 44) + 8)):
            p = [ptr(j) for j in range(8)]
            p[i] = bad
            assert call(lib, op, p=p) == BAD, i
    # an output inside an input, an output inside another output
    for i, j in ((1, 0), (1, 5), (1, 6), (1, 7)) + (((3, 1), (3, 4)) if 3 in USED[op] else ()):
        p = [ptr(m) for m in range(8)]
        p[i] = ctypes.c_void_p(((j + 1) << 44) + 16)
        assert call(lib, op, p=p) == BAD, (i, j)
        assert b"overlap" in lib.awq_last_error()


def test_refuses_activation_and_output_type(lib):
    for op in ("gated", "gated_backward"):
        assert call(lib, op, act=2) == UNS and call(lib, op, act=-1) == UNS
    assert call(lib, "linear", y=1) == UNS  # fp16 in, bf16 out
    assert call(lib, "linear", dtype=1, y=0) == UNS
    assert call(lib, "linear", y=3) == UNS


@pytest.mark.parametrize("op", OPS)
def test_short_workspace(lib, op):
    size = getattr(lib, f"awq_w4a16_{op}_workspace_size")
    for n, k, o, dtype in ((4, 256, 32, 0), (300, 512, 100, 1), (4096, 5120, 13824, 1), (33, 128, 7, 0)):
        need = size(n, k, o, 128, dtype)
        assert need < 1 << 34
        if need:
            assert call(lib, op, n=n, k=k, o=o, dtype=dtype, size=need - 1) == WS
            p = [ptr(i) for i in range(8)]
            p[2] = None
            assert call(lib, op, n=n, k=k, o=o, dtype=dtype, p=p) == BAD
            p[2] = ctypes.c_void_p((1 << 44) + 16)  # inside the input
            assert call(lib, op, n=n, k=k, o=o, dtype=dtype, p=p) == BAD


def test_binding_refusals():
    import post_bit_weight_awq_amd as awq
    q, s, z = P.make_layer(8, 256, 64, 0)
    x = torch.zeros(2, 256, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        awq.awq_w4a16_linear(x, q, s, z)
    with pytest.raises(TypeError, match="float16 or torch.bfloat16"):
        awq.awq_w4a16_linear(x.float(), q, s, z)
    with pytest.raises(ValueError, match="2-D"):
        awq.awq_w4a16_gated(x[0], q, s, z)
    with pytest.raises(ValueError, match="groups"):
        awq.awq_w4a16_input_grad(x, q, s[:, :3], z)


# ------------------------------------------------ the plain forms themselves
def test_plain_weights_brute_force():
    q, s, z = P.make_layer(3, 128, 32, 1, zeros="any")
    w = P.weights(q, s, z)
    for o in range(3):
        for k in range(128):
            c = (int(q[o, k // 8]) >> (4 * (k % 8))) & 15
            d = float(w[o, k]) / float(s[o, k // 32])
            exact = c - float(z[o, k // 32])
            # 11 bits, or within 2^-15 (two roundings to its multiples)
            assert abs(d - exact) <= max(2.0 ** -11 * abs(exact), 2.0 ** -15)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_plain_gradients_against_differences(name):
    """Central differences of L = sum(C * H) in X, step and zero."""
    g = torch.Generator().manual_seed(3)
    q, s, z = P.make_layer(12, 128, 64, 2, zeros="any")
    d64, s64 = P.codes(q), s.to(P.F64)
    x = torch.randn(5, 128, generator=g, dtype=P.F64)
    c = torch.randn(5, 6, generator=g, dtype=P.F64)

    def loss(x, s, z):
        w = (d64 - z.repeat_interleave(64, 1)) * s.repeat_interleave(64, 1)
        h = x @ w.T
        return float((c * P.act(h[:, :6], name)[0] * h[:, 6:]).sum())

    z64 = z.to(P.F64)
    w = (d64 - z64.repeat_interleave(64, 1)) * s64.repeat_interleave(64, 1)
    pre = x @ w.T
    dpre = P.gated_grad(c, pre, name)[0]
    dx = dpre @ w
    dw = (dpre.T @ x).view(12, 2, 64)
    ds = (dw * (d64.view(12, 2, 64) - z64[..., None])).sum(-1)
    dz = -s64 * dw.sum(-1)
    for got, at, h in ((dx, 0, 1e-5), (ds, 1, 1e-7), (dz, 2, 1e-4)):
        v = torch.randn(got.shape, generator=g, dtype=P.F64)
        args = [x, s64, z64]
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + h * v, args[at] - h * v
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        want = float((got * v).sum())
        assert abs(num - want) <= 1e-5 * float((got * v).abs().sum()), at
