"""Adapters beside a packed product without a GPU: refusals of the C calls and
of the binding, and the plain form's gradients against differences."""
import ctypes

import pytest
import torch

import w4_adapt_plain as AP
import w4_plain as P
from post_bit_weight_awq_amd import _lib

BAD, UNS, WS = _lib.AWQ_ERR_INVALID_ARG, _lib.AWQ_ERR_UNSUPPORTED, _lib.AWQ_ERR_WORKSPACE
BIG = 1 << 44
NAMES = ("x", "y", "low", "q", "s", "z", "a", "b", "scale", "ids", "ws", "dy", "da", "db")
USED = {"adapted": ("x", "y", "q", "s", "z", "a", "b", "scale", "ids"),
        "adapted_backward": ("dy", "x", "low", "q", "s", "z", "a", "b", "scale", "ids", "y", "da", "db")}
OPS = tuple(USED)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def ptr(name):
    return (NAMES.index(name) + 1) << 46  # far apart, never dereferenced


def call(lib, op, n=4, k=256, o=32, group=128, dtype=0, y=None, count=3, rank=16, p=None, size=BIG):
    p = {**{i: ptr(i) for i in NAMES}, **(p or {})}
    layer = (p["q"], p["s"], p["z"], p["a"], p["b"], p["scale"], count, rank, p["ids"])
    if op == "adapted":
        return lib.awq_w4a16_adapted(p["x"], dtype, n, k, o, group, *layer, p["y"], dtype if y is None else y, p["low"],
                                     p["ws"], size, None)
    return lib.awq_w4a16_adapted_backward(p["dy"], p["x"], p["low"], dtype, n, k, o, group, *layer, p["y"], p["da"],
                                          p["db"], p["ws"], size, None)


def need(lib, op, n=4, k=256, o=32, group=128, dtype=0, y=None, count=3, rank=16, keep=0):
    if op == "adapted":
        return lib.awq_w4a16_adapted_workspace_size(n, k, o, group, dtype, dtype if y is None else y, count, rank, keep)
    return lib.awq_w4a16_adapted_backward_workspace_size(n, k, o, group, dtype, count, rank)


@pytest.mark.parametrize("op", OPS)
def test_refuses_sizes_and_types(lib, op):
    for kw in (dict(n=0), dict(n=(1 << 20) + 1), dict(k=0), dict(k=200), dict(k=1 << 21), dict(o=0), dict(o=1 << 21),
               dict(k=1 << 20, o=1 << 19), dict(count=0), dict(count=-2), dict(count=32769),
               dict(count=32768, rank=128, k=8192), dict(count=32768, rank=128, o=8192)):
        assert call(lib, op, **kw) == BAD, kw
        assert need(lib, op, **kw) == ctypes.c_size_t(-1).value and lib.awq_last_error()
    for kw in (dict(group=16), dict(dtype=2), dict(dtype=-1), dict(rank=0), dict(rank=4), dict(rank=12), dict(rank=136)):
        assert call(lib, op, **kw) == UNS, kw
        assert need(lib, op, **kw) == ctypes.c_size_t(-1).value
    if op == "adapted":
        for kw in (dict(y=1), dict(y=3), dict(dtype=1, y=0)):
            assert call(lib, op, **kw) == UNS and need(lib, op, **kw) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("op", OPS)
def test_refuses_pointers(lib, op):
    for i in USED[op]:
        for bad in (None, ptr(i) + (2 if i in ("scale", "ids") else 8)):
            assert call(lib, op, p={i: bad}) == BAD, i
    written = ("y", "low") if op == "adapted" else ("y", "da", "db")
    assert need(lib, op, n=300, keep=1) > 0
    for i in written + ("ws",):
        for j in USED[op]:
            if i != j:
                assert call(lib, op, n=300, p={i: ptr(j)}) == BAD, (i, j)
                assert b"overlap" in lib.awq_last_error()


@pytest.mark.parametrize("op", OPS)
def test_short_workspace(lib, op):
    for n, k, o, dtype, rank in ((1, 256, 32, 0, 8), (4, 5120, 640, 1, 64), (300, 512, 100, 1, 24), (4096, 5120, 13824, 1, 128)):
        kw = dict(n=n, k=k, o=o, dtype=dtype, rank=rank)
        size = need(lib, op, **kw, keep=1)
        assert size < 1 << 34
        if size:
            assert call(lib, op, **kw, size=size - 1) == WS
            assert call(lib, op, **kw, p={"ws": None}) == BAD


def test_binding_refusals():
    import post_bit_weight_awq_amd as awq
    layer = P.make_layer(8, 256, 64, 0)
    x = torch.zeros(2, 256, dtype=torch.float16)
    a, b = torch.zeros(3, 16, 256, dtype=torch.float16), torch.zeros(3, 8, 16, dtype=torch.float16)
    sc, ids = torch.ones(3), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        awq.awq_w4a16_adapted(x, *layer, a, b, sc, ids)
    with pytest.raises(ValueError, match="GPU"):
        awq.awq_w4a16_adapted_backward(x[:, :8], x, torch.zeros(2, 16), *layer, a, b, sc, ids)
    with pytest.raises(RuntimeError, match="requires a gradient"):
        awq.awq_w4a16_adapted(x.requires_grad_(), *layer, a, b, sc, ids)


def test_plain_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    layer = P.make_layer(12, 128, 64, 2, zeros="any")
    w = P.codes(layer[0]) - layer[2].to(P.F64).repeat_interleave(64, 1)
    w = w * layer[1].to(P.F64).repeat_interleave(64, 1)
    x, dy = (torch.randn(5, n, generator=g, dtype=P.F64) for n in (128, 12))
    a, b = torch.randn(3, 8, 128, generator=g, dtype=P.F64), torch.randn(3, 12, 8, generator=g, dtype=P.F64)
    sc, ids = torch.tensor([0.5, 2.0, 1.0], dtype=P.F64), torch.tensor([1, 0, -1, 1, 7])

    def loss(x, a, b):
        return float((AP.forward(x, w, a, b, sc, ids)[0] * dy).sum())

    low = AP.forward(x, w, a, b, sc, ids)[1]
    grads = AP.backward(dy, x, low, w, a, b, sc, ids)
    assert bool((grads[1][2] == 0).all()) and bool((grads[2][2] == 0).all())
    args = [x, a, b]
    for i, got in enumerate(grads):
        v = torch.randn(got.shape, generator=g, dtype=P.F64)
        hi, lo = list(args), list(args)
        h = 1e-5
        hi[i], lo[i] = args[i] + h * v, args[i] - h * v
        assert abs((loss(*hi) - loss(*lo)) / (2 * h) - float((got * v).sum())) <= 1e-5 * float((got * v).abs().sum())
