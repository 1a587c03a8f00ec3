"""The 4-bit cache without a GPU: refusals of the C calls and of the binding,
and the plain forms against brute force."""
import ctypes
import math

import pytest
import torch

import kv4_plain as K
import post_bit_weight_awq_amd as awq
from post_bit_weight_awq_amd import _lib

BAD, UNS, WS = _lib.AWQ_ERR_INVALID_ARG, _lib.AWQ_ERR_UNSUPPORTED, _lib.AWQ_ERR_WORKSPACE
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def ptr(i):
    return (i + 1) << 44  # far apart, never dereferenced


def cache(pages=8, heads=2, page=16, dim=128, group=64, **kw):
    c = _lib.AwqKv4Cache(ptr(0), ptr(1), ptr(2), ptr(3), pages, heads, page, dim, group)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append(lib, c, n=4, dtype=0, k=None, v=None, slots=None, st=(256, 128, 256, 128)):
    return lib.awq_kv4_append(ctypes.byref(c) if c else None, ptr(4) if k is None else k, ptr(5) if v is None else v, dtype,
                              n, *st, ptr(6) if slots is None else slots, None)


def gather(lib, c, n=4, dtype=0, k=None, v=None, slots=None):
    return lib.awq_kv4_gather(ctypes.byref(c) if c else None, ptr(6) if slots is None else slots, n,
                              ptr(4) if k is None else k, ptr(5) if v is None else v, dtype, None)


def attend(lib, c, n=4, heads=8, seqs=4, pages=4, dtype=0, starts=None, st=(1024, 128), scale=0.1, p=None, size=BIG):
    p = {**dict(q=ptr(4), out=ptr(5), table=ptr(6), lens=ptr(7), ws=ptr(8)), **(p or {})}
    return lib.awq_kv4_attention(ctypes.byref(c) if c else None, p["q"], dtype, n, heads, *st, seqs, starts, p["table"],
                                 pages, p["lens"], scale, p["out"], p["ws"], size, None)


CALLS = (append, gather, attend)


@pytest.mark.parametrize("call", CALLS)
def test_refuses_caches_and_types(lib, call):
    assert call(lib, None) == BAD
    for kw in (dict(page=8), dict(page=48), dict(page=256), dict(page=0), dict(dim=32), dict(dim=256), dict(dim=96),
               dict(group=16), dict(group=0), dict(group=256), dict(dim=64, group=128)):
        assert call(lib, cache(**kw)) == UNS, kw
    for kw in (dict(pages=0), dict(pages=-1), dict(pages=1 << 27), dict(heads=0), dict(heads=1025)):
        assert call(lib, cache(**kw)) == BAD, kw
    for dtype in (2, -1):
        assert call(lib, cache(), dtype=dtype) == UNS
    for n in (0, -1, (1 << 20) + 1):
        assert call(lib, cache(), n=n) == BAD
    for name in ("k_codes", "v_codes", "k_params", "v_params"):
        for bad in (None, ptr(0) + 8):
            assert call(lib, cache(**{name: bad})) == BAD, name


def test_append_and_gather_refuse_pointers_and_strides(lib):
    for call in (append, gather):
        for name in ("k", "v"):
            for bad in (0, ptr(9) + 8):
                assert call(lib, cache(), **{name: bad}) == BAD
        for bad in (0, ptr(9) + 2):
            assert call(lib, cache(), slots=bad) == BAD
        assert call(lib, cache(), k=ptr(0) + 64) == BAD and b"overlap" in lib.awq_last_error()
        assert call(lib, cache(), v=ptr(3) + 64) == BAD
    assert gather(lib, cache(), v=ptr(4) + 64) == BAD  # the two outputs
    for i in range(4):
        for bad in (-8, 4, 129):
            st = [256, 128, 256, 128]
            st[i] = bad
            assert append(lib, cache(), st=st) == BAD


def test_attention_refuses(lib):
    for heads in (0, 7, -8, 2 * 1025, 4097):
        assert attend(lib, cache(), heads=heads) == BAD, heads
    assert attend(lib, cache(), n=1 << 20, seqs=1 << 20, heads=2048) == BAD
    assert attend(lib, cache(), seqs=3) == BAD and b"starts" in lib.awq_last_error()
    for seqs in (0, (1 << 20) + 1):
        assert attend(lib, cache(), seqs=seqs, starts=ptr(9)) == BAD
    for pages in (0, -1, (1 << 26) + 1):
        assert attend(lib, cache(), pages=pages) == BAD
    for scale in (math.nan, math.inf, -math.inf):
        assert attend(lib, cache(), scale=scale) == BAD
    for name in ("q", "out"):
        for bad in (None, ptr(9) + 8):
            assert attend(lib, cache(), p={name: bad}) == BAD
    for name in ("table", "lens"):
        for bad in (None, ptr(9) + 2):
            assert attend(lib, cache(), p={name: bad}) == BAD
    assert attend(lib, cache(), starts=ptr(9) + 1) == BAD
    for st in ((1025, 128), (1024, 4), (-1024, 128)):
        assert attend(lib, cache(), st=st) == BAD
    for name in ("q", "table", "lens"):
        at = {"q": 4, "table": 6, "lens": 7}[name]
        assert attend(lib, cache(), p={"out": ptr(at)}) == BAD and b"overlap" in lib.awq_last_error()
    assert attend(lib, cache(), p={"out": ptr(1) + 16}) == BAD


def test_attention_workspace(lib):
    size = lib.awq_kv4_attention_workspace_size
    c = cache()
    assert size(ctypes.byref(c), 0, 8, 4, 4, 0) == ctypes.c_size_t(-1).value
    assert size(ctypes.byref(c), 4, 8, 3, 4, 0) == ctypes.c_size_t(-1).value
    assert size(ctypes.byref(c), 4, 8, 3, 4, 1) < 1 << 34
    need = size(ctypes.byref(c), 1, 8, 1, 4096, 0)
    assert 0 < need < 1 << 34
    assert attend(lib, c, n=1, seqs=1, pages=4096, size=need - 1) == WS
    assert attend(lib, c, n=1, seqs=1, pages=4096, p={"ws": None}) == BAD
    assert attend(lib, c, n=1, seqs=1, pages=4096, p={"ws": ptr(4)}) == BAD


def test_binding_refusals():
    with pytest.raises(awq.AwqError, match="page_size"):
        awq.awq_kv4_cache(4, 2, 24, 128, device="cpu")
    with pytest.raises(awq.AwqError, match="group_size"):
        awq.awq_kv4_cache(4, 2, 16, 64, 128, device="cpu")
    with pytest.raises(awq.AwqError, match="n_pages"):
        awq.awq_kv4_cache(0, 2, 16, 64, 64, device="cpu")
    c = awq.awq_kv4_cache(4, 2, 32, 128, 32, device="cpu")
    assert (c.n_pages, c.n_heads, c.page_size, c.head_dim, c.group_size) == (4, 2, 32, 128, 32)
    k = torch.zeros(3, 2, 128, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: awq.awq_kv4_append(k, k, c, i), lambda: awq.awq_kv4_gather(c, i),
                 lambda: awq.awq_kv4_attention(k, c, i[:, None], i)):
        with pytest.raises(ValueError, match="GPU"):
            call()


# ---------------------------------------------------------------- plain forms
def test_plain_layout_brute_force():
    for d, group in ((64, 32), (128, 128), (128, 32)):
        g = torch.Generator().manual_seed(d + group)
        ck = torch.randint(0, 16, (2, 3, 32, d), generator=g, dtype=torch.int32)
        cv = torch.randint(0, 16, (2, 3, 32, d), generator=g, dtype=torch.int32)
        pk = torch.randn(2, 3, 32, d // group, 2, generator=g).half()
        pv = torch.randn(2, 3, 32, d // group, 2, generator=g).half()
        cache = K.store(ck, pk, cv, pv)
        k, v = K.read(cache)
        j = d // 32
        for _ in range(200):
            p, h, i, c = (int(torch.randint(0, n, (1,), generator=g)) for n in (2, 3, 32, d))
            b = c // 8
            w = int(cache[0][p, h, i, j * (b % 4) + b // 4]) >> (4 * (c % 8)) & 15
            assert w == int(ck[p, h, i, c])
            assert float(k[p, h, i, c]) == w * float(pk[p, h, i, c // group, 0]) + float(pk[p, h, i, c // group, 1])
            w = int(cache[1][p, h, i // 16, b, i % 16]) >> (4 * (c % 8)) & 15
            assert w == int(cv[p, h, i, c])
            assert float(v[p, h, i, c]) == w * float(pv[p, h, i, c // group, 0]) + float(pv[p, h, i, c // group, 1])


def test_plain_quantize_bounds():
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(50, 128, generator=g) * torch.logspace(-3, 3, 50)[:, None]).half()
    c, p = K.quantize(x, 32)
    step = p[..., 0].to(K.F64).repeat_interleave(32, -1)
    err = (K.value(c, p) - x.to(K.F64)).abs()
    # half a step, and the step's and offset's own roundings
    size = x.to(K.F64).abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
    assert bool((err <= step / 2 + 16 * 2.0 ** -11 * step + 2.0 ** -11 * size + 2.0 ** -24).all())
    c, p = K.quantize(torch.full((1, 64), 3.25).half(), 64)
    assert bool((K.value(c, p) == 3.25).all())
    x = torch.zeros(1, 64)
    x[0, 5] = math.inf
    c, p = K.quantize(x.half(), 32)
    assert bool(K.value(c, p)[0, :32].isnan().all()) and bool((K.value(c, p)[0, 32:] == 0).all())


def test_attention_refuses_scales_that_leave_the_range(lib):
    for scale in (2.0 ** 33, -1e38, 3e38):
        assert attend(lib, cache(), scale=scale) == BAD
