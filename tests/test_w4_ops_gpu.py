"""Packed-weight operators on the GPU against their plain binary64 forms."""
import sys

import pytest

torch = pytest.importorskip("torch")

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


def rnd(n, m, t, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn(n, m, generator=g)
    x[:, torch.rand(m, generator=g) < 0.02] *= 16
    return x.to(t).cuda()


def close(got, want, bound, what):
    got, bad = got.to(P.F64), None
    off = (got - want).abs()
    ok = (off <= bound) | (got == want)
    if not bool(ok.all()):
        bad = (off / bound.clamp_min(1e-300))[~ok].max()
        at = (~ok).nonzero()[0].tolist()
        pytest.fail(f"{what}: {int((~ok).sum())} of {ok.numel()} off, worst {float(bad):.3g} bounds, "
                    f"first at {at}: {float(got[tuple(at)])} for {float(want[tuple(at)])}")


class Guarded:
    """An output inside a larger buffer whose other values must not change."""

    def __init__(self, shape, t):
        n = 1
        for s in shape:
            n *= s
        self.buf = torch.full((n + 512,), 7.0, dtype=t, device="cuda")
        self.t = self.buf[256:256 + n].view(shape)
        self.t.fill_(float("nan"))

    def check(self):
        torch.cuda.synchronize()
        assert bool((self.buf[:256] == 7).all()) and bool((self.buf[-256:] == 7).all()), "guard"
        return self.t


def poisoned(awq, op, n, k, o, group, t):
    """A workspace of exactly the stated size, full of NaN bytes."""
    size = getattr(awq.load(), f"awq_w4a16_{op}_workspace_size")(n, k, o, group, 0 if t == F16 else 1)
    return torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")


# tokens from 1 to past every tile, one output row, odd widths, one group's
# width to many; a last tile of one row and one column
SHAPES = [(1, 128, 1), (1, 512, 512), (1, 1152, 333), (2, 256, 48), (3, 640, 17), (4, 4096, 129), (5, 384, 96),
          (8, 512, 1000), (16, 1024, 250), (17, 256, 65), (33, 640, 130), (64, 896, 512), (65, 128, 257),
          (100, 2048, 96), (128, 512, 384), (129, 1280, 193), (257, 384, 514), (300, 1024, 768),
          (513, 256, 1032)]
TYPES = [(F16, 128), (F16, 64), (F16, 32), (BF16, 128), (BF16, 64), (BF16, 32)]
IDS = [f"{str(t)[6:]}-g{g}" for t, g in TYPES]
by_type = pytest.mark.parametrize("t,group", TYPES, ids=IDS)
by_shape = pytest.mark.parametrize("n,k,o", SHAPES)


def check_linear(awq, x, layer, y_dtype, what, name="linear"):
    n, k = x.shape
    o, group = layer[0].shape[0], k // layer[1].shape[1]
    out = Guarded((n, o), y_dtype)
    awq.awq_w4a16_linear(x, *layer, out=out.t, workspace=poisoned(awq, "linear", n, k, o, group, x.dtype))
    want, e = P.linear(x, P.weights(*layer))
    close(out.check(), want, P.rounded(want, e, y_dtype), what)


@by_shape
@by_type
def test_linear(awq, n, k, o, t, group):
    _say(f"linear {n}x{k}->{o} {t} g{group}")
    layer = P.make_layer(o, k, group, n + k + o, "cuda")
    x = rnd(n, k, t, n)
    for y in (t, F32):
        check_linear(awq, x, layer, y, f"Y {y}")


@pytest.mark.parametrize("n", [1, 7, 40, 200, 600])
@pytest.mark.parametrize("zeros", ["far", "any"])
@by_type
def test_linear_zeros(awq, n, t, group, zeros):
    """Zero points far outside 0..15 and fractional ones."""
    _say(f"linear zeros {zeros} {n} {t} g{group}")
    layer = P.make_layer(200, 512, group, 5, "cuda", zeros)
    check_linear(awq, rnd(n, 512, t, 9), layer, F32, zeros)


def check_gated(awq, n, k, f, t, group, act):
    layer = P.make_layer(2 * f, k, group, n + k + f, "cuda")
    x = rnd(n, k, t, n + 1)
    h, pre = Guarded((n, f), t), Guarded((n, 2 * f), t)
    ws = poisoned(awq, "gated", n, k, f, group, t)
    awq.awq_w4a16_gated(x, *layer, act=act, out=h.t, pre=pre.t, workspace=ws)
    want, e, wpre, epre = P.gated(x, P.weights(*layer), act)
    close(h.check(), want, P.rounded(want, e, t), "H")
    close(pre.check(), wpre, P.rounded(wpre, epre, t), "pre")
    alone = awq.awq_w4a16_gated(x, *layer, act=act)
    torch.cuda.synchronize()
    assert torch.equal(alone.view(torch.int16), h.t.view(torch.int16)), "H with and without pre"


def odd_shapes():
    """Sums of an odd number of 64- and 128-wide steps, whose last one has no
    partner, in tiles of every height, whole and split; then any shapes."""
    g = torch.Generator().manual_seed(31)
    draw = lambda lo, hi: int(torch.randint(lo, hi, (), generator=g))
    return ([(70, 512, 320), (100, 256, 192), (128, 640, 64), (128, 128, 64), (120, 1152, 1600), (66, 2176, 832),
             (129, 384, 320), (250, 1408, 448), (90, 4224, 4160), (400, 896, 960)] +
            [(draw(65, 700), 128 * draw(1, 20), draw(1, 900)) for _ in range(8)])


@pytest.mark.parametrize("n,k,o", odd_shapes())
@by_type
def test_odd_numbers_of_steps(awq, n, k, o, t, group):
    """The product, both forms' gradient for the input and the gated form."""
    _say(f"odd steps {n}x{k},{o} {t} g{group}")
    check_linear(awq, rnd(n, k, t, n), P.make_layer(o, k, group, n + k + o, "cuda"), t, "Y")
    test_input_grad(awq, n, k, o, t, group)
    half = (o + 1) // 2
    check_gated(awq, n, k, half, t, group, "silu")
    test_gated_backward(awq, n, k, half, t, group)


@by_shape
@by_type
def test_gated(awq, n, k, o, t, group):
    act = "silu" if (n + o) % 2 else "gelu"
    _say(f"gated {n}x{k}->{o} {t} g{group} {act}")
    check_gated(awq, n, k, o, t, group, act)


@by_shape
@by_type
def test_input_grad(awq, n, k, o, t, group):
    _say(f"input_grad {n}x{k}<-{o} {t} g{group}")
    layer = P.make_layer(o, k, group, n + k + o, "cuda")
    dy = rnd(n, o, t, n + 2, 0.01)
    out = Guarded((n, k), t)
    awq.awq_w4a16_input_grad(dy, *layer, out=out.t, workspace=poisoned(awq, "input_grad", n, k, o, group, t))
    want, e = P.input_grad(dy, P.weights(*layer), t)
    close(out.check(), want, P.rounded(want, e, t), "dX")


@by_shape
@by_type
def test_gated_backward(awq, n, k, o, t, group):
    act = "gelu" if (n + o) % 2 else "silu"
    _say(f"gated_backward {n}x{k}<-{o} {t} g{group} {act}")
    layer = P.make_layer(2 * o, k, group, n + k + o, "cuda")
    dh, pre = rnd(n, o, t, n + 3, 0.05), rnd(n, 2 * o, t, n + 4, 2.0)
    dx, dpre = Guarded((n, k), t), Guarded((n, 2 * o), t)
    ws = poisoned(awq, "gated_backward", n, k, o, group, t)
    awq.awq_w4a16_gated_backward(dh, pre, *layer, act=act, out=dx.t, dpre=dpre.t, workspace=ws)
    want, e = P.gated_grad(dh, pre, act)
    close(dpre.check(), want, P.rounded(want, e, t), "dpre")
    # dX is defined from dpre as stored
    want, e = P.input_grad(dpre.t, P.weights(*layer), t)
    close(dx.check(), want, P.rounded(want, e, t), "dX")


@by_shape
@by_type
def test_param_grad(awq, n, k, o, t, group):
    _say(f"param_grad {n}x{k},{o} {t} g{group}")
    layer = P.make_layer(o, k, group, n + k + o, "cuda", "any" if n % 2 else "packed")
    dy, x = rnd(n, o, t, n + 5, 0.01), rnd(n, k, t, n + 6)
    ds, dz = Guarded((o, k // group), F32), Guarded((o, k // group), F32)
    ws = poisoned(awq, "param_grad", n, k, o, group, t)
    awq.awq_w4a16_param_grad(dy, x, *layer, dstep=ds.t, dzero=dz.t, workspace=ws)
    ws_, es, wz, ez = P.param_grad(dy, x, *layer)
    close(ds.check(), ws_, P.rounded(ws_, es, F32), "dstep")
    close(dz.check(), wz, P.rounded(wz, ez, F32), "dzero")


# ----------------------------------------------------------- values at the ends
@pytest.mark.parametrize("n", [1, 3, 20, 150, 520])
@by_type
def test_rows_of_any_magnitude(awq, n, t, group):
    """Each token's row has its own scale, from the type's smallest to its
    largest values, rows of zeros among them; a row's result goes by that row
    alone."""
    _say(f"magnitudes {n} {t} g{group}")
    k, o = 256, 136
    layer = P.make_layer(o, k, group, 4, "cuda")
    x = rnd(n, k, F32, 11)
    lo, hi = (-20, 2) if t == F16 else (-110, 100)
    e = torch.linspace(lo, hi, n, dtype=torch.float64, device="cuda").round()
    x = (x * torch.exp2(e)[:, None]).to(t)
    x[n // 2] = 0
    check_linear(awq, x, layer, F32, "rows")
    dy = x[:, :o].contiguous()
    got = awq.awq_w4a16_input_grad(dy, *layer)
    want, e = P.input_grad(dy, P.weights(*layer), t)
    close(got, want, P.rounded(want, e, t), "dX rows")


@pytest.mark.parametrize("n", [1, 4, 30, 300])
@by_type
def test_non_finite_tokens_stay_in_their_rows(awq, n, t, group):
    _say(f"non-finite {n} {t} g{group}")
    k, o = 384, 200
    layer = P.make_layer(o, k, group, 6, "cuda")
    w = P.weights(*layer)
    x = rnd(n, k, t, 12)
    clean = awq.awq_w4a16_linear(x, *layer, out_dtype=F32)
    dirty = x.clone()
    rows = sorted({0, n // 2, n - 1})
    for i, r in enumerate(rows):
        dirty[r, 5 + 40 * i] = (float("nan"), float("inf"), float("-inf"))[i]
    got = awq.awq_w4a16_linear(dirty, *layer, out_dtype=F32)
    want = dirty.to(P.F64) @ w.T
    keep = [r for r in range(n) if r not in rows]
    assert torch.equal(got[keep], clean[keep])
    for r in rows:
        assert torch.equal(got[r].isnan(), want[r].isnan()) and torch.equal(got[r].isinf(), want[r].isinf())
        inf = want[r].isinf()
        assert torch.equal(got[r][inf].to(P.F64), want[r][inf])
    # the same through the gradient for the input
    dy = rnd(n, o, t, 13)
    clean = awq.awq_w4a16_input_grad(dy, *layer)
    dirty = dy.clone()
    for i, r in enumerate(rows):
        dirty[r, 3 + 30 * i] = (float("nan"), float("inf"), float("-inf"))[i]
    got = awq.awq_w4a16_input_grad(dirty, *layer)
    want = dirty.to(P.F64) @ w
    assert torch.equal(got[keep], clean[keep])
    for r in rows:
        assert torch.equal(got[r].isnan(), want[r].isnan())
        inf = want[r].isinf()
        assert torch.equal(got[r][inf].to(P.F64), want[r][inf])


@pytest.mark.parametrize("n", [1, 4, 30, 64, 300])
@pytest.mark.parametrize("far", [False, True])
@by_type
def test_infinities_meet_any_zero(awq, n, far, t, group):
    """Fractional zeros, or large ones that bf16 does not hold, beside rows of
    integers: an infinity times a weight of either kind is an infinity, times 0
    a NaN."""
    _say(f"infinities {n} far={far} {t} g{group}")
    k, o = 256, 100
    q, s, z = P.make_layer(o, k, group, 16, "cuda", "far" if far else "any")
    z[::3] = z[::3].round().clamp(0, 15)
    x = rnd(n, k, t, 17)
    x[0, 7], x[n // 2, 130], x[n - 1, 255] = float("inf"), float("-inf"), float("inf")
    want = x.to(P.F64) @ P.weights(q, s, z).T
    got = awq.awq_w4a16_linear(x, q, s, z, out_dtype=F32).to(P.F64)
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t", [F16, BF16])
def test_gate_extremes(awq, t, act):
    """Gates far from zero: the value saturates to g or 0, the slope to 1 or 0."""
    g = torch.tensor([0.0, -0.0, 1e-4, -1e-4, 5, -5, 12, -12, 40, -40, 88, -88, 104, -104, 300, -300, 6e4, -6e4],
                     device="cuda").to(t)
    f = g.numel()
    pre = torch.stack([torch.cat([g, torch.full_like(g, u)]) for u in (1.0, -3.0)])
    dh = torch.full((2, f), 0.5, dtype=t, device="cuda")
    layer = P.make_layer(2 * f, 128, 128, 7, "cuda")
    dx, dpre = awq.awq_w4a16_gated_backward(dh, pre, *layer, act=act)
    want, e = P.gated_grad(dh, pre, act)
    close(dpre, want, P.rounded(want, e, t), "dpre")
    want, e = P.input_grad(dpre, P.weights(*layer), t)
    close(dx, want, P.rounded(want, e, t), "dX")


# ------------------------------------------------------------ how calls are made
def a_run(awq, n=70, k=512, f=150, t=BF16, group=64, seed=0):
    """Forward with pre kept, backward, parameter gradients, and the next layer."""
    up = P.make_layer(2 * f, k, group, seed, "cuda")
    x, dh = rnd(n, k, t, seed + 1), rnd(n, f, t, seed + 2, 0.1)

    def go(stream=None):
        kw = {"stream": stream}
        h, pre = awq.awq_w4a16_gated(x, *up, keep_pre=True, **kw)
        dx, dpre = awq.awq_w4a16_gated_backward(dh, pre, *up, **kw)
        ds, dz = awq.awq_w4a16_param_grad(dpre, x, *up, **kw)
        y = awq.awq_w4a16_linear(x, *up, out_dtype=F32, **kw)
        back = awq.awq_w4a16_input_grad(dpre, *up, **kw)
        return [h, pre, dx, dpre, ds, dz, y, back]

    return go, (up, x, dh)


def same(a, b):
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


RUNS = [dict(n=1), dict(n=12, f=97), dict(n=70), dict(n=300, t=F16, group=128, f=260), dict(n=700, group=32, f=131)]


@pytest.mark.parametrize("kw", RUNS, ids=str)
def test_run_is_deterministic_and_on_the_given_stream(awq, kw):
    _say("run", kw)
    go, _ = a_run(awq, **kw)
    first = go()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = go(s1), go(s2)  # both at once
    torch.cuda.synchronize()
    same(first, a)
    same(first, b)


@pytest.mark.parametrize("kw", RUNS, ids=str)
def test_run_in_a_graph(awq, kw):
    """Captured once, replayed with other inputs and eager work between."""
    _say("graph", kw)
    go, (up, x, dh) = a_run(awq, **kw)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
    for i in range(3):
        x.copy_(rnd(*x.shape, x.dtype, 100 + i))
        dh.copy_(rnd(*dh.shape, dh.dtype, 200 + i, 0.1))
        eager = go()
        graph.replay()
        torch.cuda.synchronize()
        same(eager, out)


def test_run_gradients_against_differences(awq):
    """dstep, dzero and dX of the run against central differences of the
    binary64 loss sum(dH * H), in a random direction of each."""
    n, k, f, group = 40, 256, 48, 64
    go, (up, x, dh) = a_run(awq, n=n, k=k, f=f, t=F16, group=group, seed=3)
    _, _, dx, _, ds, dz, _, _ = go()
    q, step, zero = P.codes(up[0]), up[1].to(P.F64), up[2].to(P.F64)

    def loss(x, s, z):
        w = (q - P.spread(z, k)) * P.spread(s, k)
        h = x @ w.T
        return float((dh.to(P.F64) * P.act(h[:, :f], "silu")[0] * h[:, f:]).sum())

    g = torch.Generator().manual_seed(5)
    for got, at, h in ((dx, 0, 1e-4), (ds, 1, 1e-6), (dz, 2, 1e-3)):
        v = torch.randn(got.shape, generator=g, dtype=P.F64).cuda()
        args = [x.to(P.F64), step, zero]
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + h * v, args[at] - h * v
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        # pre, dpre, the weights and dX round to fp16, each by 2^-11 of a term;
        # a rounded pre moves dpre by at most about three times that
        terms = (P.param_grad(go()[3].abs(), x.abs(), *up)[1] / (2 * (n + group + 64) * P.U32) if at == 1 else None)
        if at == 0:
            size = (go()[3].to(P.F64).abs() @ P.weights(*up).abs() * v.abs()).sum()
        elif at == 1:
            size = (terms * v.abs()).sum()
        else:
            size = ((go()[3].to(P.F64).abs().T @ x.to(P.F64).abs()).view(2 * f, k // group, group).sum(-1) * step * v.abs()).sum()
        assert abs(num - float((got.to(P.F64) * v).sum())) <= 8 * 2.0 ** -11 * float(size), at


@pytest.mark.parametrize("group", [32, 64, 128])
def test_search_pack_serve(awq, group):
    """A searched and packed layer served by the new product: the same values
    as the packed product that takes groups of 128, and the plain form."""
    import synth
    _, X, W = synth.make_custom(64, 512, 320, seed=8)
    Xd, Wd = torch.from_numpy(X).cuda(), torch.from_numpy(W).cuda()
    cfg = awq.default_config(group_size=group)
    res = awq.awq_search_layer(Xd, Wd, awq.awq_act_stats(Xd), cfg)
    layer = awq.awq_pack(Wd, res.s_best, cfg)
    for n in (1, 5, 64):
        x = (Xd[:n].float() / res.s_best).half()
        check_linear(awq, x, layer, F32, "served")
        check_linear(awq, x, layer, F16, "served")
        if group == 128:
            old, new = awq.awq_w4a16_matmul(x, *layer), awq.awq_w4a16_linear(x, *layer, out_dtype=F32)
            e = P.linear(x, P.weights(*layer))[1]
            # the older product subtracts the zero after the sums, whose terms
            # are up to 15 + |z| against |q - z|
            big = 2 * (512 + 64) * P.U32 * (x.to(P.F64).abs() @ ((15 + P.spread(layer[2], 512).abs()) * P.spread(layer[1], 512)).T)
            close(old, new.to(P.F64), e + big, "both products")


def test_binding_refusals_on_device(awq):
    q, s, z = P.make_layer(8, 256, 64, 0, "cuda")
    x = torch.zeros(2, 256, dtype=F16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        awq.awq_w4a16_linear(torch.zeros(256, 2, dtype=F16, device="cuda").T, q, s, z)
    with pytest.raises(ValueError, match="shape"):
        awq.awq_w4a16_linear(x[:, :128].contiguous(), q, s, z)
    with pytest.raises(TypeError, match="out_dtype"):
        awq.awq_w4a16_linear(x, q, s, z, out_dtype=BF16)
    with pytest.raises(ValueError, match="as many up rows"):
        awq.awq_w4a16_gated(x, *P.make_layer(7, 256, 64, 0, "cuda"))
    with pytest.raises(ValueError, match="act"):
        awq.awq_w4a16_gated(x, q, s, z, act="relu")
    with pytest.raises(ValueError, match="one device|GPU"):
        awq.awq_w4a16_linear(x, q, s.cpu(), z)
    with pytest.raises(awq.AwqError, match="n_tokens"):
        awq.awq_w4a16_linear(x[:0], q, s, z)
    with pytest.raises(awq.AwqError, match="group_size"):
        awq.awq_w4a16_linear(x, q, s[:, :1].contiguous(), z[:, :1].contiguous())
    with pytest.raises(awq.AwqError, match="overlap"):
        buf = torch.zeros(2, 256, dtype=F16, device="cuda")
        awq.awq_w4a16_linear(buf, q, s, z, out=buf.view(-1)[8:24].view(2, 8))
    with pytest.raises(awq.AwqError, match="aligned"):
        off = torch.zeros(2 * 256 + 1, dtype=F16, device="cuda")[1:].view(2, 256)
        awq.awq_w4a16_linear(off, q, s, z)


@pytest.mark.parametrize("n", [1, 40, 130, 520])
@by_type
def test_steps_of_any_size(awq, n, t, group):
    """Steps of 0, subnormal, negative and 128 to 300 beside ordinary ones; a
    row whose first, last or only groups have none."""
    _say(f"steps {n} {t} g{group}")
    k, o = 512, 72
    q, s, z = P.make_layer(o, k, group, 21, "cuda")
    s[0] = 0
    s[1, 0] = 0
    s[2, -1] = 0
    s[3, ::2] = 0
    s[4] = 2.0 ** -24
    s[5, 0] = 2.0 ** -24
    s[6] = -s[6]
    s[7, -1] = 300.0
    s[8] = 128.0
    s[9, 0], s[9, 1] = 2.0 ** -24, 200.0
    layer = (q, s, z)
    x = rnd(n, k, t, 22, 0.25)
    check_linear(awq, x, layer, F32, "Y")
    w = P.weights(*layer)
    y, e = P.linear(x, w)
    assert bool((awq.awq_w4a16_linear(x, *layer, out_dtype=F32)[:, 0] == 0).all())
    dy = rnd(n, o, t, 23, 0.01)
    got = awq.awq_w4a16_input_grad(dy, *layer)
    want, e = P.input_grad(dy, w, t)
    close(got, want, P.rounded(want, e, t), "dX")
    ds, dz = awq.awq_w4a16_param_grad(dy, x, *layer)
    ws_, es, wz, ez = P.param_grad(dy, x, *layer)
    close(ds, ws_, P.rounded(ws_, es, F32), "dstep")
    close(dz, wz, P.rounded(wz, ez.abs(), F32), "dzero")


# shapes that take each way through the kernels: the streaming kernel with two,
# four and eight groups of wavefronts at every token count, tiles of every
# height, whole tiles followed by split ones, rows whose parameters do not fit
# the streaming kernel
WAYS = [(1, 256, 24700), (4, 128, 14400), (5, 128, 14400), (16, 128, 14337), (17, 128, 24600), (32, 256, 24577),
        (33, 128, 25000), (48, 128, 24576), (49, 128, 20500), (64, 256, 20481), (20, 256, 4096), (47, 384, 200),
        (49, 640, 4099), (64, 4096, 512), (10, 17408, 40), (80, 1024, 4096), (190, 2048, 2100), (700, 512, 5000),
        (2100, 512, 8200)]


@pytest.mark.parametrize("t,group", [(F16, 128), (F16, 64), (BF16, 128), (BF16, 32)], ids=str)
@pytest.mark.parametrize("n,k,o", WAYS)
def test_products_every_way(awq, n, k, o, t, group):
    _say(f"ways {n}x{k}->{o} {t} g{group}")
    layer = P.make_layer(o, k, group, n + k + o, "cuda")
    check_linear(awq, rnd(n, k, t, n), layer, t if n % 2 else F32, "Y")
    check_gated(awq, n, k, o // 2, t, group, "silu" if n % 2 else "gelu")


GRAD_WAYS = [(40, 2048, 4100), (100, 4096, 640), (300, 4096, 1000), (700, 1024, 3000), (2100, 8192, 256),
             (513, 128, 9000), (33, 4480, 4400), (300, 4480, 4400)]


@pytest.mark.parametrize("t,group", [(F16, 128), (F16, 32), (BF16, 64)], ids=str)
@pytest.mark.parametrize("n,k,o", GRAD_WAYS)
def test_gradients_every_way(awq, n, k, o, t, group):
    _say(f"gradient ways {n}x{k}<-{o} {t} g{group}")
    layer = P.make_layer(o, k, group, n + k + o, "cuda")
    w = P.weights(*layer)
    dy, x = rnd(n, o, t, n + 2, 0.01), rnd(n, k, t, n + 3)
    out = Guarded((n, k), t)
    awq.awq_w4a16_input_grad(dy, *layer, out=out.t, workspace=poisoned(awq, "input_grad", n, k, o, group, t))
    want, e = P.input_grad(dy, w, t)
    close(out.check(), want, P.rounded(want, e, t), "dX")
    ds, dz = Guarded((o, k // group), F32), Guarded((o, k // group), F32)
    awq.awq_w4a16_param_grad(dy, x, *layer, dstep=ds.t, dzero=dz.t,
                             workspace=poisoned(awq, "param_grad", n, k, o, group, t))
    ws_, es, wz, ez = P.param_grad(dy, x, *layer)
    close(ds.check(), ws_, P.rounded(ws_, es, F32), "dstep")
    close(dz.check(), wz, P.rounded(wz, ez, F32), "dzero")


# ------------------------------------------------- arrays past 2^31 elements
MANY = 1 << 20


def on_gpu(n, m, t, seed, whole=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if whole:
        return torch.randint(-1, 2, (n, m), generator=g, device="cuda", dtype=torch.int8).to(t)
    return torch.randn(n, m, generator=g, device="cuda", dtype=F32).to(t)


def some_rows():
    """The ends, and both sides of element 2^31 of 2304 columns."""
    at = (1 << 31) // 2304
    return torch.tensor([*range(4), *range(at - 3, at + 4), *range(MANY - 70, MANY)], device="cuda")


@pytest.mark.parametrize("t,group", [(F16, 128), (BF16, 32)], ids=str)
def test_products_past_2_31_elements(awq, t, group):
    _say(f"many rows {t} g{group}")
    rows = some_rows()
    x = on_gpu(MANY, 128, t, 1)
    layer = P.make_layer(2304, 128, group, 2, "cuda")
    y = awq.awq_w4a16_linear(x, *layer)
    w = P.weights(*layer)
    want, e = P.linear(x[rows], w)
    close(y[rows], want, P.rounded(want, e, t), "Y")
    del y
    h, pre = awq.awq_w4a16_gated(x, *layer, keep_pre=True)
    want, e, wpre, epre = P.gated(x[rows], w, "silu")
    close(h[rows], want, P.rounded(want, e, t), "H")
    close(pre[rows], wpre, P.rounded(wpre, epre, t), "pre")
    dx, dpre = awq.awq_w4a16_gated_backward(h, pre, *layer)
    want, e = P.gated_grad(h[rows], pre[rows], "silu")
    close(dpre[rows], want, P.rounded(want, e, t), "dpre")
    want, e = P.input_grad(dpre[rows], w, t)
    close(dx[rows], want, P.rounded(want, e, t), "dX from many rows")
    del pre, dpre, h, dx
    wide = P.make_layer(65, 2304, group, 3, "cuda")
    dy = on_gpu(MANY, 65, t, 4)
    dx = awq.awq_w4a16_input_grad(dy, *wide)
    want, e = P.input_grad(dy[rows], P.weights(*wide), t)
    close(dx[rows], want, P.rounded(want, e, t), "dX")


@pytest.mark.parametrize("t,group", [(F16, 32), (BF16, 128)], ids=str)
def test_param_grad_past_2_31_elements(awq, t, group):
    """Values of -1, 0 and 1: every product and sum is a whole number that
    binary32 holds, so any order gives the same."""
    _say(f"many rows, parameters {t} g{group}")
    layer = P.make_layer(2304, 128, group, 5, "cuda")
    dy, x = on_gpu(MANY, 2304, t, 6, True), on_gpu(MANY, 128, t, 7, True)
    ds, dz = awq.awq_w4a16_param_grad(dy, x, *layer)
    d = torch.zeros(2304, 128, dtype=P.F64, device="cuda")
    for i in range(0, MANY, 1 << 17):
        d += dy[i:i + (1 << 17)].to(F32).T.contiguous() @ x[i:i + (1 << 17)].to(F32)
    d = d.view(2304, 128 // group, group)
    q = P.differences(layer[0], layer[2]).view(d.shape)
    assert torch.equal(ds.to(P.F64), (d * q).sum(-1))
    sums = d.sum(-1)
    assert bool(((dz + layer[1].float() * sums.float()).abs() <= P.U32 * dz.abs()).all())


@pytest.mark.parametrize("n,t", [(1, F16), (20, BF16), (100, F16), (600, BF16)], ids=str)
def test_codes_past_2_31_bytes(awq, n, t):
    _say(f"codes {n} {t}")
    o, k, group = 131200, 32896, 128
    g = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randint(-2 ** 31, 2 ** 31, (o, k // 8), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    s = (0.002 + 0.01 * torch.rand(o, k // group, generator=g, device="cuda")).to(F16)
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda").to(F16)
    x = on_gpu(n, k, t, n + 1)
    rows = torch.tensor([*range(3), 65599, 65600, 65601, *range(130556, 130562), *range(o - 70, o)], device="cuda")
    w = P.weights(q[rows], s[rows], z[rows])
    y = awq.awq_w4a16_linear(x, q, s, z)
    want, e = P.linear(x, w)
    close(y[:, rows], want, P.rounded(want, e, t), "Y")
    words = torch.tensor([0, 1, k // 16, k // 8 - 1], device="cuda")
    cols = (8 * words[:, None] + torch.arange(8, device="cuda")).flatten()
    d = P.codes(q[:, words].contiguous()) - z[:, cols // group].to(P.F64)
    dy = on_gpu(n, o, t, n + 2)
    dx = awq.awq_w4a16_input_grad(dy, q, s, z)
    want, e = P.input_grad(dy, d * s[:, cols // group].to(P.F64), t)
    close(dx[:, cols], want, P.rounded(want, e, t), "dX")
    ds, dz = awq.awq_w4a16_param_grad(dy, x, q, s, z)
    ws_, es, wz, ez = P.param_grad(dy[:, rows], x, q[rows], s[rows], z[rows])
    close(ds[rows], ws_, P.rounded(ws_, es, F32), "dstep")
    close(dz[rows], wz, P.rounded(wz, ez, F32), "dzero")
