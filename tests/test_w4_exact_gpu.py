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


def close(got, want, bound, what):
    got = got.to(P.F64)
    ok = ((got - want).abs() <= bound) | (got == want)
    if not bool(ok.all()):
        at = (~ok).nonzero()[0].tolist()
        worst = ((got - want).abs() / bound.clamp_min(1e-300))[~ok].max()
        pytest.fail(f"{what}: {int((~ok).sum())} of {ok.numel()} off, worst {float(worst):.3g} bounds, first at {at}: "
                    f"{float(got[tuple(at)])} for {float(want[tuple(at)])}")


# ------------------------------------------------------------------- long sums
@pytest.mark.parametrize("n,o", [(4096, 4096), (1024, 4096)])
@pytest.mark.parametrize("steps", ["one", "equal", "none between"])
def test_units_do_not_drift(awq, steps, n, o):
    """What the first of 432 groups adds goes unchanged through the others, whose units are the same (one step for all
    rows, one per row, groups without a step between).  Whole tiles, so that the sum is not split.  The first group's
    32 products are positive: their sum and the last product by the unit are off by 33 half steps at most, and by
    sqrt(33) of them or less in the mean square; twice that, as the matrix unit may cut a sum rather than round it."""
    _say("drift", steps, n, o)
    k, group = 13824, 32
    ng = k // group
    q, s, z = P.make_layer(o, k, group, 3, "cuda")
    z.zero_()
    g = torch.Generator().manual_seed(4)
    own = ((1024 + torch.randint(0, 1024, (o, 1), generator=g)).to(torch.float64) * 2.0 ** -18).to(F16).cuda()
    if steps == "one":
        s.fill_(1312 * 2.0 ** -18)
    else:
        s.copy_(own.expand(o, ng))
        if steps == "none between":
            s[:, 1::2] = 0
    x = torch.zeros(n, k, dtype=F16, device="cuda")
    x[:, :group] = torch.rand(n, group, generator=g).to(F16).cuda()
    got = awq.awq_w4a16_linear(x, q, s, z, out_dtype=F32).to(P.F64)
    w = E.weights(q[:, :group // 8].contiguous(), s[:, :1].contiguous(), z[:, :1].contiguous())
    want = x[:, :group].to(P.F64) @ w.T
    off = (got - want) / want.clamp_min(1e-9)
    assert float(off.abs().max()) <= 2 * 33 * P.U32
    assert float(off.square().mean().sqrt()) <= 2 * 33 ** 0.5 * P.U32


# ------------------------------------------------------------ zeros of any value
ODD_ZEROS = [0.001, -0.001, 2.0 ** -24, 2.998, 3.002, 0.3333, 1.001, 7.004, 7.996, 11.99, 14.99, -0.3, -5.7, -16.98,
             17.02, 20.3, 31.97, 240.5, 300.6, 1023.5, 2032, 2040, -2047, 2049, 5000, -5008, 65504, -65504, 0, 15]


def odd_layer(o, k, group, seed):
    """Zeros of every kind, a different one per group, among them a row of fractions in 0..15 and one of whole ones."""
    q, s, z = P.make_layer(o, k, group, seed, "cuda")
    g = torch.Generator().manual_seed(seed)
    v = torch.tensor(ODD_ZEROS, dtype=torch.float64)
    z.copy_(v[torch.randint(0, len(v), z.shape, generator=g)].to(F16))
    z[0] = (15 * torch.rand(z.shape[1], generator=g)).to(F16).cuda()
    z[1] = 7
    return q, s, z


def size(q, z, k):
    """|q - z| and what a split of z into a part that the codes' differences hold and a remainder adds: at most a
    quarter, beyond 240 |z|."""
    z = P.spread(z, k).abs()
    return q.abs() + torch.where(z > 240, 2 * z, 0.25)


BY_TYPE = pytest.mark.parametrize("t,group", [(F16, 128), (F16, 64), (F16, 32), (BF16, 128), (BF16, 64), (BF16, 32)],
                                  ids=lambda v: str(v).replace("torch.", ""))


@pytest.mark.parametrize("n", [1, 4, 12, 30, 48, 64, 100, 200, 600])
@BY_TYPE
def test_each_weight_alone(awq, n, t, group):
    """One column per token, all others 0: the output is one weight times a power of two, the fp32 output off by the
    few roundings of its own operations."""
    _say(f"each weight {n} {t} g{group}")
    k, o = 384, 75
    layer = odd_layer(o, k, group, n + group)
    x = torch.zeros(n, k, dtype=t, device="cuda")
    at = (torch.arange(n, device="cuda") * 7 + 3) % k
    x[torch.arange(n, device="cuda"), at] = torch.exp2((torch.arange(n, device="cuda") % 5 - 2).float()).to(t)
    d, s = E.differences(layer[0], layer[2]), P.spread(layer[1], k)
    xd = x.to(P.F64)
    close(awq.awq_w4a16_linear(x, *layer, out_dtype=F32), xd @ (d * s).T,
          8 * P.U32 * (xd.abs() @ (size(d, layer[2], k) * s).T), "Y")


@pytest.mark.parametrize("n,k,o", [(1, 512, 200), (3, 1152, 40), (16, 640, 333), (40, 512, 200), (64, 256, 20481), (64, 384, 520),
                                   (70, 512, 640), (200, 1152, 250), (600, 640, 700), (1100, 512, 4100)])
@BY_TYPE
def test_products_with_any_zero(awq, n, k, o, t, group):
    _say(f"any zero {n}x{k}->{o} {t} g{group}")
    layer = odd_layer(2 * o, k, group, n + o)
    layer[2].clamp_(-300, 300)
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, k, generator=g).to(t).cuda()
    w = E.weights(*layer)
    xd = x.to(P.F64)
    sums = xd.abs() @ (size(E.differences(layer[0], layer[2]), layer[2], k) * P.spread(layer[1], k)).T
    want, e = xd @ w.T, 2 * (k + 128) * P.U32 * sums
    close(awq.awq_w4a16_linear(x, *layer, out_dtype=F32), want, e, "fp32")
    close(awq.awq_w4a16_linear(x, *layer), want, P.rounded(want, e, t), "16 bits")
    h, pre = awq.awq_w4a16_gated(x, *layer, keep_pre=True)
    close(pre, want, P.rounded(want, e, t), "pre")
    a, u, ea, eu = P.act(want[:, :o], "silu")[0], want[:, o:], e[:, :o], e[:, o:]
    ea = 1.13 * ea + 16 * P.U32 * want[:, :o].abs()
    close(h, a * u, P.rounded(a * u, (a.abs() + ea) * eu + ea * u.abs() + 2 * P.U32 * (a * u).abs(), t), "H")


@pytest.mark.parametrize("n", [1, 4, 30, 64, 100, 300])
@BY_TYPE
def test_infinities_beside_zeros_next_to_a_code(awq, n, t, group):
    """An infinity times q - z is one of q - z's sign, however near z lies to q, and NaN for q = z alone."""
    _say(f"infinities next to codes {n} {t} g{group}")
    k, o = 256, 96
    q, s, z = P.make_layer(o, k, group, 16, "cuda")
    off = torch.tensor([2.0 ** -7, -2.0 ** -7, 2.0 ** -9, -2.0 ** -9, 0], device="cuda")
    z.copy_((z.float() + off[torch.arange(o, device="cuda") % 5][:, None]).to(F16))
    x = torch.randn(n, k, generator=torch.Generator().manual_seed(n)).to(t).cuda()
    x[0, 7], x[n // 2, 130], x[n - 1, 255] = float("inf"), float("-inf"), float("inf")
    want = x.to(P.F64) @ E.weights(q, s, z).T
    got = awq.awq_w4a16_linear(x, q, s, z, out_dtype=F32).to(P.F64)
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf])


def test_large_finite_rows_keep_their_remainders(awq):
    """Sums of a group past binary32's end, within it in the operators' unit of 512 steps: so are the token sums that a
    zero's remainder multiplies."""
    _say("large finite rows")
    k, o = 256, 64
    q, s, z = P.make_layer(o, k, 128, 18, "cuda", "any")
    s.fill_(2.0 ** -24)
    for n in (1, 20, 100):
        x = torch.full((n, k), 6.0e37, dtype=BF16, device="cuda")
        x[:, 1::2] = 4.0e37
        w = E.weights(q, s, z)
        xd = x.to(P.F64)
        e = 2 * (k + 128) * P.U32 * (xd @ (size(E.differences(q, z), z, k) * P.spread(s, k)).T)
        close(awq.awq_w4a16_linear(x, q, s, z, out_dtype=F32), xd @ w.T, e, n)


@pytest.mark.parametrize("n,k,o", [(1, 256, 300), (3, 640, 17), (33, 512, 130), (129, 384, 193), (600, 1024, 260)])
@BY_TYPE
def test_param_grad_with_any_zero(awq, n, k, o, t, group):
    _say(f"dstep {n}x{k},{o} {t} g{group}")
    layer = odd_layer(o, k, group, n + k)
    g = torch.Generator().manual_seed(n)
    dy, x = (0.01 * torch.randn(n, o, generator=g)).to(t).cuda(), torch.randn(n, k, generator=g).to(t).cuda()
    ds, dz = awq.awq_w4a16_param_grad(dy, x, *layer)
    d = (dy.to(P.F64).T @ x.to(P.F64)).view(o, k // group, group)
    da = (dy.to(P.F64).abs().T @ x.to(P.F64).abs()).view(d.shape)
    q = E.differences(layer[0], layer[2]).view(d.shape)
    e = 2 * (n + group + 64) * P.U32
    close(ds, (d * q).sum(-1), e * (da * q.abs()).sum(-1) + 2.0 ** -149, "dstep")
    s = layer[1].to(P.F64)
    close(dz, -s * d.sum(-1), e * s * da.sum(-1) + 2.0 ** -149, "dzero")


# ----------------------------------------------------------------- large weights
@pytest.mark.parametrize("n,o", [(1, 72), (40, 72), (130, 200), (300, 1000), (600, 72)])
@BY_TYPE
def test_input_grad_of_weights_past_fp16(awq, n, o, t, group):
    """Weights beyond 65504, by their step or by their zero, beside ordinary ones: dX is finite where the sum is."""
    _say(f"large weights {n} {o} {t} g{group}")
    k = 640
    q, s, z = P.make_layer(o, k, group, 9, "cuda", "any")
    s[3, 0], s[7, -1], s[11] = 60000.0, -9000.0, 130.0
    z[13], z[17, 0], s[17, 0] = 60000.0, -65504.0, 100.0
    z[19, 1], s[19, 1] = 2000.0, 127.0
    g = torch.Generator().manual_seed(n)
    dy = (2.0 ** -14 * torch.randn(n, o, generator=g)).to(t).cuda()
    dy[:, 17] = 2.0 ** -24
    got = awq.awq_w4a16_input_grad(dy, q, s, z)
    # each weight off by two roundings to 11 bits, its zero by 2^-16 and a half of its last place
    w, a = E.weights(q, s, z), dy.to(P.F64).abs()
    y = dy.to(P.F64) @ w
    sl = P.spread(s, k).abs()
    b = 2 * (o + 64) * P.U32 * (a @ w.abs()) + a @ (2.0 ** -10 * w.abs() + 2.0 ** -15 * sl + 2.0 ** -24)
    assert bool(got.isfinite().all())
    close(got, y, P.rounded(y, b, t), "dX")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gate_gradient_of_large_factors(awq, act):
    """dH U leaves binary32's range and the slope brings it back."""
    _say("large factors", act)
    g = torch.tensor([-60.0, -30.0, -8.0, -3.0], device="cuda").to(BF16)
    f = 64
    gate = g.repeat(f // 4)
    pre = torch.stack([torch.cat([gate, torch.full_like(gate, u)]) for u in (1e20, -1e25, 3.0)])
    dh = torch.full((3, f), 1e18, dtype=BF16, device="cuda")
    dh[0, ::3] = 1e19
    layer = P.make_layer(2 * f, 128, 128, 7, "cuda")
    _, dpre = awq.awq_w4a16_gated_backward(dh, pre, *layer, act=act)
    want, e = P.gated_grad(dh, pre, act)
    finite = want.abs() < 3.38e38
    close(torch.where(finite, dpre.to(P.F64), 0), torch.where(finite, want, 0), P.rounded(want, e, BF16), "dpre")


# ------------------------------------------------------------------ the binding
def test_tracked_tensors_are_refused(awq):
    """Any tensor of a call, outputs too; a Function joins the calls to autograd."""
    _say("tracked tensors")
    n, k, o = 5, 256, 96
    q, s, z = P.make_layer(o, k, 64, 3, "cuda")
    x = torch.randn(n, k, device="cuda").to(F16)
    dy = torch.randn(n, o, device="cuda").to(F16)
    y = torch.zeros(n, o, dtype=F16, device="cuda", requires_grad=True)
    for a, kw in (((x, q, s.clone().requires_grad_(), z), {}), ((x, q, s, z.clone().requires_grad_()), {}),
                  ((x, q, s, z), {"out": y})):
        with pytest.raises(RuntimeError, match="requires a gradient"):
            awq.awq_w4a16_linear(*a, **kw)
    with pytest.raises(RuntimeError, match="X requires a gradient"):
        awq.awq_w4a16_param_grad(dy, x.clone().requires_grad_(), q, s, z)

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, s, z):
            ctx.save_for_backward(x, s, z)
            return awq.awq_w4a16_linear(x, q, s, z)

        @staticmethod
        def backward(ctx, dy):
            x, s, z = ctx.saved_tensors
            ds, dz = awq.awq_w4a16_param_grad(dy, x, q, s, z)
            return awq.awq_w4a16_input_grad(dy, q, s, z), ds.to(F16), dz.to(F16)

    args = [t.clone().requires_grad_() for t in (x, s, z)]
    Linear.apply(*args).backward(dy)
    ds, dz = awq.awq_w4a16_param_grad(dy, x, q, s, z)
    for got, want in zip(args, (awq.awq_w4a16_input_grad(dy, q, s, z), ds.to(F16), dz.to(F16))):
        assert torch.equal(got.grad, want)


# ------------------------------------------------------------ how calls are made
def poisoned(awq, op, n, k, o, group, t):
    """A workspace of exactly the stated size, full of NaN bytes."""
    size = getattr(awq.load(), f"awq_w4a16_{op}_workspace_size")(n, k, o, group, 0 if t == F16 else 1)
    return torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("n,k,o", [(65, 128, 33), (70, 512, 640), (200, 1152, 250), (600, 640, 700), (2, 131072, 40), (90, 4224, 4160)])
@BY_TYPE
def test_any_zero_in_a_used_workspace(awq, n, k, o, t, group):
    """What a call has not written itself stays out of its result: NaN all over the workspace, zeros with remainders in
    some blocks of 32 rows and groups alone."""
    _say(f"poisoned {n}x{k}->{o} {t} g{group}")
    q, s, z = P.make_layer(2 * o, k, group, n, "cuda")
    z[-1, -1], z[o // 2, 0] = 3.3, 0.4
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, k, generator=g).to(t).cuda()
    got = awq.awq_w4a16_linear(x, q, s, z, out_dtype=F32, workspace=poisoned(awq, "linear", n, k, 2 * o, group, t))
    xd, d = x.to(P.F64), E.differences(q, z)
    e = 2 * (k + 128) * P.U32 * (xd.abs() @ (size(d, z, k) * P.spread(s, k)).T)
    want = xd @ E.weights(q, s, z).T
    close(got, want, e, "Y")
    _, pre = awq.awq_w4a16_gated(x, q, s, z, keep_pre=True, workspace=poisoned(awq, "gated", n, k, o, group, t))
    close(pre, want, P.rounded(want, e, t), "pre")


@pytest.mark.parametrize("n", [1, 20, 64, 100, 600])
@pytest.mark.parametrize("t", [F16, BF16], ids=str)
def test_zeros_and_steps_change_between_replays(awq, n, t):
    """A captured call looks at the layer as it then is: whole zeros, fractions, steps beyond fp16's weights, back."""
    _say(f"replays {n} {t}")
    k, o, group = 512, 200, 64
    q, s, z = P.make_layer(o, k, group, 4, "cuda")
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, k, generator=g).to(t).cuda()
    dy = (0.001 * torch.randn(n, o, generator=g)).to(t).cuda()
    whole, step = z.clone(), s.clone()

    def go():
        y = awq.awq_w4a16_linear(x, q, s, z, out_dtype=F32)
        return [y, awq.awq_w4a16_input_grad(dy, q, s, z), *awq.awq_w4a16_param_grad(dy, x, q, s, z)]

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go()
    seen = []
    for part, large in ((0.0, False), (0.37, False), (0.37, True), (0.0, False)):
        z.copy_((whole.float() + part).to(F16))
        s.copy_(step)
        if large:
            s[3, 1] = 400.0
        eager = go()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, out):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        seen.append([v.clone() for v in out])
    assert not torch.equal(seen[0][0], seen[1][0])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(seen[0], seen[3]))
