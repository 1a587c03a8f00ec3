"""Adapters beside a packed product on the GPU, against the plain forms."""
import math

import pytest
import torch

import post_bit_weight_awq_amd as awq
import w4_adapt_plain as AP
import w4_plain as P

pytestmark = pytest.mark.gpu
H, B, F32 = torch.float16, torch.bfloat16, torch.float32


def make(n, k, o, group, dtype, rank, count, seed, ids="any", zeros="packed"):
    g = torch.Generator().manual_seed(seed)
    layer = P.make_layer(o, k, group, seed, zeros=zeros)
    loud = torch.where(torch.rand(k, generator=g) < 0.01, 8.0, 1.0)
    x = (torch.randn(n, k, generator=g) * loud).to(dtype)
    dy = (1e-2 * torch.randn(n, o, generator=g)).to(dtype)
    a = (0.05 * torch.randn(count, rank, k, generator=g)).to(dtype)
    b = (0.05 * torch.randn(count, o, rank, generator=g)).to(dtype)
    scale = 0.5 + torch.rand(count, generator=g)
    if ids == "any":  # every token another one, some none
        i = torch.randint(-1, count, (n,), generator=g)
    elif ids == "runs":
        i = torch.randint(-1, count, (9,), generator=g)[torch.arange(n) * 9 // n]
    elif ids == "none":
        i = torch.full((n,), -1)
    elif ids == "odd":  # places that are none
        i = torch.tensor([-1, count, 2 ** 31 - 1, -2 ** 31, 0, count - 1])[torch.randint(0, 6, (n,), generator=g)]
    else:
        i = torch.full((n,), count - 1)
    return layer, x, dy, a, b, scale, i.to(torch.int32)


def gpu(v):
    return tuple(gpu(i) for i in v) if isinstance(v, tuple) else v.cuda()


def inside(got, want, bound, name):
    got = got.cpu().to(P.F64)
    e = (got - want).abs()
    assert bool((e <= bound).all()), (name, float((e / bound.clamp(min=1e-300)).max()))


def forward(case, y_type, keep):
    layer, x, _, a, b, scale, ids = case
    dl, dx, da, db, ds, di = gpu(layer), x.cuda(), a.cuda(), b.cuda(), scale.cuda(), ids.cuda()
    got = awq.awq_w4a16_adapted(dx, *dl, da, db, ds, di, out_dtype=y_type, keep_low=keep)
    y, e, low, el = AP.forward_bounds(x, layer, a, b, scale, ids, y_type)
    inside(got[0] if keep else got, y, AP.rounded(y, e, y_type), "y")
    if keep:
        inside(got[1], low, el, "low")
    return got


SHAPES = [(1, 512, 48, 128), (3, 1024, 333, 64), (16, 256, 1000, 32), (17, 512, 250, 128), (47, 384, 100, 64), (64, 256, 24576, 128),
          (64, 128, 40, 32), (65, 512, 300, 128), (200, 1152, 517, 64), (333, 256, 129, 32), (1100, 384, 640, 128)]


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n,k,o,group", SHAPES)
@pytest.mark.parametrize("rank,count,ids", [(8, 1, "one"), (16, 5, "any"), (24, 3, "runs"), (64, 40, "any"), (128, 2, "odd")])
def test_forward(dtype, n, k, o, group, rank, count, ids):
    case = make(n, k, o, group, dtype, rank, count, n + rank, ids)
    forward(case, dtype, False)
    forward(case, F32, True)


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n", [1, 40, 600])
def test_forward_zeros_and_none(dtype, n):
    """Zeros of any value; tokens without an adapter have the plain product's bits."""
    forward(make(n, 512, 300, 64, dtype, 16, 3, n, "runs", zeros="any"), dtype, True)
    case = make(n, 512, 300, 64, dtype, 16, 3, n, "none")
    y, low = forward(case, F32, True)
    assert torch.equal(y, awq.awq_w4a16_linear(case[1].cuda(), *gpu(case[0]), out_dtype=F32)) and bool((low == 0).all())


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n", [1, 7, 63, 130])
def test_forward_splits_of_long_rows(dtype, n):
    """Long rows: single tokens share the sum of low among blocks."""
    forward(make(n, 13824, 160, 128, dtype, 16, 4, n), dtype, False)


def backward(case, w=None):
    layer, x, dy, a, b, scale, ids = case
    low = AP.forward(x, AP.weights(*layer), a, b, scale, ids)[1].float()
    low[(ids < 0) | (ids >= len(scale))] = math.nan  # not looked at
    got = awq.awq_w4a16_adapted_backward(dy.cuda(), x.cuda(), low.cuda(), *gpu(layer), a.cuda(), b.cuda(), scale.cuda(), ids.cuda())
    want = AP.backward_bounds(dy, x, torch.nan_to_num(low), layer, a, b, scale, ids)
    inside(got[0], want[0][0], AP.rounded(*want[0], dy.dtype), "dx")
    for i, name in ((1, "da"), (2, "db")):
        inside(got[i], want[i][0], AP.rounded(*want[i], F32), name)
    return got


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n,k,o,group", [(1, 256, 40, 128), (31, 512, 333, 64), (65, 128, 1, 32), (200, 1152, 517, 64), (333, 256, 130, 32),
                                         (1100, 384, 640, 128), (2100, 256, 200, 64)])
@pytest.mark.parametrize("rank,count,ids", [(8, 1, "one"), (16, 5, "any"), (24, 3, "runs"), (64, 40, "any"), (128, 2, "odd"), (72, 2, "none")])
def test_backward(dtype, n, k, o, group, rank, count, ids):
    backward(make(n, k, o, group, dtype, rank, count, n + rank, ids))


@pytest.mark.parametrize("dtype", [H, B])
def test_backward_zeros_and_big_weights(dtype):
    backward(make(150, 512, 300, 64, dtype, 16, 3, 5, "runs", zeros="any"))
    case = make(150, 512, 300, 64, dtype, 16, 3, 5, "runs")
    case[0][1][7, 2] = 200.0  # a step beyond what the matrix units take
    backward(case)


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n", [5, 300])
def test_far_magnitudes(dtype, n):
    """low beyond fp16 and far below it, per token."""
    case = make(n, 512, 100, 128, dtype, 16, 2, 3)
    layer, x, dy, a, b, scale, ids = case
    f = torch.logspace(-2, 3, n)[:, None]
    x = (torch.randn(n, 512, generator=torch.Generator().manual_seed(1)) * f).to(dtype)
    a = (a.float() * 40).to(dtype)
    case = (layer, x, dy, a, b, scale, ids)
    forward(case, F32, True)
    backward(case)


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n", [6, 70])
def test_non_finite_tokens_stay_alone(dtype, n):
    case = make(n, 512, 100, 128, dtype, 16, 2, 3)
    layer, x, dy, a, b, scale, ids = case
    ids[:] = torch.arange(n, dtype=torch.int32) % 2
    want = forward(case, F32, True)
    bad = x.clone()
    bad[1, 4], bad[3, 9] = math.nan, math.inf
    got = awq.awq_w4a16_adapted(bad.cuda(), *gpu(layer), a.cuda(), b.cuda(), scale.cuda(), ids.cuda(), out_dtype=F32, keep_low=True)
    keep = [t for t in range(n) if t not in (1, 3)]
    for u, v in zip(got, want):
        assert torch.equal(u[keep], v[keep]) and not bool(u[[1, 3]].isfinite().all(1).any())
    # another adapter's infinities do not reach a token
    a2, b2 = a.clone(), b.clone()
    a2[1, 3, 5], b2[1, 7, 2] = math.inf, math.nan
    got = awq.awq_w4a16_adapted(x.cuda(), *gpu(layer), a2.cuda(), b2.cuda(), scale.cuda(), ids.cuda(), out_dtype=F32, keep_low=True)
    for u, v in zip(got, want):
        assert torch.equal(u[::2], v[::2])


def test_gradients_against_differences():
    """The kernels' own gradients against central differences of the kernels' forward pass."""
    layer, x, dy, a, b, scale, ids = make(70, 256, 96, 64, H, 16, 3, 7)
    c = torch.randn(70, 96, generator=torch.Generator().manual_seed(2)).half()
    dl = gpu(layer)
    ds, di = scale.cuda(), ids.cuda()

    def loss(x, a, b):
        return float((awq.awq_w4a16_adapted(x.cuda(), *dl, a.cuda(), b.cuda(), ds, di, out_dtype=F32).double() * c.cuda().double()).sum())

    _, low = awq.awq_w4a16_adapted(x.cuda(), *dl, a.cuda(), b.cuda(), ds, di, keep_low=True)
    grads = awq.awq_w4a16_adapted_backward(c.cuda(), x.cuda(), low, *dl, a.cuda(), b.cuda(), ds, di)
    args = [x, a, b]
    for i, got in enumerate(grads):
        g = torch.Generator().manual_seed(i)
        # Y is linear in each argument: a step of the values' own size has no error of its own
        v = (args[i].float() * torch.where(torch.rand(args[i].shape, generator=g) < 0.5, 1.0, -1.0)).to(H)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = (args[i].float() + v.float()).half(), (args[i].float() - v.float()).half()
        num = (loss(*hi) - loss(*lo)) / 2
        want = (got.double().cpu() * v.double())
        # 2 v is exact; dX is rounded to fp16 and its weights are (2^-11 each)
        assert abs(num - float(want.sum())) <= 2.0 ** -10 * float(want.abs().sum())


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_streams_workspaces_and_graphs(dtype, n):
    """Another stream, a used workspace, the same bits again; a captured training step replayed on other tokens and adapters."""
    layer, x, dy, a, b, scale, ids = make(n, 1024, 200, 64, dtype, 16, 3, 7)
    dl, dx, ddy, da, db, ds, di = gpu(layer), x.cuda(), dy.cuda(), a.cuda(), b.cuda(), scale.cuda(), ids.cuda()
    stack = (*dl, da, db, ds, di)
    want = awq.awq_w4a16_adapted(dx, *stack)
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(awq.awq_w4a16_adapted(dx, *stack, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = awq.awq_w4a16_adapted(dx, *stack, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    y, low = awq.awq_w4a16_adapted(dx, *stack, keep_low=True)
    outs = [torch.empty_like(dx), torch.empty_like(da, dtype=F32), torch.empty_like(db, dtype=F32)]

    def step():
        awq.awq_w4a16_adapted(dx, *stack, out=y, low=low, workspace=ws)
        awq.awq_w4a16_adapted_backward(ddy, dx, low, *stack, out=outs[0], dA=outs[1], dB=outs[2], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        dx.copy_(torch.roll(x.cuda(), i, 0) * (i + 1))
        di.copy_((ids + i) % 4 - 1)
        ws.fill_(255 - i)
        graph.replay()
        got = [v.clone() for v in (y, low, *outs)]
        for v in (y, low, *outs):
            v.zero_()
        ws.fill_(i)
        step()
        assert all(torch.equal(u, v) for u, v in zip(got, (y, low, *outs)))
        torch.cuda.synchronize()


class Adapted(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, b, layer, scale, ids):
        y, low = awq.awq_w4a16_adapted(x, *layer, a, b, scale, ids, keep_low=True)
        ctx.save_for_backward(x, a, b, low, *layer, scale, ids)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, a, b, low, q, s, z, scale, ids = ctx.saved_tensors
        dx, da, db = awq.awq_w4a16_adapted_backward(dy.contiguous(), x, low, q, s, z, a, b, scale, ids)
        return dx, da.to(a.dtype), db.to(b.dtype), None, None, None


def test_two_layers_under_autograd():
    """Gradients of a chain of two adapted layers against binary64's."""
    l1, x, _, a1, b1, scale, ids = make(50, 256, 384, 64, H, 16, 3, 7)
    l2, _, dy, a2, b2, _, _ = make(50, 384, 128, 128, H, 16, 3, 8)
    leaves = [v.cuda().requires_grad_() for v in (x, a1, b1, a2, b2)]
    ds, di = scale.cuda(), ids.cuda()
    y = Adapted.apply(leaves[0], leaves[1], leaves[2], gpu(l1), ds, di)
    y = Adapted.apply(y, leaves[3], leaves[4], gpu(l2), ds, di)
    y.backward(dy.cuda())
    f = [v.to(P.F64).requires_grad_() for v in (x, a1, b1, a2, b2)]

    def plain(x, w, a, b):
        mine = (ids[:, None] == torch.arange(3)).to(P.F64)[:, :, None]
        low = torch.einsum("tk,ark->tar", x, a) * mine * scale.to(P.F64)[None, :, None]
        return x @ w.T + torch.einsum("tar,aor->to", low, b)

    z = plain(plain(f[0], AP.weights(*l1), f[1], f[2]), AP.weights(*l2), f[3], f[4])
    z.backward(dy.to(P.F64))
    for got, want in zip(leaves, f):
        # each 16-bit rounding on the way (y, weights, dx, the gradients' type) is
        # half a step of 2^-10; they add like independent errors of a norm
        rel = float((got.grad.double().cpu() - want.grad).norm() / want.grad.norm())
        assert rel <= 6 * 2.0 ** -11, rel


def test_more_blocks_than_one_dimension_takes():
    """So many adapters that the launch that lays them out has more than 2^32 threads: the last ones too."""
    n, k, o, count = 5, 8192, 8192, 32768
    layer, x, dy, _, _, _, _ = make(n, k, o, 128, B, 8, 1, 3)
    ids = torch.tensor([count - 1, 0, -1, count - 1, 20000], dtype=torch.int32)
    used = [0, 20000, count - 1]
    g = torch.Generator().manual_seed(4)
    few_a, few_b = (0.05 * torch.randn(3, 8, k, generator=g)).to(B), (0.05 * torch.randn(3, o, 8, generator=g)).to(B)
    a, b = torch.zeros(count, 8, k, dtype=B, device="cuda"), torch.zeros(count, o, 8, dtype=B, device="cuda")
    a[used], b[used] = few_a.cuda(), few_b.cuda()
    scale = torch.linspace(0.5, 1.5, count)
    low = torch.randn(n, 8, generator=g)
    dx, da, db = awq.awq_w4a16_adapted_backward(dy.cuda(), x.cuda(), low.cuda(), *gpu(layer), a, b, scale.cuda(), ids.cuda())
    few_ids = torch.tensor([2, 0, -1, 2, 1], dtype=torch.int32)
    want = AP.backward_bounds(dy, x, low, layer, few_a, few_b, scale[used], few_ids)
    inside(dx, want[0][0], AP.rounded(*want[0], B), "dx")
    inside(da[used], want[1][0], AP.rounded(*want[1], F32), "da")
    inside(db[used], want[2][0], AP.rounded(*want[2], F32), "db")
    assert int(da.count_nonzero(dim=(1, 2)).count_nonzero()) == 3 == int(db.count_nonzero(dim=(1, 2)).count_nonzero())
