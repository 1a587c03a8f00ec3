"""A decoder's attention block on the GPU as a server runs it: a fused projection
with adapters, the 4-bit cache, attention over it, the projection back.  Every
step is held to its plain form on what the step before left."""
import pytest
import torch

import kv4_plain as K
import post_bit_weight_awq_amd as awq
import w4_adapt_plain as AP
import w4_plain as P
from test_kv4_gpu import append_plain, back, on_gpu, same
from test_w4_adapt_gpu import gpu, inside

pytestmark = pytest.mark.gpu
H, B = torch.float16, torch.bfloat16


class Block:
    """Heads of D columns, `per` to a kv head; two packed layers and adapters for each."""

    def __init__(self, hidden, kv, per, d, group, page, pages, dtype, seed, rank=16, count=3):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.heads, self.d, self.group, self.dtype = kv, kv * per, d, group, dtype
        out = (self.heads + 2 * kv) * d
        self.qkv, self.proj = P.make_layer(out, hidden, 128, seed), P.make_layer(hidden, self.heads * d, 64, seed + 1)
        norm = lambda *s: (0.05 * torch.randn(*s, generator=g)).to(dtype)
        self.a1, self.b1 = norm(count, rank, hidden), norm(count, out, rank)
        self.a2, self.b2 = norm(count, rank, self.heads * d), norm(count, hidden, rank)
        self.scale = 0.5 + torch.rand(count, generator=g)
        self.hold = K.make_cache(pages, kv, page, d, group, seed + 2)
        self.cache = on_gpu(self.hold)
        self.on = [gpu(v) for v in (self.qkv, self.a1, self.b1, self.scale, self.proj, self.a2, self.b2)]

    def run(self, x, ids, slots, table, lens, starts=None):
        """All on the GPU, with nothing between the steps."""
        qkv, a1, b1, scale, proj, a2, b2 = self.on
        y = awq.awq_w4a16_adapted(x, *qkv, a1, b1, scale, ids).view(x.shape[0], -1, self.d)
        q, k, v = y[:, :self.heads], y[:, self.heads:self.heads + self.kv], y[:, self.heads + self.kv:]
        awq.awq_kv4_append(k, v, self.cache, slots)
        o = awq.awq_kv4_attention(q, self.cache, table, lens, starts=starts)
        return y, o, awq.awq_w4a16_adapted(o.view(x.shape[0], -1), *proj, a2, b2, scale, ids)

    def check(self, x, ids, slots, table, lens, starts=None):
        n = x.shape[0]
        y, o, z = (t.cpu() for t in self.run(x.cuda(), ids.cuda(), slots.cuda(), table.cuda(), lens.cuda(),
                                             None if starts is None else starts.cuda()))
        t = self.dtype
        want, e, _, _ = AP.forward_bounds(x, self.qkv, self.a1, self.b1, self.scale, ids, t)
        inside(y.view(n, -1), want, AP.rounded(want, e, t), "projection")
        q, k, v = y[:, :self.heads], y[:, self.heads:self.heads + self.kv], y[:, self.heads + self.kv:]
        self.hold = append_plain(self.hold, k, v, slots, self.group)
        assert same(back(self.cache), self.hold)
        want, bound = K.attention_all(q, self.hold, table, lens, starts, self.d ** -0.5, t)
        assert bool(((o.to(P.F64) - want).abs() <= bound).all())
        want, e, _, _ = AP.forward_bounds(o.view(n, -1), self.proj, self.a2, self.b2, self.scale, ids, t)
        inside(z, want, AP.rounded(want, e, t), "projection back")


@pytest.mark.parametrize("dtype,kv,per,d,group,page", [(H, 2, 2, 128, 128, 16), (B, 1, 8, 64, 32, 32), (B, 4, 1, 64, 64, 64)])
def test_prompts_then_tokens(dtype, kv, per, d, group, page):
    """Ragged prompts, then steps of one token each, one of them with an idle sequence."""
    runs, width = [37, 1, 70], 3 if page > 32 else 6
    b = Block(256, kv, per, d, group, page, 3 * width + 1, dtype, 5)
    g = torch.Generator().manual_seed(9)
    table = torch.randperm(3 * width + 1, generator=g)[:3 * width].view(3, width).to(torch.int32)
    slot = lambda s, i: int(table[s, i // page]) * page + i % page
    starts = torch.tensor([0, 37, 38, 108], dtype=torch.int32)
    slots = torch.tensor([slot(s, i) for s, n in enumerate(runs) for i in range(n)], dtype=torch.int32)
    ids = torch.tensor([2, -1, 0], dtype=torch.int32)
    lens = torch.tensor(runs, dtype=torch.int32)
    b.check(torch.randn(108, 256, generator=g).to(dtype), ids.repeat_interleave(lens), slots, table, lens, starts)
    for step in range(3):
        at = [slot(s, int(n)) for s, n in enumerate(lens)]
        lens = lens + 1
        seen = lens.clone()
        if step == 1:  # the second sequence is idle: its row sees nothing and is written nowhere
            at[1], seen[1], lens[1] = -1, 0, lens[1] - 1
        b.check(torch.randn(3, 256, generator=g).to(dtype), ids, torch.tensor(at, dtype=torch.int32), table, seen)


@pytest.mark.parametrize("dtype", [H, B])
def test_a_step_in_a_graph(dtype):
    """A captured step, replayed for new tokens, has the bits of the calls one by one."""
    n, page, width = 20, 32, 4
    x, ids, slots, lens = (torch.zeros(n, 256, dtype=dtype, device="cuda"), *(torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3)))
    two = [Block(256, 2, 4, 64, 32, page, n * width, dtype, 3) for _ in range(2)]
    table = torch.arange(n * width, dtype=torch.int32).view(n, width).cuda()
    step = lambda b: b.run(x, ids, slots, table, lens)
    slots.fill_(-1)
    step(two[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(two[0])
    g = torch.Generator().manual_seed(1)
    have = torch.randint(0, 90, (n,), generator=g)
    for i in range(4):
        x.copy_(torch.randn(n, 256, generator=g).to(dtype))
        ids.copy_(torch.randint(-1, 3, (n,), generator=g))
        slots.copy_(torch.arange(n) * width * page + have + i)
        lens.copy_(have + i + 1)
        graph.replay()
        torch.cuda.synchronize()
        want = step(two[1])
        assert all(torch.equal(a, c) for a, c in zip(got, want))
        assert same(back(two[0].cache), back(two[1].cache))
