"""Forms of the 4-bit cache's kernels that need long inputs: runs of tokens whose keys are split into parts that meet in a
second launch, and appends of four heads at a time."""
import math

import pytest
import torch

import kv4_plain as K
import kv4_rows as R
import post_bit_weight_awq_amd as awq
from test_kv4_gpu import SIZES, append_plain, attend, back, check, make, on_gpu, rows, same

H, B = torch.float16, torch.bfloat16


def test_rows_at_a_time_are_the_plain_form():
    for runs in (None, [5, 0, 9, 3]):
        cache, table, l, q, starts = make([40, 3, 9, 0], 2, 3, 16, 64, 32, B, 4, runs)
        table[0, 1] = -1
        want, got = (f(q, cache, table, l, starts, 0.2, B) for f in (K.attention_all, R.attention_all))
        for a, b in zip(want, got):
            assert bool(((a - b).abs() <= 2.0 ** -40 * (1 + a.abs())).all())


# a sequence of many parts, one whose first rows see nothing of its later parts, one of one part, none, fewer keys than rows
LENS, RUNS = [3000, 1200, 40, 0, 9], [70, 900, 40, 0, 20]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("d,group", SIZES)
@pytest.mark.parametrize("h,per,page", [(1, 4, 16), (2, 1, 64), (1, 7, 128)])
def test_runs_in_parts(dtype, d, group, h, per, page):
    cache, table, l, q, starts = make(LENS, h, per, page, d, group, dtype, page, RUNS)
    got = attend(on_gpu(cache), q.cuda(), table, l, starts)
    want, bound = R.attention_all(q.cuda(), tuple(t.cuda() for t in cache), table, l, starts, d ** -0.5, dtype)
    check(got, want.cpu(), bound.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("d,group", [(128, 64), (64, 32)])
def test_parts_with_bad_pages_and_nan(dtype, d, group):
    page = 32
    cache, table, l, q, starts = make(LENS, 2, 2, page, d, group, dtype, 3, RUNS)
    table[0, 40:43], table[0, 60] = -1, cache[0].shape[0]  # inside middle parts
    table[1, 16:32] = -7                                  # the second part of the second sequence, whole
    got = attend(on_gpu(cache), q.cuda(), table, l, starts)
    want, bound = R.attention_all(q.cuda(), tuple(t.cuda() for t in cache), table, l, starts, d ** -0.5, dtype)
    check(got, want.cpu(), bound.cpu())
    # NaN at keys that only a sequence's last rows see, in its last part: those rows alone have it
    for s, back_by in ((0, 5), (1, 130)):
        kc, vc, kp, vp = (x.clone() for x in cache)
        j = LENS[s] - back_by
        at = int(table[s, j // page])
        for p in (kp, vp):
            p[at, :, j % page] = math.nan
        bad = attend(on_gpu((kc, vc, kp, vp)), q.cuda(), table, l, starts)
        end = int(starts[s + 1])
        hit = torch.zeros(q.shape[0], dtype=torch.bool)
        hit[end - back_by:end] = True
        assert bool(bad[hit].isnan().all()) and torch.equal(bad[~hit], got[~hit])
    # nothing but bad pages
    table[:] = 2 ** 31 - 1
    assert bool((attend(on_gpu(cache), q.cuda(), table, l, starts) == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [H, B])
def test_parts_in_a_graph(dtype):
    """Replayed for other lengths and runs, behind a used workspace: the bits of the call by itself."""
    cache, table, l, q, starts = make(LENS, 2, 4, 64, 128, 128, dtype, 5, RUNS)
    c, qd, td, ld, sd = on_gpu(cache), q.cuda(), table.cuda(), l.cuda(), starts.cuda()
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(qd)
    call = lambda: awq.awq_kv4_attention(qd, c, td, ld, starts=sd, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, runs in ((LENS, RUNS), ([1500, 1216, 2, 31, 16], [700, 100, 2, 31, 1]), ([3008, 0, 0, 0, 0], [1030, 0, 0, 0, 0]),
                       ([513, 512, 40, 64, 9], [513, 512, 1, 1, 3])):
        ld.copy_(torch.tensor(lens, dtype=torch.int32))
        sd.copy_(torch.tensor([sum(runs[:i]) for i in range(6)], dtype=torch.int32))
        out.zero_()
        graph.replay()
        got = out.clone()
        ws.fill_(len(runs) + lens[0] % 200)
        out.zero_()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        want, bound = R.attention_all(qd, tuple(t.cuda() for t in cache), table, lens, sd.cpu(), 128 ** -0.5, dtype)
        check(got, want.cpu(), bound.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,d,group,page,dtype", [(4095, 40, 128, 32, 64, B), (4095, 40, 128, 128, 16, H), (2731, 12, 128, 64, 32, B),
                                                    (8191, 8, 64, 32, 128, H), (8191, 8, 64, 64, 16, B)])
def test_append_of_four_heads_bit_for_bit(n, h, d, group, page, dtype):
    """Prompts of heads that come in fours, from slices of a fused projection's output, with padding among them."""
    pages = -(-n // page) + 2
    cache = K.make_cache(pages, h, page, d, group, 1)
    x, k, v = rows(n, h, d, dtype, 2, True)
    g = torch.Generator().manual_seed(3)
    order = torch.randperm(pages, generator=g)
    at = torch.arange(n)
    slots = (order[at // page] * page + at % page).to(torch.int32)
    none = torch.randint(0, n, (50,), generator=g)
    slots[none] = torch.where(none % 2 == 0, -1, pages * page + 5).to(torch.int32)
    # a stretch of tokens in mixed order
    slots[100:200] = slots[100:200][torch.randperm(100, generator=g)]
    c = on_gpu(cache)
    xd = x.cuda()
    awq.awq_kv4_append(xd[:, h:2 * h], xd[:, 2 * h:], c, slots.cuda())
    assert same(back(c), append_plain(cache, k, v, slots, group))
