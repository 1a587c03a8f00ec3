"""The 4-bit cache and attention over it on the GPU, against the plain forms."""
import math

import pytest
import torch

import kv4_plain as K
import post_bit_weight_awq_amd as awq

pytestmark = pytest.mark.gpu
H, B = torch.float16, torch.bfloat16
SIZES = [(128, 128), (128, 64), (128, 32), (64, 64), (64, 32)]


def on_gpu(cache):
    return awq.Kv4Cache(*(x.cuda() for x in cache))


def back(c):
    return tuple(x.cpu() for x in (c.k_codes, c.v_codes, c.k_params, c.v_params))


def same(a, b):
    return all(torch.equal(x.view(torch.int16 if x.dtype == H else x.dtype), y.view(torch.int16 if y.dtype == H else y.dtype))
               for x, y in zip(a, b))


def rows(n, h, d, dtype, seed, strided):
    """Keys and values; strided: slices of a fused projection's output."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, 3 * h, d, generator=g) * 2).to(dtype)
    k, v = x[:, h:2 * h], x[:, 2 * h:]
    return (x, k, v) if strided else (x, k.contiguous(), v.contiguous())


def append_plain(cache, k, v, slots, group):
    kc, vc, kp, vp = (x.clone() for x in cache)
    d = k.shape[-1]
    page = kc.shape[2]
    ck, pk = K.quantize(k, group)
    cv, pv = K.quantize(v, group)
    wk, wv = K.words(ck), K.words(cv)
    for t, s in enumerate(slots.tolist()):
        if s < 0 or s >= kc.shape[0] * page:
            continue
        p, i = s // page, s % page
        kc[p, :, i, K.k_at(d)] = wk[t]
        vc[p, :, i // 16, :, i % 16] = wv[t]
        kp[p, :, i], vp[p, :, i] = pk[t], pv[t]
    return kc, vc, kp, vp


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("d,group", SIZES)
@pytest.mark.parametrize("n,h,page,strided", [(1, 1, 16, False), (7, 3, 32, True), (133, 2, 128, True), (64, 8, 64, False)])
def test_append_bit_for_bit(dtype, d, group, n, h, page, strided):
    pages = -(-n // page) + 2
    cache = K.make_cache(pages, h, page, d, group, 1)
    x, k, v = rows(n, h, d, dtype, 2, strided)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:n].to(torch.int32)
    if n > 5:
        slots[2], slots[4] = -1, pages * page + 3  # padding and a place that is none
        slots[5] = pages * page - 1
    c = on_gpu(cache)
    xd = x.cuda()
    kd, vd = (xd[:, h:2 * h], xd[:, 2 * h:]) if strided else (k.cuda(), v.cuda())
    awq.awq_kv4_append(kd, vd, c, slots.cuda())
    want = append_plain(cache, k, v, slots, group)
    assert same(back(c), want)  # other places as they were
    # read back, some places twice and a padded one
    at = torch.cat([slots, slots[:3], torch.tensor([-7], dtype=torch.int32)])
    gk, gv = awq.awq_kv4_gather(c, at.cuda(), dtype=dtype)
    for got, ref in zip((gk, gv), K.read(want)):
        for t, s in enumerate(at.tolist()):
            w = ref[s // page, :, s % page] if 0 <= s < pages * page else torch.zeros(h, d, dtype=K.F64)
            assert torch.equal(got[t].cpu(), w.to(torch.float32).to(dtype))


@pytest.mark.parametrize("dtype", [H, B])
def test_append_extremes(dtype):
    d, group, page = 128, 32, 16
    k = torch.zeros(8, 1, d)
    k[0, 0, 3] = math.nan
    k[0, 0, 40] = math.inf
    k[0, 0, 70] = -math.inf
    k[1] = 3.25                         # equal values
    k[2, 0, ::2], k[2, 0, 1::2] = 65504, -65504
    k[3] = torch.linspace(-1, 1, d) * (3e38 if dtype is B else 6e4)
    k[4] = torch.linspace(1, 2, d) * 2e-7  # subnormal steps
    k[5] = 1000 + torch.linspace(0, 1, d)
    k[6] = torch.linspace(-3, 3, d) ** 3
    k = k.to(dtype)
    v = k.flip(0).contiguous()
    cache = K.make_cache(1, 1, page, d, group, 1)
    slots = torch.arange(8, dtype=torch.int32) + 5
    c = on_gpu(cache)
    awq.awq_kv4_append(k.cuda(), v.cuda(), c, slots.cuda())
    want = append_plain(cache, k, v, slots, group)
    got = back(c)
    for a, b in zip(got, want):
        assert torch.equal(torch.nan_to_num(a.float(), nan=7e30), torch.nan_to_num(b.float(), nan=7e30))
    gk, _ = awq.awq_kv4_gather(c, slots.cuda(), dtype=dtype)
    assert bool(gk[0, 0, :96].isnan().all()) and bool((gk[0, 0, 96:] == 0).all()) and bool((gk[1] == 3.25).all())


def attend(cache, q, table, lens, starts=None, scale=None, out=None):
    return awq.awq_kv4_attention(q, cache, table.cuda(), lens.cuda(), starts=None if starts is None else starts.cuda(),
                                 scale=scale, out=out)


def table_of(lens, page, pages, seed, width=None):
    need = [-(-n // page) for n in lens]
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    width = width or max(1, max(need))
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    assert at <= pages
    return t


def check(got, want, bound):
    rows_ = ~want.isnan()
    e = (got.cpu().to(K.F64) - want)[rows_].abs()
    assert bool((e <= bound[rows_]).all()), float((e / bound[rows_].clamp(min=1e-300)).max())


def make(lens, h, per, page, d, group, dtype, seed, runs=None, width=None):
    pages = sum(-(-n // page) for n in lens) + 1
    cache = K.make_cache(pages, h, page, d, group, seed)
    table = table_of(lens, page, pages, seed, width)
    n = len(lens) if runs is None else sum(runs)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(n, h * per, d, generator=g).to(dtype)
    starts = None
    if runs is not None:
        starts = torch.tensor([sum(runs[:i]) for i in range(len(runs) + 1)], dtype=torch.int32)
    return cache, table, torch.tensor(lens, dtype=torch.int32), q, starts


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("d,group", SIZES)
@pytest.mark.parametrize("h,per,page", [(1, 1, 16), (2, 4, 32), (1, 8, 64), (3, 3, 128), (1, 16, 16), (2, 11, 64), (1, 40, 32)])
def test_decode(dtype, d, group, h, per, page):
    lens = [1, 0, 15, 16, 17, 31, 33, 64, 129, 300]
    cache, table, l, q, _ = make(lens, h, per, page, d, group, dtype, per + page)
    got = attend(on_gpu(cache), q.cuda(), table, l)
    check(got, *K.attention_all(q, cache, table, l, None, d ** -0.5, dtype))
    assert bool((got[1] == 0).all())


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("d,group,page,h,per,n", [(128, 128, 16, 1, 2, 4111), (128, 64, 128, 2, 1, 2500), (64, 32, 32, 1, 4, 3003),
                                                  (128, 32, 64, 1, 12, 1025)])
def test_decode_splits(dtype, d, group, page, h, per, n):
    """One or two sequences: the keys are split over blocks; a short one beside a long one leaves splits empty."""
    lens = [n, 77]
    cache, table, l, q, _ = make(lens, h, per, page, d, group, dtype, n, width=-(-n // page) + 40)
    got = attend(on_gpu(cache), q.cuda(), table, l, scale=0.11)
    check(got, *K.attention_all(q, cache, table, l, None, 0.11, dtype))


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("d,group", SIZES)
@pytest.mark.parametrize("h,per,page", [(2, 1, 16), (1, 4, 64), (1, 7, 32)])
def test_chunks(dtype, d, group, h, per, page):
    """Ragged runs: none, one token, more tokens than keys, a run that begins a sequence."""
    lens, runs = [5, 70, 40, 0, 3, 161, 33], [5, 0, 1, 2, 7, 90, 33]
    cache, table, l, q, starts = make(lens, h, per, page, d, group, dtype, page, runs)
    got = attend(on_gpu(cache), q.cuda(), table, l, starts)
    check(got, *K.attention_all(q, cache, table, l, starts, d ** -0.5, dtype))


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("per", [1, 8])
def test_few_tokens_each(dtype, per):
    """Runs so short that they are served as single tokens are."""
    lens, runs = [300, 40, 1, 513, 90], [1, 2, 0, 2, 1]
    cache, table, l, q, starts = make(lens, 2, per, 32, 128, 64, dtype, 9, runs, width=60)
    got = attend(on_gpu(cache), q.cuda(), table, l, starts)
    check(got, *K.attention_all(q, cache, table, l, starts, 128 ** -0.5, dtype))


def test_rows_of_no_sequence_stay():
    lens, runs = [40, 20], [6, 3]
    cache, table, l, q, starts = make(lens, 1, 2, 16, 64, 32, H, 3, runs)
    q = torch.cat([q, q[:5]])
    for starts_ in (starts, starts + 2):
        out = torch.full((14, 2, 64), 7.0, dtype=H, device="cuda")
        attend(on_gpu(cache), q.cuda(), table, l, starts_, out=out)
        want, bound = K.attention_all(q, cache, table, l, starts_, 0.125, H)
        check(out, want, bound)
        assert bool((out.cpu()[want.isnan()] == 7).all())


@pytest.mark.parametrize("runs", [None, [40, 33]])
def test_strided_queries(runs):
    lens = [100, 47]
    cache, table, l, q, starts = make(lens, 2, 2, 16, 128, 64, B, 4, runs)
    fused = torch.zeros(q.shape[0], 8, 128, dtype=B)
    fused[:, 2:6] = q
    got = attend(on_gpu(cache), fused.cuda()[:, 2:6], table, l, starts)
    check(got, *K.attention_all(q, cache, table, l, starts, 128 ** -0.5, B))


@pytest.mark.parametrize("runs", [None, [50, 2, 30]])
def test_nan_where_no_row_looks(runs):
    """NaN and infinities behind a sequence's end, in other pages, and at keys that only later rows see."""
    lens, page = [50, 17, 60], 32
    cache, table, l, q, starts = make(lens, 2, 2, page, 128, 64, H, 6, runs)
    kc, vc, kp, vp = (x.clone() for x in cache)
    used = torch.zeros(kp.shape[0], page, dtype=torch.bool)
    for s, n in enumerate(lens):
        for j in range(n):
            used[table[s, j // page], j % page] = True
    for p in (kp, vp):
        p.transpose(1, 2)[~used] = math.nan
    kp.transpose(1, 2)[~used, :, :, 0] = math.inf
    got = attend(on_gpu((kc, vc, kp, vp)), q.cuda(), table, l, starts)
    check(got, *K.attention_all(q, cache, table, l, starts, 128 ** -0.5, H))
    # the last key of the first sequence
    at = (int(table[0, 49 // page]), 49 % page)
    for p in (kp, vp):
        p[at[0], :, at[1]] = math.nan
    bad = attend(on_gpu((kc, vc, kp, vp)), q.cuda(), table, l, starts)
    last = 0 if runs is None else runs[0] - 1
    assert bool(bad[last].isnan().all())
    keep = [t for t in range(q.shape[0]) if t != last]
    assert torch.equal(bad[keep], got[keep])


@pytest.mark.parametrize("runs", [None, [45, 2]])
def test_bad_pages_are_not_seen(runs):
    lens = [100, 64]
    cache, table, l, q, starts = make(lens, 1, 4, 16, 128, 128, H, 8, runs)
    table[0, 2], table[0, 4], table[1, 0] = -1, cache[0].shape[0], 2 ** 31 - 1
    table[1, 3] = -2 ** 31
    got = attend(on_gpu(cache), q.cuda(), table, l, starts)
    check(got, *K.attention_all(q, cache, table, l, starts, 128 ** -0.5, H))
    table[:] = -5
    got = attend(on_gpu(cache), q.cuda(), table, l, starts)
    assert bool((got == 0).all())


def test_lengths_past_the_table_and_shared_pages():
    cache, table, l, q, _ = make([64, 64], 1, 1, 16, 64, 64, B, 8)
    table[1, :3] = table[0, :3]
    l = torch.tensor([1000, 57], dtype=torch.int32)
    got = attend(on_gpu(cache), q.cuda(), table, l)
    check(got, *K.attention_all(q, cache, table, l, None, 0.125, B))
    assert bool((attend(on_gpu(cache), q.cuda(), table, torch.tensor([-3, 0], dtype=torch.int32)) == 0).all())


def test_odd_queries():
    """An infinity or NaN in one query leaves the others; large scores; scale 0."""
    cache, table, l, q, _ = make([90, 33, 40], 1, 2, 16, 128, 64, H, 8)
    want = attend(on_gpu(cache), q.cuda(), table, l)
    bad = q.clone()
    bad[1, 0, 5] = math.inf
    bad[2, 1, 0] = math.nan
    got = attend(on_gpu(cache), bad.cuda(), table, l)
    assert bool(got[1, 0].isnan().all()) and bool(got[2, 1].isnan().all())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1, 1], want[1, 1]) and torch.equal(got[2, 0], want[2, 0])
    for scale in (0.0, 30.0, -3.0):
        got = attend(on_gpu(cache), q.cuda(), table, l, scale=scale)
        check(got, *K.attention_all(q, cache, table, l, None, scale, H))


def test_far_pages():
    """Pages behind 2^31 words and 2^32 bytes."""
    pages, h, page, d = 70000, 16, 128, 128
    c = awq.Kv4Cache(torch.empty(pages, h, page, 16, dtype=torch.int32, device="cuda"),
                     torch.empty(pages, h, page // 16, 16, 16, dtype=torch.int32, device="cuda"),
                     torch.empty(pages, h, page, 1, 2, dtype=H, device="cuda"),
                     torch.empty(pages, h, page, 1, 2, dtype=H, device="cuda"))
    _, k, v = rows(200, h, d, H, 5, False)
    order = torch.tensor([pages - 1, pages - 3], dtype=torch.int64)
    j = torch.arange(200)
    slots = (order[j // page] * page + j % page).to(torch.int32)
    awq.awq_kv4_append(k.cuda(), v.cuda(), c, slots.cuda())
    gk, gv = awq.awq_kv4_gather(c, slots.cuda())
    small = K.store(*K.quantize(torch.zeros(2, h, page, d).half(), 128), *K.quantize(torch.zeros(2, h, page, d).half(), 128))
    small = append_plain(small, k, v, j.to(torch.int32), 128)
    for got, want in zip((gk, gv), K.read(small)):
        assert torch.equal(got.cpu(), want.transpose(1, 2).flatten(0, 1)[:200].float().half())
    q = torch.randn(3, h, d, generator=torch.Generator().manual_seed(1)).half()
    want, bound = K.attention_all(q, small, torch.tensor([[0, 1]], dtype=torch.int32), [200], [0, 3], d ** -0.5, H)
    for starts in (torch.tensor([0, 3], dtype=torch.int32),):
        got = attend(c, q.cuda(), order[None].to(torch.int32), torch.tensor([200], dtype=torch.int32), starts)
        check(got, want, bound)
    got = attend(c, q[2:].cuda(), order[None].to(torch.int32), torch.tensor([200], dtype=torch.int32))
    check(got, want[2:], bound[2:])


def test_a_sequence_grown_token_by_token():
    """Append and attend step by step against the whole prompt at once, in pages that fill up."""
    n, h, per, d, page = 37, 2, 2, 64, 16
    c = awq.awq_kv4_cache(4, h, page, d, 32)
    whole = awq.awq_kv4_cache(4, h, page, d, 32)
    _, k, v = rows(n, h, d, B, 5, False)
    q = torch.randn(n, h * per, d, generator=torch.Generator().manual_seed(1)).to(B).cuda()
    k, v = k.cuda(), v.cuda()
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    j = torch.arange(n)
    slots = (table[0].long()[j // page] * page + j % page).to(torch.int32).cuda()
    awq.awq_kv4_append(k, v, whole, slots)
    got = attend(whole, q, table, torch.tensor([n], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32))
    want, bound = K.attention_all(q.cpu(), back(whole), table, [n], [0, n], d ** -0.5, B)
    check(got, want, bound)
    steps = []
    for t in range(n):
        awq.awq_kv4_append(k[t:t + 1], v[t:t + 1], c, slots[t:t + 1])
        steps.append(attend(c, q[t:t + 1], table, torch.tensor([t + 1], dtype=torch.int32)))
    assert same(back(c), back(whole))
    check(torch.cat(steps), want, bound)


@pytest.mark.parametrize("runs", [None, [40, 33]])
def test_streams_workspaces_and_graphs(runs):
    """Another stream, a used workspace, the same bits again, and a captured append and attention replayed on new data."""
    lens = [700, 47]
    cache, table, l, q, starts = make(lens, 2, 2, 16, 128, 64, B, 4, runs)
    c = on_gpu(cache)
    dt, dl, ds = table.cuda(), l.cuda(), None if starts is None else starts.cuda()
    qd = q.cuda()
    want = awq.awq_kv4_attention(qd, c, dt, dl, starts=ds)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(awq.awq_kv4_attention(qd, c, dt, dl, starts=ds, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = awq.awq_kv4_attention(qd, c, dt, dl, starts=ds, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    n = q.shape[0]
    _, k, v = rows(n, 2, 128, B, 1, False)
    kd, vd = k.cuda(), v.cuda()
    slots = torch.arange(n, dtype=torch.int32).cuda() + 3
    out = torch.empty_like(qd)

    def step():
        awq.awq_kv4_append(kd, vd, c, slots)
        awq.awq_kv4_attention(qd, c, dt, dl, starts=ds, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        kd.copy_(torch.roll(k.cuda(), i, 0))
        qd.copy_(torch.roll(q.cuda(), i, 0))
        dl.copy_(l.cuda() - i)
        graph.replay()
        got = out.clone()
        ws.fill_(i)
        step()
        assert torch.equal(got, out)
        torch.cuda.synchronize()


def test_more_blocks_than_one_dimension_takes():
    """Launches of more than 2^32 threads: the last tokens, heads and sequences are reached."""
    d, page, n = 64, 16, 2 ** 20
    hold = K.make_cache(4, 130, page, d, 32, 1)
    c = on_gpu(hold)
    k = torch.randn(4099, 1, d, generator=torch.Generator().manual_seed(2)).to(B)
    kd = k.cuda()[torch.arange(n, device="cuda") % 4099].expand(n, 130, d)
    slots = torch.full((n,), -1, dtype=torch.int32)
    tail = torch.arange(n - 60, n)
    slots[tail] = torch.arange(60, dtype=torch.int32)
    slots[5] = 61
    awq.awq_kv4_append(kd, kd, c, slots.cuda())
    at = torch.cat([tail, torch.tensor([5])])
    x = k[at % 4099].expand(61, 130, d)
    want = append_plain(hold, x, x, slots[at], 32)
    assert same(back(c), want)
    every = torch.arange(n, dtype=torch.int32, device="cuda") % 64
    few = awq.awq_kv4_gather(c, every[:64], dtype=B)
    for got, part in zip(awq.awq_kv4_gather(c, every, dtype=B), few):
        assert bool((got.view(-1, 64, 130, d) == part).all())


@pytest.mark.parametrize("heads,run", [(17, None), (114, 17)])
def test_more_units_than_one_dimension_takes(heads, run):
    d, page = 64, 16
    c = on_gpu(K.make_cache(3, heads, page, d, 32, 1))
    q = torch.randn(1, heads, d, generator=torch.Generator().manual_seed(2)).half().cuda()
    if run is None:
        seqs, few = 2 ** 20, 17
        lens = torch.arange(seqs, dtype=torch.int32) % few
        starts = lambda s: None
        n = 1
    else:
        seqs, few = 2 ** 15 + 5, 1
        lens = torch.full((seqs,), 16, dtype=torch.int32)
        starts = lambda s: torch.arange(s + 1, dtype=torch.int32) * run
        n = run
    table = torch.full((seqs, 1), 2, dtype=torch.int32)
    part = attend(c, q.expand(few * n, heads, d), table[:few], lens[:few], starts(few))
    got = attend(c, q.expand(seqs * n, heads, d), table, lens, starts(seqs))
    whole = seqs // few * few * n
    assert bool((got[:whole].view(-1, few * n, heads, d) == part).all())
    assert torch.equal(got[whole:], part[:seqs * n - whole])


@pytest.mark.parametrize("runs", [None, [40, 33]])
@pytest.mark.parametrize("scale", [2.0 ** 32, -2.0 ** 32])
def test_largest_scales(scale, runs):
    """All weight is on one key: its values, off by their two bf16 parts (2^-17), the
    quotient of the sums (a few 2^-24) and the output's rounding."""
    lens, h, d = [50, 700], 2, 128
    hold = K.make_cache(50, h, 16, d, 64, 3)
    g = torch.Generator().manual_seed(5)
    table = torch.randperm(50, generator=g)[:44 + 4].view(1, -1)[:, :44].repeat(2, 1).to(torch.int32)
    n = len(lens) if runs is None else sum(runs)
    q = torch.randn(n, 2 * h, d, generator=g).half()
    starts = None if runs is None else torch.tensor([0, runs[0], n], dtype=torch.int32)
    got = attend(on_gpu(hold), q.cuda(), table, torch.tensor(lens, dtype=torch.int32), starts, scale=scale).cpu().to(K.F64)
    k, v = K.read(hold)
    size = K.size_of(d, hold[3])
    for s in range(2):
        a, b = (s, s + 1) if runs is None else (int(starts[s]), int(starts[s + 1]))
        for t in range(a, b):
            j = torch.arange(lens[s] - (b - 1 - t))
            p, i = table[s, j // 16].long(), j % 16
            for x in range(2 * h):
                best = int((scale * (k[p, x // 2, i] @ q[t, x].to(K.F64))).argmax())
                one, big = v[p[best], x // 2, i[best]], size[p[best], x // 2, i[best]]
                bound = 2.0 ** -16 * big
                assert bool(((got[t, x] - one).abs() <= bound + K.half_step(H) * (one.abs() + bound) + K.tiny(H)).all()), (t, x)
