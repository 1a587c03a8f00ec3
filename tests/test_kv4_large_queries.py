"""Queries of any finite size: bf16's reach 3e38, where sums of (16 + code) Q before the step enters, and scores before
the scale, lie past binary32."""
import math

import pytest
import torch

import kv4_plain as K
import kv4_rows as R
from kv4_plain import F64, U32
from test_kv4_gpu import attend, check, make, on_gpu

pytestmark = pytest.mark.gpu
H, B = torch.float16, torch.bfloat16

# one launch for single tokens and their split keys, runs of tokens, runs in parts
FORMS = [([90, 33, 1], None), ([3003], None), ([70, 40], [33, 40]), ([1100, 30], [150, 30])]


@pytest.mark.parametrize("lens,runs", FORMS)
@pytest.mark.parametrize("d,group", [(128, 128), (128, 32), (64, 64)])
@pytest.mark.parametrize("up", [90, 96, 110, 124, 126])
def test_scores_of_ordinary_size(lens, runs, d, group, up):
    """Queries of 2^up with a scale that brings their scores back: weights as of ordinary queries."""
    cache, table, l, q, starts = make(lens, 1, 4, 32, d, group, B, 7, runs)
    q = (q.float().clamp(-3.9, 3.9) * 2.0 ** up).to(B)
    assert bool(q.isfinite().all())
    scale = 2.0 ** -(up + 3)  # a power of two, exact in binary32 where it is subnormal too
    got = attend(on_gpu(cache), q.cuda(), table, l, starts, scale=scale)
    want, bound = R.attention_all(q.cuda(), tuple(t.cuda() for t in cache), table, l, starts, scale, B)
    assert bool(bound.isfinite().all())
    check(got, want.cpu(), bound.cpu())


@pytest.mark.parametrize("lens,runs", FORMS)
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149])
def test_the_least_scales(lens, runs, scale):
    """All keys weigh alike at 0; at the least scale the largest queries still count."""
    cache, table, l, q, starts = make(lens, 1, 4, 32, 128, 64, B, 7, runs)
    q = (q.float().clamp(-3.9, 3.9) * 2.0 ** 126).to(B)
    got = attend(on_gpu(cache), q.cuda(), table, l, starts, scale=scale)
    want, bound = R.attention_all(q.cuda(), tuple(t.cuda() for t in cache), table, l, starts, scale, B)
    check(got, want.cpu(), bound.cpu())


@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("lens,runs", FORMS)
def test_all_weight_on_one_key(dtype, lens, runs):
    """The type's largest queries at ordinary and the largest scales: the row's best key alone counts.  Its values are off by
    their two bf16 parts (2^-17), the quotient of the sums (a few 2^-24) and the output's rounding."""
    h, d = 1, 128
    cache, table, l, q, starts = make(lens, h, 2, 32, d, 64, dtype, 9, runs)
    big = torch.finfo(dtype).max
    q = torch.where(q > 0, big, -big).to(dtype)
    k, v = K.read(cache)
    sk, sv = K.size_of(d, cache[2]), K.size_of(d, cache[3])
    for scale in (d ** -0.5, -2.0 ** 32):
        got = attend(on_gpu(cache), q.cuda(), table, l, starts, scale=scale).cpu().to(F64)
        assert not bool(got.isnan().any())
        held = 0
        for s in range(len(lens)):
            a, b = (s, s + 1) if starts is None else (int(starts[s]), int(starts[s + 1]))
            for t in range(a, b):
                j = torch.arange(lens[s] - (b - 1 - t))
                p, i = table[s, j // 32].long(), j % 32
                for x in range(2):
                    f = q[t, x].to(F64)
                    z, e = scale * (k[p, 0, i] @ f), abs(scale) * 2 * (d + 64) * U32 * (sk[p, 0, i] @ f.abs())
                    best = int(z.argmax())
                    rest = (z + e).index_fill(0, torch.tensor([best]), -math.inf)
                    if z[best] - e[best] <= rest.max() + 100:
                        continue  # the two best lie within what binary32 holds of them
                    held += 1
                    one, size = v[p[best], 0, i[best]], sv[p[best], 0, i[best]]
                    bound = 2.0 ** -16 * size
                    assert bool(((got[t, x] - one).abs() <= bound + K.half_step(dtype) * (one.abs() + bound) + K.tiny(dtype)).all()), (t, x)
        assert held > 0


@pytest.mark.parametrize("lens,runs", FORMS)
def test_small_and_large_queries_beside_each_other(lens, runs):
    """Rows of 2^-130 to 2^126 in one tile, and values that far apart in one row, at the largest scale that keeps them apart."""
    cache, table, l, q, starts = make(lens, 1, 4, 32, 128, 128, B, 11, runs)
    q = q.float().clamp(-3.9, 3.9)
    far = q.clone()
    f = 2.0 ** torch.linspace(-130, 126, q.shape[0] * 4).round().view(-1, 4, 1).to(F64)
    far = (q.to(F64) * f).to(B)
    far[:, 0] = (q[:, 0].to(F64) * 2.0 ** torch.linspace(-120, 30, 128).round().to(F64)).to(B)
    for scale in (1.0, 2.0 ** -20, 2.0 ** -129):
        got = attend(on_gpu(cache), far.cuda(), table, l, starts, scale=scale)
        want, bound = R.attention_all(far.cuda(), tuple(t.cuda() for t in cache), table, l, starts, scale, B)
        want, bound = want.cpu(), bound.cpu()
        assert not bool(got.isnan().any())
        # rows whose scores binary32 holds to no better than a hundred have no bound
        ok = bound.isfinite().all(-1)
        assert bool(ok.any())
        want[~ok] = math.nan
        check(got, want, bound)


@pytest.mark.parametrize("lens,runs", FORMS)
def test_what_is_not_finite_stays_so(lens, runs):
    cache, table, l, q, starts = make(lens, 1, 4, 32, 128, 64, B, 7, runs)
    want = attend(on_gpu(cache), q.cuda(), table, l, starts)
    last = q.shape[0] - 1
    for i, bad in enumerate((math.inf, -math.inf, math.nan)):
        x = q.clone()
        x[last, i, 40 + i] = bad
        got = attend(on_gpu(cache), x.cuda(), table, l, starts)
        assert bool(got[last, i].isnan().all())
        keep = torch.ones(q.shape[:2], dtype=torch.bool)
        keep[last, i] = False
        assert torch.equal(got[keep], want[keep])
