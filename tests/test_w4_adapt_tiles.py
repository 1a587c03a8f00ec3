"""Adapters in every tile height of the tiled products: tiles of 64 to 256 tokens, whole ones and ones whose sum is split,
with mixed adapters in a tile of 16 tokens and a ragged last tile."""
import pytest
import torch

import post_bit_weight_awq_amd as awq
import tile_choice
import w4_adapt_plain as AP
from test_w4_adapt_gpu import inside, make

H, B, F32 = torch.float16, torch.bfloat16, torch.float32

# ("f" forward or "b" backward, tokens, in, out): 32-token units of a tile, whole tiles too, split ones
TILES = {
    ("f", 1800, 256, 2050): (4, True, False), ("f", 1800, 3968, 514): (4, False, True),
    ("f", 900, 256, 8200): (6, True, False), ("f", 3600, 8192, 514): (6, False, True),
    ("f", 1400, 256, 8200): (8, True, False), ("f", 3400, 8192, 1030): (8, False, True),
    ("b", 4100, 1024, 130): (4, True, False), ("b", 400, 2048, 6150): (4, False, True),
    ("b", 4100, 2048, 130): (6, True, False), ("b", 1300, 2048, 12300): (6, False, True),
    ("b", 3100, 4096, 130): (8, True, False), ("b", 4100, 4096, 1000): (8, True, True),
}
GROUPS_OF_64 = {("f", 1500, 1024, 8200): (8, True, False)}


def test_the_shapes_take_these_tiles(tmp_path):
    for shapes, scale in ((TILES, "1.0f"), (GROUPS_OF_64, "1.2f")):
        got = tile_choice.choices(tmp_path, list(shapes), scale)
        for shape, (mt, full, left, _) in zip(shapes, got):
            assert (mt, full > 0, left > 0) == shapes[shape], shape


def on_gpu(case):
    return tuple(tuple(t.cuda() for t in v) if isinstance(v, tuple) else v.cuda() for v in case)


def check(got, want, bound, name):
    inside(got, want.cpu(), bound.cpu(), name)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n,k,o,group,rank,count", [(*s[1:], 128, r, c) for s, (r, c) in zip(
    [t for t in TILES if t[0] == "f"], [(16, 5), (64, 3), (24, 9), (8, 40), (128, 3), (16, 5)])] + [(1500, 1024, 8200, 64, 40, 7)])
def test_forward(dtype, n, k, o, group, rank, count):
    layer, x, _, a, b, scale, ids = on_gpu(make(n, k, o, group, dtype, rank, count, n + rank))
    for y_type in (dtype, F32):
        got, kept = awq.awq_w4a16_adapted(x, *layer, a, b, scale, ids, out_dtype=y_type, keep_low=True)
        y, e, low, el = AP.forward_bounds(x, layer, a, b, scale, ids, y_type)
        check(got, y, AP.rounded(y, e, y_type), "y")
        check(kept, low, el, "low")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [H, B])
@pytest.mark.parametrize("n,k,o,group,rank,count", [(*s[1:], g, r, c) for s, (g, r, c) in zip(
    [t for t in TILES if t[0] == "b"], [(128, 16, 5), (64, 64, 3), (32, 24, 9), (128, 8, 40), (64, 128, 3), (128, 16, 5)])])
def test_backward(dtype, n, k, o, group, rank, count):
    layer, x, dy, a, b, scale, ids = on_gpu(make(n, k, o, group, dtype, rank, count, n + rank))
    low = AP.forward(x, AP.weights(*layer), a, b, scale, ids)[1].float()
    got = awq.awq_w4a16_adapted_backward(dy, x, low, *layer, a, b, scale, ids)
    want = AP.backward_bounds(dy, x, low, layer, a, b, scale, ids)
    check(got[0], want[0][0], AP.rounded(*want[0], dtype), "dx")
    check(got[1], want[1][0], AP.rounded(*want[1], F32), "da")
    check(got[2], want[2][0], AP.rounded(*want[2], F32), "db")
