"""Kv4Cache holds addresses: what they point to cannot be exchanged behind its back."""
import pytest
import torch

import post_bit_weight_awq_amd as awq

ARRAYS = ("k_codes", "v_codes", "k_params", "v_params")
SIZES = ("n_pages", "n_heads", "page_size", "head_dim", "group_size")


def make(device="cpu"):
    return awq.awq_kv4_cache(4, 2, 16, 64, 32, device=device)


@pytest.mark.parametrize("name", ARRAYS + SIZES)
def test_arrays_and_sizes_are_read_only(name):
    c = make()
    before = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, torch.zeros_like(before) if name in ARRAYS else before + 1)
    with pytest.raises(AttributeError):
        delattr(c, name)
    assert getattr(c, name) is before


@pytest.mark.parametrize("name", ARRAYS)
@pytest.mark.parametrize("how", ["resize", "set", "data"])
def test_arrays_moved_in_place_are_refused(name, how):
    c = make()
    assert awq._kv4(c, -1) is c._ref
    t = getattr(c, name)
    if how == "resize":
        t.resize_(1 << 20)
    elif how == "set":
        t.set_(torch.zeros_like(t))
    else:
        t.data = torch.zeros_like(t)
    with pytest.raises(ValueError, match="moved"):
        awq._kv4(c, -1)


@pytest.mark.gpu
def test_calls_refuse_moved_arrays():
    c = make("cuda")
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    calls = (lambda: awq.awq_kv4_append(k, k, c, i - 1), lambda: awq.awq_kv4_gather(c, i),
             lambda: awq.awq_kv4_attention(k, c, i[:, None], i))
    for call in calls:
        call()
    kept = c.v_codes.clone()
    c.v_codes.data = kept
    for call in calls:
        with pytest.raises(ValueError, match="moved"):
            call()
    again = awq.Kv4Cache(c.k_codes, c.v_codes, c.k_params, c.v_params)
    awq.awq_kv4_gather(again, i)
