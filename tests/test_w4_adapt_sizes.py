"""The adapted product's workspace: its size is asked for without knowing whether low will be kept."""
import pytest

from post_bit_weight_awq_amd import _lib


@pytest.mark.parametrize("n", [1, 16, 48, 64, 65, 300, 4096])
@pytest.mark.parametrize("dtype,y", [(0, 0), (0, 2), (1, 1), (1, 2)])
def test_the_size_is_the_same_with_low_kept(n, dtype, y):
    size = lambda keep: _lib.load().awq_w4a16_adapted_workspace_size(n, 1024, 640, 64, dtype, y, 4, 24, keep)
    assert size(0) == size(1) == size(7) < 1 << 34
