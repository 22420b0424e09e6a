"""Sizes at the limits of 32-bit numbers, refused on the host before any launch
(no GPU needed): every call here passes addresses that nothing may read."""
import pytest

from tests.test_step_host import attn, rope

MOST = (1 << 31) - 1


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("capacity", [MOST, MOST - 64, MOST - 65, MOST - 127, MOST - 128, MOST - 511])
def test_table_capacity(D, capacity):
    """Tiles have up to 128 tokens and loads run two tiles ahead of the last one."""
    assert attn(D=D, qs=4 * D, ps=1, max_pages=capacity) == -2


@pytest.mark.parametrize("M", [1 << 24, (1 << 24) + 1, 1 << 29, MOST])
def test_rows_of_the_norm(M):
    """A workgroup of 256 threads for each row, in 32 bits."""
    assert rope(M=M) == -2
