"""Host-side limits of the microscaled 4-bit and 8-bit KV cache entry points
(no GPU needed)."""
import ctypes

import pytest

import weight_only_int4_quantize_b200 as w4
from tests.test_lowp_host import A, B, _cache, lib  # noqa: F401


@pytest.mark.parametrize("big", [(1 << 31) - 1, (1 << 31) - 257, (1 << 31) - 300, (1 << 31) - 383])
def test_linear_sizes_that_overflow_the_tile_arithmetic(lib, big):  # noqa: F811
    """A tile of 384 tokens reaches past the last one, and the rows that it
    counts there have to be 32-bit numbers."""
    assert lib.w4_fp4_linear(A, A, None, big, A, A, None, 8, 128, 0, B, 0, None) == 2
