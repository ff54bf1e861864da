"""Host-side limits of the microscaled 4-bit and 8-bit KV cache entry points
(no GPU needed)."""
import pytest
import torch

import weight_only_int4_quantize_b200 as w4
from tests.test_lowp_host import A, B, lib  # noqa: F401


@pytest.mark.parametrize("big", [(1 << 31) - 1, (1 << 31) - 257, (1 << 31) - 300, (1 << 31) - 383])
def test_linear_sizes_that_overflow_the_tile_arithmetic(lib, big):  # noqa: F811
    """A tile of 384 tokens reaches past the last one, and the rows that it
    counts there have to be 32-bit numbers."""
    assert lib.w4_fp4_linear(A, A, None, big, A, A, None, 8, 128, 0, B, 0, None) == 2


def test_values_without_a_truth_value(lib):  # noqa: F811
    """The error of asking for it reaches the caller before anything runs."""
    with pytest.raises(RuntimeError, match="ambiguous"):
        w4.fp4_quantize(torch.zeros(1, 128, dtype=torch.bfloat16), "mx", values=torch.ones(2))
