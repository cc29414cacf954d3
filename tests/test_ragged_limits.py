"""Sizes at the ends of their ranges, on the host: what the kernels' 32-bit
indexes cannot hold is refused before anything is enqueued."""
import pytest

from mixture_experts_ffn_align_amd import _binding as B
from tests.test_ragged_abi import desc, dgrad, fp4, fwd, wgrad

INT32_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("rows", [INT32_MAX, INT32_MAX - 254])
@pytest.mark.parametrize("call", [fwd, dgrad, wgrad, fp4], ids=lambda c: c.__name__)
def test_rows_that_overflow_a_tile_count_are_refused(call, rows):
    # An expert may own all rows, and its tiles of up to 256 rows are counted as
    # (rows + 255) / 256. A null pointer keeps a call that is not refused for its
    # rows from launching anything.
    d = desc(rows=rows, E=1, N=32, K=32, dtype=B.MOE_DTYPE_MXFP4 if call is fp4 else B.MOE_DTYPE_BF16)
    assert call(d, off=None) == B.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("call", [fwd, dgrad, wgrad, fp4], ids=lambda c: c.__name__)
def test_the_most_rows_pass_the_shape_checks(call):
    d = desc(rows=INT32_MAX - 255, E=1, N=32, K=32, dtype=B.MOE_DTYPE_MXFP4 if call is fp4 else B.MOE_DTYPE_BF16)
    assert call(d, off=None) == B.MOE_ERR_INVALID_ARG      # for the null offsets
