"""Sizes at the ends of their ranges, on the host: what the kernels' 32-bit
indexes cannot hold is refused before anything is enqueued."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
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


class Shape:
    """Stands for a GPU tensor of which only the checks' view is needed: no
    memory is behind it, and nothing is called with it."""

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.is_cuda, self.device = dtype, torch.Size(shape), True, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[-1], 1)

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def calls(monkeypatch):
    """Calls that pass the binding's checks are noted instead of made."""
    made = []
    monkeypatch.setattr(B, "_call_on", lambda device, stream, fn, *args: made.append(args) or B.MOE_OK)
    return made


PAST = 2 ** 32 + 32         # 32 in a 32-bit integer
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


@pytest.mark.parametrize("name,call", [
    ("rows", lambda n: moe.moe_grouped_matmul(Shape(BF, n, 32), Shape(BF, 2, 16, 32), Shape(I32, 3), Shape(BF, n, 16))),
    ("N", lambda n: moe.moe_grouped_matmul(Shape(BF, 4, 32), Shape(BF, 2, n, 32), Shape(I32, 3), Shape(BF, 4, n))),
    ("K", lambda n: moe.moe_grouped_matmul(Shape(BF, 4, n), Shape(BF, 2, 16, n), Shape(I32, 3), Shape(BF, 4, 16))),
    ("E", lambda n: moe.moe_grouped_matmul(Shape(BF, 4, 32), Shape(BF, n, 16, 32), Shape(I32, n + 1),
                                           Shape(BF, 4, 16))),
    ("rows", lambda n: moe.moe_grouped_matmul_dx(Shape(BF, n, 16), Shape(BF, 2, 16, 32), Shape(I32, 3),
                                                 Shape(BF, n, 32))),
    ("rows", lambda n: moe.moe_grouped_matmul_dw(Shape(BF, n, 16), Shape(BF, n, 32), Shape(I32, 3),
                                                 Shape(BF, 2, 16, 32))),
    ("rows", lambda n: moe.moe_grouped_matmul_mxfp4(Shape(U8, n, 16), Shape(U8, n, 1), Shape(U8, 2, 16, 16),
                                                    Shape(U8, 2, 16, 1), Shape(I32, 3), Shape(BF, n, 16))),
    ("K", lambda n: moe.moe_mxfp4_quantize(Shape(BF, 4, n), Shape(U8, 4, n // 2), Shape(U8, 4, n // 32))),
    ("K", lambda n: moe.moe_mxfp4_dequantize(Shape(U8, 4, n // 2), Shape(U8, 4, n // 32), Shape(BF, 4, n))),
    ("E", lambda n: moe.moe_align_offsets(Shape(I32, 8), Shape(I32, 1), n, 1, Shape(I32, n + 1))),
    ("b", lambda n: moe.moe_align_offsets(Shape(I32, 8), Shape(I32, 1), 2, n, Shape(I32, 3))),
])
def test_binding_refuses_sizes_past_32_bits(calls, name, call):
    # The C ABI's sizes are int32, and ctypes drops what does not fit.
    call(32)
    assert len(calls) == 1
    with pytest.raises(ValueError, match=f"^{name}: "):
        call(PAST)
    assert len(calls) == 1


@pytest.mark.gpu
def test_the_most_rows_of_one_expert():
    # 2^31 - 256 rows of eight elements (34 GB), all of one expert: forward and input gradient.
    rows, N, K = INT32_MAX - 255, 8, 8
    print("[gpu-case] ragged most rows", flush=True)
    w = torch.arange(N * K, dtype=torch.float32).view(1, N, K) % 7
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    x = torch.ones(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-300:] = 2.0
    y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    for call, ref in ((moe.moe_grouped_matmul, w[0].sum(1)), (moe.moe_grouped_matmul_dx, w[0].sum(0))):
        y.zero_()
        call(x, w.cuda().bfloat16(), off, y)
        ref = ref.cuda().bfloat16()
        for r in range(0, rows, 1 << 28):
            assert bool((y[r:min(rows - 300, r + (1 << 28))] == ref).all())
        assert bool((y[-300:] == 2 * ref).all())
