"""Sizes at the ends of their ranges, on the host: what the kernels' 32-bit
indexes cannot hold is refused before anything is enqueued."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from mixture_experts_ffn_align_amd import _binding as B
from tests import _ragged as R
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


def exact_products(off, E, N, K, seed, dx_too=True, ld=None):
    """Forward and input gradient on small whole numbers against 64-bit sums; `ld`: row stride of x and dx."""
    g = torch.Generator().manual_seed(seed)
    rows = int(off[-1])
    x, dy, w = R.whole(g, rows, K, top=2), R.whole(g, rows, N, top=2), R.whole(g, E, N, K, top=2)
    xd = x.cuda().bfloat16() if ld is None else torch.empty(rows, ld, dtype=BF, device="cuda")[:, :K].copy_(x)
    dyd, wd, offd = dy.cuda().bfloat16(), w.cuda().bfloat16(), off.cuda()
    y = torch.empty(rows, N, device="cuda")
    moe.moe_grouped_matmul(xd, wd, offd, y)
    assert torch.equal(y.double().cpu(), R.forward(x, w, off))
    if dx_too:
        dx = torch.empty(rows, ld or K, device="cuda")[:, :K]
        moe.moe_grouped_matmul_dx(dyd, wd, offd, dx)
        assert torch.equal(dx.double().cpu(), R.input_grad(dy, w, off))
    return x, dy, xd, dyd, offd


def offsets_from(counts):
    return torch.cat((torch.zeros(1, dtype=torch.int64), torch.tensor(counts).cumsum(0))).to(torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[2, 1], [90, 40]], ids=str)     # few rows; tiles
def test_the_widest_rows(counts):
    # K of 2^20 with rows 2^22 elements apart; then N of 2^20. Sums of 2^20 products of at most 4 are exact.
    print("[gpu-case] ragged widest rows", counts, flush=True)
    off, top = offsets_from(counts), 1 << 20
    x, dy, xd, dyd, offd = exact_products(off, 2, 8, top, 41, ld=1 << 22)
    dw = torch.empty(2, 8, top, device="cuda")
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    assert torch.equal(dw.double().cpu(), R.weight_grad(dy, x, off))
    exact_products(off, 2, top, 8, 42)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[2, 1], [90, 40]], ids=str)
def test_the_widest_mxfp4_rows(counts):
    print("[gpu-case] mxfp4 widest rows", counts, flush=True)
    off, K = offsets_from(counts), 1 << 20
    rows = int(off[-1])
    g = torch.Generator().manual_seed(43)
    # Codes 0 to 3 with a sign (up to 1.5) under exponents 0: quarter steps, sums below 2^22.
    xq, wq = (torch.randint(0, 256, (*n, K // 2), generator=g).to(torch.uint8) & 0xBB for n in ((rows,), (2, 8)))
    xs, ws = (torch.full((*n, K // 32), 127, dtype=torch.uint8) for n in ((rows,), (2, 8)))
    y = torch.empty(rows, 8, device="cuda")
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), y)
    assert torch.equal(y.double().cpu(), R.forward(R.codes_to_values(xq, xs), R.codes_to_values(wq, ws), off))


@pytest.mark.gpu
@pytest.mark.parametrize("most,N,K", [(1, 24, 40), (21, 136, 72), (1030, 16, 8)], ids=str)
def test_the_most_experts(most, N, K):
    # 2048 experts' start rows beside every tile shape's slabs: few rows, 128 x 128 and 256 x 256 tiles.
    print("[gpu-case] ragged most experts", most, N, K, flush=True)
    counts = [(7 * e) % (most + 1) if most < 1000 else 512 + (3 * e) % (most - 511) for e in range(2048)]
    off = offsets_from(counts)
    x, dy, xd, dyd, offd = exact_products(off, 2048, N, K, 44)
    dw = torch.empty(2048, N, K, device="cuda")
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    assert torch.equal(dw.double().cpu(), R.weight_grad(dy, x, off))


@pytest.mark.gpu
@pytest.mark.parametrize("K", [128, 160])
@pytest.mark.parametrize("rows,N", [(300, 24), (20000, 72)])
def test_the_most_experts_in_mxfp4(rows, N, K):
    # 300 rows take the tiles with a shared summed index, whose rings and 2049 start rows are the most LDS of all.
    print("[gpu-case] mxfp4 most experts", rows, N, K, flush=True)
    g = torch.Generator().manual_seed(45)
    off = torch.cat((torch.zeros(1, dtype=torch.int64), torch.randint(0, rows + 1, (2047,), generator=g).sort().values,
                     torch.tensor([rows]))).to(torch.int32)
    xq, wq = (torch.randint(0, 256, (*n, K // 2), generator=g).to(torch.uint8) for n in ((rows,), (2048, N)))
    xs, ws = (torch.randint(126, 129, (*n, K // 32), generator=g).to(torch.uint8) for n in ((rows,), (2048, N)))
    y = torch.empty(rows, N, device="cuda")
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), y)
    assert torch.equal(y.double().cpu(), R.forward(R.codes_to_values(xq, xs), R.codes_to_values(wq, ws), off))


@pytest.mark.gpu
def test_offsets_of_no_blocks_and_of_any_count():
    print("[gpu-case] offsets of no blocks", flush=True)
    i32 = dict(dtype=torch.int32, device="cuda")
    off = torch.full((2049,), -5, **i32)
    moe.moe_align_offsets(torch.empty(0, **i32), torch.zeros(1, **i32), 2048, 16, off)
    assert not bool(off.any())
    blocks = torch.tensor([0, 0, 2, 2, 2, -1, -1], **i32)
    for padded, ref in ((20, [0, 8, 8, 20]), (9, [0, 8, 8, 8]), (-7, [0, 0, 0, 0]), (12, [0, 8, 8, 12])):
        off = torch.full((4,), -5, **i32)
        moe.moe_align_offsets(blocks, torch.full((1,), padded, **i32), 3, 4, off)
        assert off.tolist() == ref
