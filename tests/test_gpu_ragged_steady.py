"""The ragged products where their kernels run in the steady state: summed
extents of many slabs (the ring's slots are filled again and again), whole tiles
with several tasks to a workgroup (a task's first waits count the stores of the
one before), for every tile shape, operand form and output width, exact on whole
numbers; and the columns between an output's row ends, which stay as they were.

MXFP4 exponents vary by expert and block over their whole range, those of w
against those of x, so that a block's codes or exponents taken from another
slab, slot or expert show; products stay multiples of 2^-4 up to 144, exact in
fp32 for sums of up to 7281 of them."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _ragged as R
from tests.test_gpu_mxfp4 import off_by
from tests.test_gpu_ragged import SENTINEL, announce, rows_on_gpu

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class Out:
    """Output rows with a row stride; everything but the rows' columns is checked to stay."""

    def __init__(self, rows, cols, dtype, pad):
        self.all = torch.full((rows, cols + pad), SENTINEL, dtype=dtype, device="cuda")
        self.t = self.all[:, :cols]

    def check(self, ref, keep):
        torch.cuda.synchronize()
        got, cols = self.all.cpu(), self.t.shape[1]
        assert torch.equal(got[keep, :cols].double(), ref[keep].to(got.dtype).double())
        assert bool((got[~keep] == SENTINEL).all()) and bool((got[:, cols:] == SENTINEL).all())


def case_id(v):
    return R.shape_id(v) if isinstance(v, dict) else str(v).replace("torch.", "")


def shapes(*specs):
    return [dict(counts=c, N=N, K=K, **more) for c, N, K, more in specs]


WHOLE = [1024, 2048]      # whole 128-row tiles
FEW = [1, 2, 0, 1]
MANY = [(3 * e) % 9 for e in range(40)]

# Forward: 256 x 256 tiles; 128 x 128; 64 x 64 with a shared summed index; few rows by 16 and 32 columns.
FORWARD = shapes(([8192, 8192], 2048, 320, {}), ([8192, 8192], 2048, 384, {}), ([8192, 8192], 2048, 1544, {}),
                 ([9000, 7500, 33], 2056, 584, dict(head=2, tail=7)),
                 (WHOLE, 4096, 456, {}), (WHOLE, 4096, 192, dict(tail=1)), ([700, 20, 0, 333, 901], 2056, 712, dict(head=5)),
                 ([100, 30], 72, 2568, {}), (FEW, 2048, 2056, {}), (FEW, 2048, 1544, dict(tail=2)), (MANY, 2048, 2056, {}))


@pytest.mark.parametrize("out", [None, F32], ids=["same", "fp32"])
@pytest.mark.parametrize("dtype", [BF, F16], ids=case_id)
@pytest.mark.parametrize("s", FORWARD, ids=case_id)
def test_forward(s, dtype, out):
    g = torch.Generator().manual_seed(21)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    N, K = s["N"], s["K"]
    x, w = R.whole(g, rows, K), R.whole(g, len(s["counts"]), N, K)
    announce("steady forward", R.shape_id(s), dtype, out)
    y = Out(rows, N, out or dtype, 8)
    moe.moe_grouped_matmul(rows_on_gpu(x, dtype, keep, 16), w.cuda().to(dtype), off.cuda(), y.t)
    y.check(R.forward(x, w, off), keep)


# Input gradient: 128 x 128 tiles; 64 x 64.
DX = shapes((WHOLE, 456, 4096, {}), (WHOLE, 192, 4096, {}), ([700, 20, 0, 333, 901], 712, 2056, dict(head=5, tail=3)),
            ([1300, 700], 2568, 136, dict(tail=1)), ([100, 30], 2568, 72, {}))


@pytest.mark.parametrize("out", [None, F32], ids=["same", "fp32"])
@pytest.mark.parametrize("dtype", [BF, F16], ids=case_id)
@pytest.mark.parametrize("s", DX, ids=case_id)
def test_input_gradient(s, dtype, out):
    g = torch.Generator().manual_seed(22)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    N, K = s["N"], s["K"]
    dy, w = R.whole(g, rows, N), R.whole(g, len(s["counts"]), N, K)
    announce("steady input gradient", R.shape_id(s), dtype, out)
    dx = Out(rows, K, out or dtype, 24)
    moe.moe_grouped_matmul_dx(rows_on_gpu(dy, dtype, keep, 8), w.cuda().to(dtype), off.cuda(), dx.t)
    dx.check(R.input_grad(dy, w, off), keep)


# Weight gradient: 128 x 128 tiles, whole ones and others; 64 x 64.
DW = shapes(([500, 700], 4096, 4096, dict(tail=3)), ([0, 449, 64, 320, 1], 2056, 2120, dict(head=1)),
            ([1300, 700], 72, 136, {}), ([1300, 0, 641], 200, 264, dict(tail=1)))


@pytest.mark.parametrize("out", [None, F32], ids=["same", "fp32"])
@pytest.mark.parametrize("dtype", [BF, F16], ids=case_id)
@pytest.mark.parametrize("s", DW, ids=case_id)
def test_weight_gradient(s, dtype, out):
    g = torch.Generator().manual_seed(23)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    E, N, K = len(s["counts"]), s["N"], s["K"]
    dy, x = R.whole(g, rows, N), R.whole(g, rows, K)
    announce("steady weight gradient", R.shape_id(s), dtype, out)
    dw = torch.full((E, N, K), float("nan"), dtype=out or dtype, device="cuda")
    moe.moe_grouped_matmul_dw(rows_on_gpu(dy, dtype, keep, 8), rows_on_gpu(x, dtype, keep, 16), off.cuda(), dw)
    torch.cuda.synchronize()
    assert torch.equal(dw.cpu().double(), R.weight_grad(dy, x, off).to(dw.dtype).double())


def opposed_codes(g, off, rows, N, K):
    """Random codes; x's exponents are 2^(d + {-1, 0, 1}) and w's 2^(-d + {-1, 0, 1}), d by expert and block."""
    E, blocks = off.numel() - 1, K // 32
    d = torch.randint(-126, 127, (E, blocks), generator=g)
    xq = torch.randint(0, 256, (rows, K // 2), generator=g).to(torch.uint8)
    wq = torch.randint(0, 256, (E, N, K // 2), generator=g).to(torch.uint8)
    xs = torch.full((rows, blocks), 255, dtype=torch.int64)          # rows no expert owns decode to NaN
    a, b = int(off[0]), int(off[-1])
    of = torch.repeat_interleave(torch.arange(E), (off[1:] - off[:-1]).long())
    xs[a:b] = 127 + d[of] + torch.randint(-1, 2, (b - a, blocks), generator=g)
    ws = 127 - d.unsqueeze(1) + torch.randint(-1, 2, (E, N, blocks), generator=g)
    return xq, xs.to(torch.uint8), wq, ws.to(torch.uint8)


# 128 x 128 tiles with exponents by words (K a multiple of 128) and by bytes; 64 x 64 and 64 x 32 with a
# shared summed index; few rows (two blocks in flight, and several turns).
UNEVEN = [700, 0, 333, 901]
MXFP4 = (shapes(*((UNEVEN, 2056, K, dict(tail=2)) for K in (1152, 1184, 2048, 2080)))
         + shapes(*((WHOLE, 4096, K, {}) for K in (256, 288, 2048, 2080)))
         + shapes(*(([100, 30], 72, K, dict(head=3)) for K in (5120, 5632, 5152, 7200)))
         + shapes(*((FEW, 2048, K, dict(tail=1)) for K in (2080, 4096, 4128, 6176))))


@pytest.mark.parametrize("out", [F32, BF, F16], ids=case_id)
@pytest.mark.parametrize("s", MXFP4, ids=case_id)
def test_mxfp4_product(s, out):
    g = torch.Generator().manual_seed(24)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    xq, xs, wq, ws = opposed_codes(g, off, rows, s["N"], s["K"])
    announce("steady mxfp4", R.shape_id(s), out)
    y = Out(rows, s["N"], out, 8)
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), y.t)
    y.check(R.forward(torch.nan_to_num(R.codes_to_values(xq, xs)), R.codes_to_values(wq, ws), off), keep)


@pytest.mark.parametrize("x_at,w_at", [(1, 3), (0, 2), (2, 0)])
@pytest.mark.parametrize("s", shapes((UNEVEN, 2056, 2048, {}), ([100, 30], 72, 5120, {}), (FEW, 2048, 4096, {})),
                         ids=case_id)
def test_mxfp4_product_with_exponents_at_odd_addresses(s, x_at, w_at):
    g = torch.Generator().manual_seed(25)
    off, rows = R.offsets_of(s)
    xq, xs, wq, ws = opposed_codes(g, off, rows, s["N"], s["K"])
    announce("steady mxfp4 odd addresses", R.shape_id(s), x_at, w_at)
    y = Out(rows, s["N"], F32, 8)
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), off_by(xs, x_at), wq.cuda(), off_by(ws, w_at), off.cuda(), y.t)
    y.check(R.forward(R.codes_to_values(xq, xs), R.codes_to_values(wq, ws), off), R.owned(off, rows))


@pytest.mark.parametrize("s", shapes((UNEVEN, 2056, 1184, {}), (UNEVEN, 2056, 1152, {}), ([100, 30], 72, 5120, {}),
                                     (FEW, 2048, 2080, {})), ids=case_id)
def test_mxfp4_zeros_under_the_largest_exponents(s):
    # Zero codes are zeros whatever their exponent, also where the two exponents' product is past fp32's
    # range: half of each row's blocks are zeros under 2^127 on both sides.
    g = torch.Generator().manual_seed(26)
    off, rows = R.offsets_of(s)
    xq, xs, wq, ws = opposed_codes(g, off, rows, s["N"], s["K"])
    zero = torch.rand(s["K"] // 32, generator=g) < 0.5
    lanes = zero.repeat_interleave(16)
    xq[..., lanes], wq[..., lanes] = 0, 0
    xs[..., zero], ws[..., zero] = 254, 254
    announce("steady mxfp4 zeros", R.shape_id(s))
    y = Out(rows, s["N"], F32, 8)
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), y.t)
    y.check(R.forward(R.codes_to_values(xq, xs), R.codes_to_values(wq, ws), off), R.owned(off, rows))


@pytest.mark.parametrize("out", [BF, F32], ids=case_id)
@pytest.mark.parametrize("s", R.SHAPES, ids=case_id)
def test_columns_between_rows_stay(s, out):
    # The smaller shapes: column counts that end inside every group of columns.
    g = torch.Generator().manual_seed(27)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    E, N, K = len(s["counts"]), s["N"], s["K"]
    x, dy, w = R.whole(g, rows, K), R.whole(g, rows, N), R.whole(g, E, N, K)
    announce("columns between rows", R.shape_id(s), out)
    wd, offd = w.cuda().to(BF), off.cuda()
    y, dx = Out(rows, N, out, 40), Out(rows, K, out, 40)
    moe.moe_grouped_matmul(rows_on_gpu(x, BF, keep), wd, offd, y.t)
    moe.moe_grouped_matmul_dx(rows_on_gpu(dy, BF, keep), wd, offd, dx.t)
    y.check(R.forward(x, w, off), keep)
    dx.check(R.input_grad(dy, w, off), keep)
    xq, xs, wq, ws = opposed_codes(g, off, rows, N, -(-K // 32) * 32)
    y = Out(rows, N, out, 40)
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), offd, y.t)
    y.check(R.forward(torch.nan_to_num(R.codes_to_values(xq, xs)), R.codes_to_values(wq, ws), off), keep)


@pytest.mark.parametrize("s", shapes((UNEVEN, 2056, 1184, {}), (UNEVEN, 2056, 1152, {}), ([100, 30], 72, 5120, {}),
                                     (FEW, 2048, 2080, {})), ids=case_id)
def test_mxfp4_sums_of_blocks_of_very_different_size(s):
    # Exponents of x and w without regard to each other: blocks of one sum differ by up to 2^100.
    g = torch.Generator().manual_seed(28)
    off, rows = R.offsets_of(s)
    N, K = s["N"], s["K"]
    xq, _, wq, _ = opposed_codes(g, off, rows, N, K)
    xs = torch.randint(102, 153, (rows, K // 32), generator=g).to(torch.uint8)
    ws = torch.randint(102, 153, (len(s["counts"]), N, K // 32), generator=g).to(torch.uint8)
    announce("steady mxfp4 sizes", R.shape_id(s))
    y = Out(rows, N, F32, 0)
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), y.t)
    torch.cuda.synchronize()
    xv, wv = R.codes_to_values(xq, xs), R.codes_to_values(wq, ws)
    ref, size = R.forward(xv, wv, off), R.forward(xv.abs(), wv.abs(), off)
    assert bool(((y.t.double().cpu() - ref).abs() <= R.tolerance(ref, size, K, F32)).all())


@pytest.mark.parametrize("dtype", [BF, F16], ids=case_id)
def test_sums_of_terms_of_very_different_size(dtype):
    # bf16 over 2^80, fp16 over its ordinary range.
    g = torch.Generator().manual_seed(29)
    s = dict(counts=[300, 20, 500], N=520, K=712)
    off, rows = R.offsets_of(s)
    E, N, K = 3, s["N"], s["K"]
    top = 20 if dtype == BF else 3

    def wide(*shape):
        return (torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-top, top + 1, shape, generator=g).float())
                ).to(dtype).double()

    x, dy, w = wide(rows, K), wide(rows, N), wide(E, N, K)
    announce("steady sizes", dtype)
    xd, dyd, wd, offd = x.cuda().to(dtype), dy.cuda().to(dtype), w.cuda().to(dtype), off.cuda()
    y, dx, dw = Out(rows, N, F32, 0), Out(rows, K, F32, 0), torch.empty(E, N, K, device="cuda")
    moe.moe_grouped_matmul(xd, wd, offd, y.t)
    moe.moe_grouped_matmul_dx(dyd, wd, offd, dx.t)
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    torch.cuda.synchronize()
    for got, ref, size, terms in (
            (y.t, R.forward(x, w, off), R.forward(x.abs(), w.abs(), off), K),
            (dx.t, R.input_grad(dy, w, off), R.input_grad(dy.abs(), w.abs(), off), N),
            (dw, R.weight_grad(dy, x, off), R.weight_grad(dy.abs(), x.abs(), off), 500)):
        assert bool(((got.double().cpu() - ref).abs() <= R.tolerance(ref, size, terms, F32)).all())
