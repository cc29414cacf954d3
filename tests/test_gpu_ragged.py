"""The products on ragged rows (moe_grouped_matmul, _dx, _dw) against 64-bit
references: exact on whole numbers, within the bound of fp32 sums on random
ones; rows no expert owns, strides, streams, graphs, odd offsets."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _ragged as R

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]
SENTINEL = 77.0


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


def rows_on_gpu(v, dtype, keep=None, pad=0):
    """fp64 rows on the GPU, optionally with a row stride; rows outside `keep` hold NaN."""
    v = v.clone()
    if keep is not None:
        v[~keep] = float("nan")
    if pad:
        wide = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=torch.float64)
        wide[:, :v.shape[1]] = v
        return wide.to("cuda").to(dtype)[:, :v.shape[1]]
    return v.to("cuda").to(dtype)


def out_rows(rows, cols, dtype, pad=0):
    return torch.full((rows, cols + pad), SENTINEL, dtype=dtype, device="cuda")[:, :cols]


def check_rows(y, ref, keep):
    y = y.double().cpu()
    assert torch.equal(y[keep], ref[keep].to(torch.float64))
    assert bool((y[~keep] == SENTINEL).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("s", R.SHAPES, ids=R.shape_id)
@pytest.mark.parametrize("wide", [False, True])
def test_products_are_exact_on_whole_numbers(s, dtype, wide):
    g = torch.Generator().manual_seed(1)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    E, N, K = len(s["counts"]), s["N"], s["K"]
    x, dy, w = R.whole(g, rows, K), R.whole(g, rows, N), R.whole(g, E, N, K)
    out = torch.float32 if wide else dtype
    pad = 8 if wide else 0
    announce("ragged", R.shape_id(s), dtype, wide)
    xd, dyd = rows_on_gpu(x, dtype, keep, pad), rows_on_gpu(dy, dtype, keep, 2 * pad)
    wd, offd = w.cuda().to(dtype), off.cuda()
    y, dx = out_rows(rows, N, out, pad), out_rows(rows, K, out, 3 * pad)
    dw = torch.full((E, N, K), float("nan"), dtype=out, device="cuda")
    moe.moe_grouped_matmul(xd, wd, offd, y)
    moe.moe_grouped_matmul_dx(dyd, wd, offd, dx)
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    torch.cuda.synchronize()
    check_rows(y, R.forward(x, w, off).to(out), keep)
    check_rows(dx, R.input_grad(dy, w, off).to(out), keep)
    assert torch.equal(dw.cpu().double(), R.weight_grad(dy, x, off).to(out).double())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("s", R.LARGE, ids=R.shape_id)
def test_large_tiles_are_exact_on_whole_numbers(s, dtype):
    g = torch.Generator().manual_seed(12)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    E, N, K = len(s["counts"]), s["N"], s["K"]
    x, dy, w = R.whole(g, rows, K), R.whole(g, rows, N), R.whole(g, E, N, K)
    announce("ragged large", R.shape_id(s), dtype)
    xd, dyd = rows_on_gpu(x, dtype, keep, 8), rows_on_gpu(dy, dtype, keep)
    wd, offd = w.cuda().to(dtype), off.cuda()
    y, dx = out_rows(rows, N, torch.float32), out_rows(rows, K, dtype, 8)
    dw = torch.full((E, N, K), float("nan"), dtype=torch.float32, device="cuda")
    moe.moe_grouped_matmul(xd, wd, offd, y)
    moe.moe_grouped_matmul_dx(dyd, wd, offd, dx)
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    torch.cuda.synchronize()
    check_rows(y, R.forward(x, w, off), keep)
    check_rows(dx, R.input_grad(dy, w, off).to(dtype), keep)
    assert torch.equal(dw.cpu().double(), R.weight_grad(dy, x, off))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("s", R.TALL, ids=R.shape_id)
def test_tall_tiles_are_exact_on_whole_numbers(s, dtype):
    g = torch.Generator().manual_seed(13)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    E, N, K = len(s["counts"]), s["N"], s["K"]
    x, w = R.whole(g, rows, K), R.whole(g, E, N, K)
    announce("ragged tall", R.shape_id(s), dtype)
    y = out_rows(rows, N, dtype)
    moe.moe_grouped_matmul(rows_on_gpu(x, dtype, keep), w.cuda().to(dtype), off.cuda(), y)
    torch.cuda.synchronize()
    check_rows(y, R.forward(x, w, off).to(dtype), keep)


def test_two_streams_at_once():
    # Calls share nothing: two of them overlapping on two streams give what each gives alone.
    g = torch.Generator().manual_seed(14)
    jobs = []
    for counts, N, K in (([300, 700], 1032, 520), ([5, 0, 90], 2048, 264)):
        s = dict(counts=counts, N=N, K=K)
        off, rows = R.offsets_of(s)
        x, w = R.whole(g, rows, K), R.whole(g, len(counts), N, K)
        jobs.append((x.cuda().bfloat16(), w.cuda().bfloat16(), off.cuda(), torch.zeros(rows, N, device="cuda"),
                     R.forward(x, w, off), torch.cuda.Stream()))
    announce("ragged two streams")
    torch.cuda.synchronize()
    for _ in range(5):
        for x, w, off, y, _, stream in jobs:
            moe.moe_grouped_matmul(x, w, off, y, stream=stream)
    torch.cuda.synchronize()
    for _, _, _, y, ref, _ in jobs:
        assert torch.equal(y.double().cpu(), ref)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("out", [torch.float32, None], ids=str)
@pytest.mark.parametrize("s", [R.SHAPES[i] for i in (3, 5, 8, 9, 10)], ids=R.shape_id)
def test_products_on_random_values(s, dtype, out):
    out = dtype if out is None else out
    g = torch.Generator().manual_seed(2)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    E, N, K = len(s["counts"]), s["N"], s["K"]
    x, dy, w = (torch.randn(*n, generator=g).to(dtype).double() for n in ((rows, K), (rows, N), (E, N, K)))
    announce("ragged random", R.shape_id(s), dtype, out)
    xd, dyd, wd, offd = x.cuda().to(dtype), dy.cuda().to(dtype), w.cuda().to(dtype), off.cuda()
    y, dx = out_rows(rows, N, out), out_rows(rows, K, out)
    dw = torch.empty(E, N, K, dtype=out, device="cuda")
    moe.moe_grouped_matmul(xd, wd, offd, y)
    moe.moe_grouped_matmul_dx(dyd, wd, offd, dx)
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    torch.cuda.synchronize()
    ref, size = R.forward(x, w, off), R.forward(x.abs(), w.abs(), off)
    assert bool(((y.double().cpu() - ref).abs() <= R.tolerance(ref, size, K, out))[keep].all())
    ref, size = R.input_grad(dy, w, off), R.input_grad(dy.abs(), w.abs(), off)
    assert bool(((dx.double().cpu() - ref).abs() <= R.tolerance(ref, size, N, out))[keep].all())
    ref, size = R.weight_grad(dy, x, off), R.weight_grad(dy.abs(), x.abs(), off)
    assert bool(((dw.double().cpu() - ref).abs() <= R.tolerance(ref, size, max(s["counts"]), out)).all())


def test_gradients_match_differences():
    # Loss = sum(y * c). It is linear in x and in w, so a difference over a whole
    # step is exact: (loss(x + u) - loss(x)) = <dx, u>, on whole numbers without rounding.
    s = dict(counts=[5, 0, 33, 20], N=40, K=56)
    g = torch.Generator().manual_seed(3)
    off, rows = R.offsets_of(s)
    E, N, K = 4, s["N"], s["K"]
    x, c, w = R.whole(g, rows, K), R.whole(g, rows, N), R.whole(g, E, N, K)
    ux, uw = R.whole(g, rows, K, top=1), R.whole(g, E, N, K, top=1)
    offd = off.cuda()
    dt = torch.bfloat16
    f32 = dict(dtype=torch.float32, device="cuda")

    def loss(xv, wv):
        y = torch.empty(rows, N, **f32)
        moe.moe_grouped_matmul(xv.cuda().to(dt), wv.cuda().to(dt), offd, y)
        return float((y.double().cpu() * c).sum())

    announce("ragged differences")
    dx, dw = torch.empty(rows, K, **f32), torch.empty(E, N, K, **f32)
    moe.moe_grouped_matmul_dx(c.cuda().to(dt), w.cuda().to(dt), offd, dx)
    moe.moe_grouped_matmul_dw(c.cuda().to(dt), x.cuda().to(dt), offd, dw)
    assert loss(x + ux, w) - loss(x, w) == float((dx.double().cpu() * ux).sum())
    assert loss(x, w + uw) - loss(x, w) == float((dw.double().cpu() * uw).sum())


@pytest.mark.parametrize("bad", [[0, 5, 3, 8, 8], [4, 2, 6, 1, 30], [-3, 2, 2, 9, 12], [50, 60, 70, 80, 90],
                                 [-9, -8, -7, -6, -5]], ids=str)
def test_offsets_out_of_order_or_range(bad):
    # Taken as clamped to [0, rows] and raised to the largest entry before: a
    # defined partition whatever the array holds.
    rows, E, N, K = 12, 4, 40, 72
    off, top = [], 0
    for o in bad:
        top = min(rows, max(top, o))
        off.append(top)
    off = torch.tensor(off, dtype=torch.int32)
    keep = R.owned(off, rows)
    g = torch.Generator().manual_seed(4)
    x, dy, w = R.whole(g, rows, K), R.whole(g, rows, N), R.whole(g, E, N, K)
    announce("ragged offsets", bad)
    offd = torch.tensor(bad, dtype=torch.int32).cuda()
    xd, dyd, wd = (t.cuda().to(torch.bfloat16) for t in (x, dy, w))
    y, dx = out_rows(rows, N, torch.float32), out_rows(rows, K, torch.float32)
    dw = torch.full((E, N, K), float("nan"), device="cuda")
    moe.moe_grouped_matmul(xd, wd, offd, y)
    moe.moe_grouped_matmul_dx(dyd, wd, offd, dx)
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    torch.cuda.synchronize()
    check_rows(y, R.forward(x, w, off), keep)
    check_rows(dx, R.input_grad(dy, w, off), keep)
    assert torch.equal(dw.cpu().double(), R.weight_grad(dy, x, off))


def test_no_rows():
    announce("ragged no rows")
    E, N, K = 3, 40, 136
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    w = torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda")
    x, dy = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (K, N))
    moe.moe_grouped_matmul(x, w, off, torch.empty(0, N, dtype=torch.bfloat16, device="cuda"))
    moe.moe_grouped_matmul_dx(dy, w, off, torch.empty(0, K, dtype=torch.bfloat16, device="cuda"))
    dw = torch.full((E, N, K), float("nan"), device="cuda")
    moe.moe_grouped_matmul_dw(dy, x, off, dw)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_infinities_and_nans_stay_in_their_rows(dtype):
    # A row's bad values reach that row's outputs (and its expert's weight
    # gradient), no other row's, also where an expert's rows end inside a tile.
    s = dict(counts=[5, 3, 40, 1], N=72, K=104)
    off, rows = R.offsets_of(s)
    g = torch.Generator().manual_seed(5)
    E, N, K = 4, s["N"], s["K"]
    x, dy, w = R.whole(g, rows, K), R.whole(g, rows, N), R.whole(g, E, N, K)
    x[5, 7], x[20, 3], dy[5, 9] = float("inf"), float("nan"), float("nan")
    announce("ragged bad values", dtype)
    xd, dyd, wd, offd = x.cuda().to(dtype), dy.cuda().to(dtype), w.cuda().to(dtype), off.cuda()
    y, dx = out_rows(rows, N, torch.float32), out_rows(rows, K, torch.float32)
    dw = torch.empty(E, N, K, device="cuda")
    moe.moe_grouped_matmul(xd, wd, offd, y)
    moe.moe_grouped_matmul_dx(dyd, wd, offd, dx)
    moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)
    torch.cuda.synchronize()
    y, dx, dw = y.double().cpu(), dx.double().cpu(), dw.double().cpu()
    assert torch.equal(torch.nan_to_num(y, nan=1e30), torch.nan_to_num(R.forward(x, w, off), nan=1e30))
    assert torch.equal(torch.nan_to_num(dx, nan=1e30), torch.nan_to_num(R.input_grad(dy, w, off), nan=1e30))
    assert torch.equal(torch.nan_to_num(dw, nan=1e30), torch.nan_to_num(R.weight_grad(dy, x, off), nan=1e30))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("counts", [[3, 2], [100, 61], [900, 800, 700]], ids=str)
def test_subnormal_inputs(dtype, counts):
    # The smallest subnormals times whole numbers, scaled so that every product is an ordinary fp32 value.
    unit = 2.0 ** -24 if dtype == torch.float16 else 2.0 ** -133
    scale = 1.0 if dtype == torch.float16 else 2.0 ** 60
    g = torch.Generator().manual_seed(16)
    off, rows = R.offsets_of(dict(counts=counts))
    E, N, K = len(counts), 2056, 72
    x, w = R.whole(g, rows, K) * unit, R.whole(g, E, N, K) * scale
    announce("ragged subnormals", dtype, counts)
    y = out_rows(rows, N, torch.float32)
    moe.moe_grouped_matmul(x.to(dtype).cuda(), w.to(dtype).cuda(), off.cuda(), y)
    torch.cuda.synchronize()
    assert torch.equal(y.double().cpu(), R.forward(x, w, off))


def test_another_stream_and_replayed_graph():
    s = dict(counts=[65, 0, 200, 7], N=136, K=136)
    off, rows = R.offsets_of(s)
    E, N, K = 4, s["N"], s["K"]
    g = torch.Generator().manual_seed(6)
    dt = torch.bfloat16
    announce("ragged graph")
    xd, dyd = (torch.empty(rows, n, dtype=dt, device="cuda") for n in (K, N))
    wd = R.whole(g, E, N, K).cuda().to(dt)
    offd = off.cuda()
    y, dx = out_rows(rows, N, torch.float32), out_rows(rows, K, torch.float32)
    dw = torch.empty(E, N, K, device="cuda")

    def step():
        moe.moe_grouped_matmul(xd, wd, offd, y)
        moe.moe_grouped_matmul_dx(dyd, wd, offd, dx)
        moe.moe_grouped_matmul_dw(dyd, xd, offd, dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x, dy = R.whole(g, rows, K), R.whole(g, rows, N)
        # the offsets are read on the device, so a replay follows new ones
        moved = off.clone()
        moved[1] += i
        moved[2] += i
        xd.copy_(x)
        dyd.copy_(dy)
        offd.copy_(moved)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.double().cpu(), R.forward(x, wd.double().cpu(), moved))
        assert torch.equal(dx.double().cpu(), R.input_grad(dy, wd.double().cpu(), moved))
        assert torch.equal(dw.double().cpu(), R.weight_grad(dy, x, moved))


def test_repeats_are_bitwise_equal():
    g = torch.Generator().manual_seed(7)
    s = dict(counts=[700, 20, 333], N=264, K=392)
    off, rows = R.offsets_of(s)
    E, N, K = 3, s["N"], s["K"]
    announce("ragged repeats")
    x, dy, w = (torch.randn(*n, generator=g).cuda().bfloat16() for n in ((rows, K), (rows, N), (E, N, K)))
    offd = off.cuda()
    first = None
    for _ in range(3):
        y, dx = torch.empty(rows, N, device="cuda"), torch.empty(rows, K, device="cuda")
        dw = torch.empty(E, N, K, device="cuda")
        moe.moe_grouped_matmul(x, w, offd, y)
        moe.moe_grouped_matmul_dx(dy, w, offd, dx)
        moe.moe_grouped_matmul_dw(dy, x, offd, dw)
        got = [t.cpu() for t in (y, dx, dw)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_indices_past_32_bits():
    # Operands and outputs of more than 2^31 elements: the work is at their far
    # end, the rest is zero or belongs to experts without rows.
    g = torch.Generator().manual_seed(17)
    bf = dict(dtype=torch.bfloat16, device="cuda")

    announce("ragged far rows of x")
    rows, K, N, few = 140000, 16384, 64, 50
    x = torch.zeros(rows, K, **bf)
    xs, w = R.whole(g, few, K, top=2), R.whole(g, 1, N, K, top=2)
    x[-few:] = xs.to("cuda").to(torch.bfloat16)
    y = torch.empty(rows, N, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32)
    moe.moe_grouped_matmul(x, w.cuda().to(torch.bfloat16), off.cuda(), y)
    assert torch.equal(y[-few:].double().cpu(), xs @ w[0].T) and bool((y[:-few] == 0).all())
    dw = torch.empty(1, N, K, device="cuda")
    dy = torch.zeros(rows, N, **bf)
    dys = R.whole(g, few, N, top=2)
    dy[-few:] = dys.to("cuda").to(torch.bfloat16)
    moe.moe_grouped_matmul_dw(dy, x, off.cuda(), dw)
    assert torch.equal(dw[0].double().cpu(), dys.T @ xs)
    del x, y, dw, dy

    announce("ragged far rows of y")
    rows, K, N = 300000, 8, 8192
    x = torch.ones(rows, K, **bf)
    w = R.whole(g, 1, N, K)
    y = torch.empty(rows, N, **bf)
    moe.moe_grouped_matmul(x, w.cuda().to(torch.bfloat16), torch.tensor([0, rows], dtype=torch.int32).cuda(), y)
    ref = w[0].sum(1).to("cuda").to(torch.bfloat16)
    assert bool((y[-1000:] == ref).all()) and bool((y[:1000] == ref).all())
    del x, y

    announce("ragged far experts")
    E, N, K, few = 70, 8192, 4096, 40
    w = torch.zeros(E, N, K, **bf)
    wl = R.whole(g, N, K, top=2)
    w[-1] = wl.to("cuda").to(torch.bfloat16)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[-1] = few
    x, dy = R.whole(g, few, K, top=2), R.whole(g, few, N, top=2)
    xd, dyd = x.cuda().to(torch.bfloat16), dy.cuda().to(torch.bfloat16)
    y, dx = torch.empty(few, N, device="cuda"), torch.empty(few, K, device="cuda")
    moe.moe_grouped_matmul(xd, w, off.cuda(), y)
    moe.moe_grouped_matmul_dx(dyd, w, off.cuda(), dx)
    assert torch.equal(y.double().cpu(), x @ wl.T) and torch.equal(dx.double().cpu(), dy @ wl)
    moe.moe_grouped_matmul_dw(dyd, xd, off.cuda(), w)
    assert torch.equal(w[-1].double().cpu(), (dy.T @ x).to(torch.bfloat16).double())
    assert not bool(w[:-1].any())
