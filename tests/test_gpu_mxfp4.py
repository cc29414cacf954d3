"""MXFP4: quantisation against its definition bit for bit, dequantisation
exact, the grouped product exact on values whose sums fp32 holds; the
alignment's row offsets; and the calls together as a serving step uses them."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _ragged as R
from tests.test_gpu_ragged import SENTINEL, announce, out_rows

pytestmark = pytest.mark.gpu

ALL = [torch.float32, torch.bfloat16, torch.float16]


def gpu_quantise(x):
    q = torch.full(x.shape[:-1] + (x.shape[-1] // 2,), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full(x.shape[:-1] + (x.shape[-1] // 32,), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_mxfp4_quantize(x, q, s)
    torch.cuda.synchronize()
    return q, s


def same_codes(x):
    q, s = gpu_quantise(x)
    rq, rs = R.quantise(x.double().cpu())
    return torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)


@pytest.mark.parametrize("dtype", ALL, ids=str)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (21, 2048), (70, 96), (1000, 160), (1, 4096)])
def test_quantise_matches_its_definition(rows, K, dtype):
    g = torch.Generator().manual_seed(rows)
    announce("mxfp4 quantise", rows, K, dtype)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, K // 32), generator=g).float()
                                                       ).repeat_interleave(32, 1)
    assert same_codes(x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_quantise_every_16_bit_value(dtype):
    # Every value leads a block of itself and its fractions; infinities and NaN among them.
    announce("mxfp4 every value", dtype)
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    x = v.repeat_interleave(32).view(65536, 32).clone()
    f = torch.tensor([1.0, -1.0, 0.5, 0.25, 0.125, 0.75, 0.375, 0.0625] * 4)
    x = (x.double() * f).to(dtype)
    assert same_codes(x.cuda())


def test_quantise_ties_and_extremes():
    announce("mxfp4 ties")
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.999, 0.0, -0.0, 4.0])
    near = torch.cat([ties, torch.nextafter(ties, torch.tensor(9.0)), torch.nextafter(ties, torch.tensor(-9.0))])
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -124, -20, 0, 20, 100, 124, 125):
        r = torch.zeros(64, dtype=torch.float64)
        r[:36] = near.double() * 2.0 ** e
        r[36:60] = -near[:24].double() * 2.0 ** e
        r[0] = r[32] = 4.0 * 2.0 ** e       # both blocks have the exponent e
        rows.append(r)
    assert same_codes(torch.stack(rows).float().cuda())
    big = torch.finfo(torch.float32).max
    odd = torch.zeros(6, 64)
    odd[0, 3], odd[1, 40], odd[2, 0], odd[3, 63], odd[4, :32] = float("inf"), float("nan"), big, -float("inf"), -0.0
    odd[5, 1] = 1e-45
    assert same_codes(odd.cuda())


def test_quantise_strides_and_leading_dimensions():
    announce("mxfp4 strides")
    g = torch.Generator().manual_seed(1)
    x = torch.randn(37, 200, generator=g).cuda().bfloat16()
    assert same_codes(x[:, :160])
    assert same_codes(x[:, 8:168])
    assert same_codes(torch.randn(3, 5, 96, generator=g).cuda())
    q, s = gpu_quantise(x[:0, :160])
    assert q.numel() == 0 and s.numel() == 0


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=str)
def test_dequantise_every_code_and_exponent(out):
    announce("mxfp4 dequantise", out)
    q = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 16, 16).expand(256, 16, 16).reshape(4096, 16)
    s = torch.arange(256, dtype=torch.int32).repeat_interleave(16).to(torch.uint8).view(4096, 1)
    y = torch.full((4096, 40), SENTINEL, dtype=out, device="cuda")
    moe.moe_mxfp4_dequantize(q.contiguous().cuda(), s.cuda(), y[:, :32])
    ref = R.codes_to_values(q, s).to(torch.float32).to(out)
    got = y.cpu()
    assert torch.equal(torch.nan_to_num(got[:, :32].float(), nan=1e30), torch.nan_to_num(ref.float(), nan=1e30))
    assert bool((got[:, 32:] == SENTINEL).all())


def codes(g, *shape, lo=126, hi=128):
    """Random codes and exponents: products are multiples of 2^-4 below 2^8, so fp32 sums of up to 2^12 are exact."""
    q = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), generator=g).to(torch.uint8)
    s = torch.randint(lo, hi + 1, shape[:-1] + (shape[-1] // 32,), generator=g).to(torch.uint8)
    return q, s


def product(xq, xs, wq, ws, off, out, pad=0):
    y = out_rows(xq.shape[0], wq.shape[1], out, pad)
    moe.moe_grouped_matmul_mxfp4(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), off.cuda(), y)
    torch.cuda.synchronize()
    return y.double().cpu()


@pytest.mark.parametrize("out", ALL, ids=str)
@pytest.mark.parametrize("s", [dict(s, K=-(-s["K"] // 32) * 32) for s in R.SHAPES]
                         + [dict(counts=[5, 40], N=40, K=k) for k in (96, 128, 160, 256, 288, 512, 544)]
                         + [dict(counts=[200, 300, 1], N=264, K=k) for k in (224, 256, 1056)]
                         + [dict(counts=[700, 0, 333, 901], N=2056, K=k, tail=2) for k in (96, 128, 384, 992, 1024)]
                         + [dict(counts=[1024, 2048], N=4096, K=k) for k in (160, 256)]
                         + [dict(counts=[1, 2, 0, 1], N=2048, K=k) for k in (32, 480, 512, 1056, 1024)],
                         ids=R.shape_id)
def test_product_is_exact(s, out):
    g = torch.Generator().manual_seed(8)
    off, rows = R.offsets_of(s)
    keep = R.owned(off, rows)
    xq, xs = codes(g, rows, s["K"])
    wq, ws = codes(g, len(s["counts"]), s["N"], s["K"])
    xs[~keep] = 255                          # rows no expert owns decode to NaN
    announce("mxfp4 product", R.shape_id(s), out)
    y = product(xq, xs, wq, ws, off, out, pad=8)
    ref = R.forward(torch.nan_to_num(R.codes_to_values(xq, xs)), R.codes_to_values(wq, ws), off).to(out).double()
    assert torch.equal(y[keep], ref[keep])
    assert bool((y[~keep] == SENTINEL).all())


def off_by(t, n):
    """A contiguous GPU copy of `t` that starts n bytes into its buffer."""
    flat = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")[n:]
    return flat.copy_(t.flatten()).view(t.shape)


@pytest.mark.parametrize("s", [dict(counts=[1, 2], N=40, K=256), dict(counts=[100, 30], N=72, K=384),
                               dict(counts=[700, 0, 333, 901], N=2056, K=256)], ids=R.shape_id)
def test_product_with_exponents_at_odd_addresses(s):
    g = torch.Generator().manual_seed(15)
    off, rows = R.offsets_of(s)
    xq, xs = codes(g, rows, s["K"])
    wq, ws = codes(g, len(s["counts"]), s["N"], s["K"])
    announce("mxfp4 odd addresses", R.shape_id(s))
    y = product(xq, off_by(xs, 1), wq, off_by(ws, 3), off, torch.float32)
    assert torch.equal(y, R.forward(R.codes_to_values(xq, xs), R.codes_to_values(wq, ws), off))


def test_product_of_quantised_values():
    # Whole exponent range of ordinary values; the bound of fp32 sums.
    g = torch.Generator().manual_seed(9)
    s = dict(counts=[1, 30, 0, 150], N=136, K=768)
    off, rows = R.offsets_of(s)
    xq, xs = R.quantise((torch.randn(rows, 768, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))).double())
    wq, ws = R.quantise((torch.randn(4, 136, 768, generator=g) * 0.02).double())
    announce("mxfp4 product random")
    y = product(xq, xs, wq, ws, off, torch.float32)
    xv, wv = R.codes_to_values(xq, xs), R.codes_to_values(wq, ws)
    ref, size = R.forward(xv, wv, off), R.forward(xv.abs(), wv.abs(), off)
    assert bool(((y - ref).abs() <= R.tolerance(ref, size, 768, torch.float32)).all())


def test_product_spreads_nan_exponents_to_their_outputs_only():
    g = torch.Generator().manual_seed(10)
    s = dict(counts=[20, 3], N=72, K=288)
    off, rows = R.offsets_of(s)
    xq, xs = codes(g, rows, 288)
    wq, ws = codes(g, 2, 72, 288)
    xs[4, 8], ws[1, 9, 0] = 255, 255
    announce("mxfp4 product nan")
    y = product(xq, xs, wq, ws, off, torch.float32)
    ref = R.forward(R.codes_to_values(xq, xs), R.codes_to_values(wq, ws), off)
    assert bool(ref.isnan().any())
    assert torch.equal(torch.nan_to_num(y, nan=1e30), torch.nan_to_num(ref, nan=1e30))


@pytest.mark.parametrize("M,k,E,b", [(1, 8, 128, 1), (21, 8, 128, 8), (300, 2, 5, 64), (64, 4, 300, 1), (3, 1, 1, 16)])
def test_align_offsets(M, k, E, b):
    from tests._gpu import run_align
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, E + 1, (M, k), generator=g).to(torch.int32)    # some routes are invalid
    announce("align offsets", M, k, E, b)
    _, blocks, npad = run_align(ids.numpy(), E, b)
    off = torch.full((E + 1,), -5, dtype=torch.int32, device="cuda")
    moe.moe_align_offsets(torch.from_numpy(blocks).cuda(), torch.tensor([npad], dtype=torch.int32).cuda(), E, b, off)
    count = torch.bincount(ids[(ids >= 0) & (ids < E)].long(), minlength=E)
    ref = torch.cat((torch.zeros(1, dtype=torch.int64), (-(-count // b) * b).cumsum(0)))
    assert torch.equal(off.cpu().long(), ref)


@pytest.mark.parametrize("M", [1, 37, 300])
def test_serving_step_on_four_bits(M):
    # Route, align, quantise, gather, project: the calls on one stream, as a server chains them.
    E, N, K, k = 16, 136, 288, 2
    g = torch.Generator().manual_seed(M)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(M)]).to(torch.int32)
    x = torch.randn(M, K, generator=g).bfloat16()
    w = torch.randn(E, N, K, generator=g) * 0.05
    announce("mxfp4 serving step", M)
    cap = moe.moe_align_capacity(M, k, E, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    routes, blocks, npad, off = (torch.empty(n, **i32) for n in (cap, cap, 1, E + 1))
    moe.moe_align(ids.cuda(), E, 1, routes, blocks, npad)
    moe.moe_align_offsets(blocks, npad, E, 1, off)
    xq, xs = gpu_quantise(x.cuda())
    wq, ws = gpu_quantise(w.cuda())
    token = (routes // k).long()
    y = torch.empty(M * k, N, device="cuda")
    moe.moe_grouped_matmul_mxfp4(xq[token], xs[token], wq, ws, off, y)
    torch.cuda.synchronize()
    xv, wv = (R.codes_to_values(*R.quantise(t.double())) for t in (x, w))
    order = torch.sort(ids.flatten(), stable=True)
    xr = xv[order.indices // k]
    count = torch.bincount(order.values.long(), minlength=E)
    offr = torch.cat((torch.zeros(1, dtype=torch.int64), count.cumsum(0)))
    ref, size = R.forward(xr, wv, offr), R.forward(xr.abs(), wv.abs(), offr)
    assert bool(((y.double().cpu() - ref).abs() <= R.tolerance(ref, size, K, torch.float32)).all())


def test_quantise_and_product_in_a_replayed_graph():
    E, N, K, rows = 3, 72, 160, 50
    g = torch.Generator().manual_seed(11)
    announce("mxfp4 graph")
    off = torch.tensor([0, 7, 7, 50], dtype=torch.int32)
    wq, ws = codes(g, E, N, K)
    wqd, wsd, offd = wq.cuda(), ws.cuda(), off.cuda()
    x = torch.empty(rows, K, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    xq, xs, y = torch.empty(rows, K // 2, **u8), torch.empty(rows, K // 32, **u8), torch.empty(rows, N, device="cuda")

    def step():
        moe.moe_mxfp4_quantize(x, xq, xs)
        moe.moe_grouped_matmul_mxfp4(xq, xs, wqd, wsd, offd, y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        v = R.whole(g, rows, K, top=6)
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        ref = R.forward(R.codes_to_values(*R.quantise(v)), R.codes_to_values(wq, ws), off)
        assert torch.equal(y.double().cpu(), ref)


def test_indices_past_32_bits():
    g = torch.Generator().manual_seed(18)
    rows, K, N, few = 140000, 32768, 64, 20
    announce("mxfp4 far rows")
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    xs = R.whole(g, few, K)
    x[-few:] = xs.to("cuda").to(torch.bfloat16)
    q, s = gpu_quantise(x)
    rq, rs = R.quantise(xs)
    assert torch.equal(q[-few:].cpu(), rq) and torch.equal(s[-few:].cpu(), rs) and not bool(q[:-few].any())
    moe.moe_mxfp4_dequantize(q, s, x)
    assert torch.equal(x[-few:].double().cpu(), R.codes_to_values(rq, rs)) and not bool(x[:-few].any())
    del x
    wq, ws = codes(g, 1, N, K, lo=127, hi=127)
    y = torch.empty(rows, N, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32)
    moe.moe_grouped_matmul_mxfp4(q, s, wq.cuda(), ws.cuda(), off.cuda(), y)
    # codes of whole numbers up to 4 times multiples of 0.5 up to 6: sums below 2^20 in steps of 0.5
    assert torch.equal(y[-few:].double().cpu(), R.codes_to_values(rq, rs) @ R.codes_to_values(wq, ws)[0].T)
    assert bool((y[:-few] == 0).all())
