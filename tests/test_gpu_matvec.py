"""Products with packed 4-bit weights (moe_matvec_int4) against 64-bit
references: exact on whole numbers, within the bound of fp32 sums on random
values; every group, tails, strides, expert IDs, streams and graphs."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _route as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
SENTINEL = 77.0


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


def packed(gen, E, N, K, group, whole=False):
    """(q, scale, zero) on the host; whole: scales that are powers of two, so that sums are exact."""
    q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=gen).to(torch.int32)
    shape = (E, N, K // group)
    s = torch.exp2(torch.randint(-2, 3, shape, generator=gen).float()) if whole else \
        0.002 + 0.008 * torch.rand(shape, generator=gen)
    return q, s.to(F16), torch.randint(0, 16, shape, generator=gen, dtype=torch.uint8)


def projection(q, s, z, group):
    return moe.DeviceProjection(moe.MOE_W_INT4_AWQ, group, q.cuda(), s.cuda(), None if z is None else z.cuda())


def reference(x, W, ids=None):
    if ids is None:
        return x.double() @ W[0].T
    y = torch.zeros(x.shape[0], ids.shape[1], W.shape[1], dtype=torch.float64)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            if 0 <= int(ids[t, j]) < W.shape[0]:
                y[t, j] = W[int(ids[t, j])] @ x[t].double()
    return y


# N, K, group: tiles that end inside, chunks that end inside, groups smaller and larger than a chunk,
# as long as the sum, of odd multiples of 32.
SHAPES = [(1, 32, 32), (16, 128, 128), (17, 96, 32), (24, 160, 32), (8, 192, 64), (40, 384, 128), (33, 672, 96),
          (5, 1024, 1024), (100, 480, 160), (48, 2048, 128), (264, 1056, 32), (72, 768, 256), (31, 4064, 32),
          (16, 8192, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "N%d_K%d_g%d" % s)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_exact_on_whole_numbers(shape, dtype):
    N, K, group = shape
    gen = torch.Generator().manual_seed(N + K)
    q, s, z = packed(gen, 1, N, K, group, whole=True)
    p, sym = projection(q, s, z, group), projection(q, s, None, group)
    W, S = R.dequantise(q, s, z, group), R.dequantise(q, s, torch.full_like(z, 8), group)
    for M, out, pad in ((1, F32, 0), (2, dtype, 8), (15, F32, 8), (16, F32, 0), (17, dtype, 0), (32, F32, 0),
                        (33, F32, 24), (63, F32, 0), (64, dtype, 8), (65, F32, 0), (131, F32, 0)):
        x = torch.randint(-3, 4, (M, K), generator=gen)
        xd = torch.full((M, K + pad), float("nan"), dtype=dtype, device="cuda")
        xd[:, :K] = x.cuda()
        y = torch.full((M, N + 3), SENTINEL, dtype=out, device="cuda")
        announce("matvec", shape, dtype, M)
        moe.moe_matvec_int4(xd[:, :K], p, y[:, :N])
        torch.cuda.synchronize()
        assert torch.equal(y[:, :N].cpu().double(), reference(x, W).to(out).double())
        assert bool((y[:, N:] == SENTINEL).all())
        moe.moe_matvec_int4(xd[:, :K], sym, y[:, :N])
        assert torch.equal(y[:, :N].cpu().double(), reference(x, S).to(out).double())


@pytest.mark.parametrize("E,N,K,group", [(1, 16, 32, 32), (5, 24, 160, 32), (8, 100, 768, 128), (130, 33, 256, 64)])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_experts_rows(E, N, K, group, dtype):
    gen = torch.Generator().manual_seed(E + N)
    q, s, z = packed(gen, E, N, K, group, whole=True)
    p, W = projection(q, s, z, group), R.dequantise(q, s, z, group)
    for M, k in ((1, 1), (1, 8), (3, 2), (9, 5)):
        x = torch.randint(-3, 4, (M, K), generator=gen)
        ids = torch.randint(-1, E + 1, (M, k), generator=gen).to(torch.int32)      # some no experts, some repeated
        ids[0, 0] = E - 1
        if M > 1:
            ids[1, 0], ids[1, 1] = 2 ** 31 - 1, -2 ** 31
        y = torch.full((M, k, N), float("nan"), device="cuda")
        announce("matvec experts", E, N, K, dtype, M, k)
        moe.moe_matvec_int4(x.cuda().to(dtype), p, y, topk_ids=ids.cuda())
        assert torch.equal(y.cpu().double(), reference(x, W, ids))


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("N,K,group,M", [(40, 2048, 128, 1), (50, 1056, 32, 20), (20, 8192, 128, 64)])
def test_random_values(dtype, N, K, group, M):
    gen = torch.Generator().manual_seed(3)
    q, s, z = packed(gen, 1, N, K, group)
    x = torch.randn(M, K, generator=gen).to(dtype)
    announce("matvec random", N, K, M, dtype)
    for out in (F32, dtype):
        y = torch.empty(M, N, dtype=out, device="cuda")
        moe.moe_matvec_int4(x.cuda(), projection(q, s, z, group), y)
        ref = reference(x, R.dequantise(q, s, z, group))
        # A group sums (16 + q) x and x, each addition off by a step of a partial sum; the groups' sums,
        # scaled, add up over K / group steps (and three between waves).
        scale = s.double().repeat_interleave(group, -1)[0]
        zero = z.double().repeat_interleave(group, -1)[0]
        mag = x.double().abs() @ (scale * (32.0 + zero)).T
        sums = (2 * group + 4 + K / group + 3) * 2.0 ** -23 * mag
        assert bool(((y.double().cpu() - ref).abs() <= sums + HALF[out] * (ref.abs() + sums) + 2.0 ** -25).all())
        # and as near as fp32 sums come at random: errors of a group's sums, of magnitude sqrt(group),
        # add up like sqrt(K); a hundred times less than the bound above.
        if out is F32:
            assert float((y.double().cpu() - ref).norm() / ref.norm()) < 4e-6


def test_nan_and_infinite_inputs_stay_in_their_rows():
    gen = torch.Generator().manual_seed(4)
    q, s, z = packed(gen, 1, 40, 256, 64)
    x = torch.randn(20, 256, generator=gen).to(BF16)
    p = projection(q, s, z, 64)
    clean, y = torch.empty(20, 40, device="cuda"), torch.empty(20, 40, device="cuda")
    announce("matvec nan")
    moe.moe_matvec_int4(x.cuda(), p, clean)
    x[3, 7], x[18, 200] = float("nan"), float("inf")
    moe.moe_matvec_int4(x.cuda(), p, y)
    bad = torch.zeros(20, dtype=torch.bool, device="cuda")
    bad[[3, 18]] = True
    assert not bool(y[bad].isfinite().any()) and torch.equal(y[~bad], clean[~bad])


def test_rows_do_not_depend_on_the_batch():
    gen = torch.Generator().manual_seed(5)
    q, s, z = packed(gen, 1, 72, 1056, 32)
    p = projection(q, s, z, 32)
    x = torch.randn(64, 1056, generator=gen).to(BF16).cuda()
    announce("matvec batch")
    whole = torch.empty(64, 72, device="cuda")
    moe.moe_matvec_int4(x, p, whole)
    for a, b in ((0, 16), (5, 6), (40, 64), (3, 30)):
        y = torch.empty(b - a, 72, device="cuda")
        moe.moe_matvec_int4(x[a:b], p, y)
        # A row's sums run in the order its kernel has, whatever the other rows are.
        assert torch.allclose(y, whole[a:b], rtol=0, atol=1e-4)
    same = torch.empty_like(whole)
    moe.moe_matvec_int4(x.flip(0).contiguous(), p, same)
    assert torch.equal(same.flip(0), whole)


def test_graph_and_side_stream():
    gen = torch.Generator().manual_seed(6)
    q, s, z = packed(gen, 6, 136, 512, 128)
    p = projection(q, s, z, 128)
    x = torch.randn(2, 512, generator=gen).to(BF16).cuda()
    ids = torch.tensor([[0, 5, 2], [4, -1, 4]], dtype=torch.int32, device="cuda")
    y = torch.empty(2, 3, 136, device="cuda")
    announce("matvec graph")
    moe.moe_matvec_int4(x, p, y, topk_ids=ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_matvec_int4(x, p, y, topk_ids=ids)
    for _ in range(3):
        x.normal_(), y.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        moe.moe_matvec_int4(x, p, y, topk_ids=ids, stream=side)
        side.synchronize()
        assert torch.equal(got, y)
    assert moe.moe_matvec_int4(x[:0], p, y[:0], topk_ids=ids[:0]) == moe.MOE_OK
