"""Every kernel shape of the products with packed 4-bit weights against exact
sums: the sizes are held to reach all of them by the rule that picks the shape."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _matvec as V
from tests import _route as R

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    return V.compile_rule(str(tmp_path_factory.mktemp("shape")))


def chosen(shape, case):
    M, k, N, K, group = case
    return shape(k > 0, M * max(k, 1), N, K, group)


def test_sizes_reach_every_shape(shape):
    got = {chosen(shape, c) for c in V.CASES}
    want = {(*s, splits, flush) for s, all_splits in V.BUILT.items() for splits in all_splits for flush in (1, 2, 4)}
    assert got == want, (sorted(want - got), sorted(got - want))


def test_rule_gives_built_shapes_only(shape):
    for rows in (1, 2, 4, 5, 16, 17, 32, 33, 48, 49, 64, 65, 128, 200, 4096, 2 ** 31 - 256):
        for N in (1, 16, 4096, 8176, 8177, 8192, 16383, 16384, 16385, 32768, 1 << 20):
            for K in (32, 512, 1024, 2048, 2080, 4064, 4096, 8192, 1 << 20):
                for routed in (False, True):
                    c = shape(routed, rows, N, K, 32)
                    assert c[3] in V.BUILT[c[:3]] and c[4] == 1, (routed, rows, N, K, c)
                    assert routed or c[1] >= min(rows, 64)


def test_no_rule_for_one_count_of_tiles(shape):
    # Where the summed index changes the count of tiles from which another shape is taken, it does so by a range
    # of counts, not by one.
    for rows in (1, 16, 64):
        edges = set()
        for K in (256, 768, 1024, 1536, 2048, 4064):
            shapes = [shape(False, rows, 16 * tiles, K, 32) for tiles in range(500, 2100)]
            edges |= {500 + i for i in range(1, len(shapes)) if shapes[i] != shapes[i - 1]}
        edges = sorted(edges)
        assert all(b - a >= 64 for a, b in zip(edges, edges[1:])), (rows, edges)


def exact(x, q, s, z, group):
    """fp64 [M, N] on the GPU: whole numbers times quarters, so sums are exact in any order."""
    v = torch.empty(*q.shape, 8, dtype=torch.float64, device="cuda")
    for i, element in enumerate(R.SLOT):
        v[..., element] = ((q >> (4 * i)) & 15).double()
    v = v.flatten(-2).unflatten(-1, (-1, group))
    return x.double() @ ((v - z.double().unsqueeze(-1)) * s.double().unsqueeze(-1)).flatten(-2).T


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("case", V.CASES, ids=lambda c: "M%d_k%d_N%d_K%d_g%d" % c)
def test_exact_in_every_shape(case, dtype, shape):
    # Inputs to 3, values to 15 (15 quarters to 60): sums are multiples of 1/4 below 2^21, exact in fp32.
    M, k, N, K, group = case
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    E = 3 if k else 1
    dev = dict(generator=g, device="cuda")
    q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), dtype=torch.int32, **dev)
    s = torch.exp2(torch.randint(-2, 3, (E, N, K // group), **dev).float()).half()
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, **dev)
    x = torch.randint(-3, 4, (M, K), **dev).to(dtype)
    p = moe.DeviceProjection(moe.MOE_W_INT4_AWQ, group, q, s, z)
    print("[gpu-case] matvec shape", case, dtype, chosen(shape, case), flush=True)
    out = F32 if (M + N + K + group) % 3 else dtype
    if k == 0:
        wide = torch.full((M, N + 2), 77.0, dtype=out, device="cuda")
        moe.moe_matvec_int4(x, p, wide[:, :N])
        assert torch.equal(wide[:, :N].double(), exact(x, q[0], s[0], z[0], group).to(out).double())
        assert bool((wide[:, N:] == 77.0).all())
        return
    ids = torch.randint(-1, E, (M, k), dtype=torch.int32, **dev)
    ids[0, 0], ids[M - 1, k - 1] = E - 1, E
    y = torch.full((M, k, N), float("nan"), dtype=out, device="cuda")
    moe.moe_matvec_int4(x, p, y, topk_ids=ids)
    all_of = torch.stack([exact(x, q[e], s[e], z[e], group).to(out).double() for e in range(E)])
    here = ((ids >= 0) & (ids < E)).unsqueeze(-1)
    rows = torch.arange(M, device="cuda").unsqueeze(-1)
    want = torch.where(here, all_of[ids.clamp(0, E - 1).long(), rows], torch.zeros((), dtype=torch.float64, device="cuda"))
    assert torch.equal(y.double(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("N,K,group", [(72, 1056, 32), (8197, 2176, 128)])
def test_rows_in_batches_of_other_sizes(N, K, group, dtype, shape):
    # By the same kernel a row has the same bits whatever stands beside it; by another its sums have another order,
    # and both are within the bound of fp32 sums.
    g = torch.Generator(device="cuda").manual_seed(5)
    dev = dict(generator=g, device="cuda")
    q = torch.randint(-2 ** 31, 2 ** 31, (1, N, K // 8), dtype=torch.int32, **dev)
    s = (0.002 + 0.008 * torch.rand(1, N, K // group, **dev)).half()
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, **dev)
    p = moe.DeviceProjection(moe.MOE_W_INT4_AWQ, group, q, s, z)
    x = torch.randn(64, K, **dev).to(dtype)
    print("[gpu-case] matvec batches", N, K, dtype, flush=True)
    whole = torch.empty(64, N, device="cuda")
    moe.moe_matvec_int4(x, p, whole)
    ref = exact(x, q[0], s[0], z[0], group)
    # A group sums (16 + q) x and x, each addition off by a step of a partial sum; the groups' sums, scaled, add up
    # over K / group steps, and seven between waves.
    scale = s[0].double().repeat_interleave(group, -1)
    zero = z[0].double().repeat_interleave(group, -1)
    bound = (2 * group + 4 + K / group + 7) * 2.0 ** -23 * (x.double().abs() @ (scale * (32.0 + zero)).T)
    same = 0
    for a, b in ((0, 64), (0, 49), (7, 64), (3, 60), (0, 48), (16, 64), (0, 16), (5, 6), (40, 64), (60, 64)):
        y = torch.empty(b - a, N, device="cuda")
        moe.moe_matvec_int4(x[a:b], p, y)
        if shape(False, b - a, N, K, group) == shape(False, 64, N, K, group):
            assert torch.equal(y, whole[a:b])
            same += 1
        assert bool(((y.double() - ref[a:b]).abs() <= bound[a:b]).all())
    assert same == 4


@pytest.mark.gpu
def test_largest_inputs_that_do_not_overflow():
    # A sum of 128 products is below 128 * 31 |x| < 2^12 |x|: bf16 inputs below 2^116 stay within fp32.
    N, K = 40, 512
    g = torch.Generator(device="cuda").manual_seed(6)
    dev = dict(generator=g, device="cuda")
    print("[gpu-case] matvec largest inputs", flush=True)
    for group in (32, 64, 128, 512):
        q = torch.randint(-2 ** 31, 2 ** 31, (1, N, K // 8), dtype=torch.int32, **dev)
        q[:, 0], q[:, 1] = -1, 0                                   # the largest and the smallest sums
        s = torch.full((1, N, K // group), 2.0 ** -14, dtype=F16, device="cuda")
        z = torch.randint(0, 16, s.shape, dtype=torch.uint8, **dev)
        z[:, 0], z[:, 1] = 0, 15
        x = torch.where(torch.rand(5, K, **dev) < 0.5, -(2.0 ** 115), 2.0 ** 115)
        x[0] = 2.0 ** 115
        y = torch.empty(5, N, device="cuda")
        moe.moe_matvec_int4(x.to(BF16), moe.DeviceProjection(moe.MOE_W_INT4_AWQ, group, q, s, z), y)
        assert torch.equal(y.double(), exact(x, q[0], s[0], z[0], group))     # whole numbers of 2^101, below 2^13 of them
