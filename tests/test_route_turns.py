"""More work than a grid takes in one turn (2^20 workgroups) in routing, the
weighted sums and the 4-bit products: a workgroup's second task reuses its LDS
and registers. And the last of many matrices against products in 64 bits."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _route as R

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(g, lo, hi, *shape, dtype=BF16):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int8).to(dtype)


# Rows per workgroup: sixteen by the kernel for small rows, four by the other (more than 16 slots, or groups).
@pytest.mark.parametrize("M,E,k,groups,bias", [(2 ** 24 + 33, 8, 2, {}, True),
                                               (2 ** 24 + 33, 8, 3, dict(groups=4, topk_groups=2, group_top=2), False),
                                               (2 ** 22 + 9, 18, 17, {}, False),
                                               (2 ** 22 + 9, 34, 3, dict(groups=17, topk_groups=5, group_top=2), True)])
def test_routing(M, E, k, groups, bias):
    g = gen(E)
    logits = torch.randn(M, E, generator=g, device="cuda")
    logits[M - 3, 2] = float("nan")            # such a row takes its wave's detour in the second turn
    b = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
    dw = torch.randn(M, k, generator=g, device="cuda")
    ids, w, d = torch.empty(M, k, dtype=I32, device="cuda"), torch.empty(M, k, device="cuda"), torch.empty_like(logits)
    announce("route turns", M, E, k)
    for score, renormalize in ((R.SOFTMAX, False), (R.SIGMOID, True)):
        kw = dict(score=score, renormalize=renormalize, scale=1.5)
        moe.moe_route(logits, ids, w, bias=b, **kw, **groups)
        moe.moe_route_grad(logits, ids, dw, d, **kw)
        half = M // 2 + 5                      # calls that end within a turn
        for a, z in ((0, half), (half, M)):
            i2, w2, d2 = torch.empty_like(ids[a:z]), torch.empty_like(w[a:z]), torch.empty_like(d[a:z])
            moe.moe_route(logits[a:z], i2, w2, bias=b, **kw, **groups)
            moe.moe_route_grad(logits[a:z], i2, dw[a:z], d2, **kw)
            assert torch.equal(i2, ids[a:z])
            for one, other in ((w2, w[a:z]), (d2, d[a:z])):
                assert torch.equal(one.view(I32), other.view(I32))       # (bits: a NaN is one, too)


def test_sums():
    # 2^28 threads a turn, one piece of eight columns each.
    M = 2 ** 28 + 77
    rows = whole(gen(1), -100, 100, M, 8)
    y = torch.zeros_like(rows)
    announce("combine turns")
    moe.moe_combine(rows, None, None, y)
    assert torch.equal(y, rows)


@pytest.mark.parametrize("M,H,k", [(2 ** 23 + 9, 8, 2), (2 ** 22 + 5, 264, 1), (2 ** 21 + 3, 520, 1), (2 ** 20 + 3, 1032, 1)])
def test_gradients_of_sums(M, H, k):
    g = gen(H)
    dy, rows = whole(g, -3, 4, M, H), whole(g, -3, 4, M * k, H)
    w = whole(g, -3, 4, M, k, dtype=F32)
    drows, dw = torch.zeros_like(rows), torch.full_like(w, float("nan"))
    announce("combine gradient turns", M, H)
    moe.moe_combine_grad(dy, rows, None, w, drows, dw)
    step = M // 8 + 1
    for a in range(0, M, step):
        z = min(a + step, M)
        r = rows[a * k:z * k].view(z - a, k, H)
        assert torch.equal(drows[a * k:z * k].view(z - a, k, H), w[a:z].to(BF16).unsqueeze(-1) * dy[a:z].unsqueeze(1))
        assert torch.equal(dw[a:z], (r.float() * dy[a:z].float().unsqueeze(1)).sum(2))


def packed(g, E, N, K, group):
    q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), dtype=I32, generator=g, device="cuda")
    s = torch.exp2(torch.randint(-2, 3, (E, N, K // group), generator=g, device="cuda").float()).half()
    z = torch.randint(0, 16, s.shape, dtype=torch.uint8, generator=g, device="cuda")
    return moe.DeviceProjection(moe.MOE_W_INT4_AWQ, group, q, s, z)


def matrix(p, e, first=0, last=None):
    """fp64 rows first..last of matrix e."""
    q, s, z = (t[e, first:last] for t in (p.q, p.scale, p.zero))
    v = torch.empty(*q.shape, 8, dtype=torch.float64, device="cuda")
    for i, element in enumerate(R.SLOT):
        v[..., element] = ((q >> (4 * i)) & 15).double()
    v = v.flatten(-2).unflatten(-1, (-1, p.group))
    return ((v - z.double().unsqueeze(-1)) * s.double().unsqueeze(-1)).flatten(-2)


# One task per route and sixteen features: chunks of 128 and of 256.
@pytest.mark.parametrize("M,N,K,group", [(2 ** 20 + 5, 16, 32, 32), (2 ** 18 + 3, 56, 4096, 128)])
def test_routed_products(M, N, K, group):
    g = gen(N)
    p = packed(g, 2, N, K, group)
    x = whole(g, -3, 4, M, K)
    ids = torch.randint(-1, 3, (M, 1), dtype=I32, generator=g, device="cuda")
    y = torch.full((M, 1, N), float("nan"), device="cuda")
    announce("matvec turns", M, N, K)
    moe.moe_matvec_int4(x, p, y, topk_ids=ids)
    step = M // 4 + 1
    for a in range(0, M, step):
        xs, want = x[a:a + step].double(), torch.zeros(x[a:a + step].shape[0], N, dtype=torch.float64, device="cuda")
        for e in range(2):
            want = torch.where(ids[a:a + step] == e, xs @ matrix(p, e).T, want)
        assert torch.equal(y[a:a + step, 0].double(), want)


def test_products_of_many_rows():
    # 64 rows and 64 features a task.
    M, N, K = 64 * 1024 + 37, 64 * 1024 + 24, 32
    g = gen(3)
    p = packed(g, 1, N, K, 32)
    x = whole(g, -3, 4, M, K)
    y = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    announce("matvec many rows")
    moe.moe_matvec_int4(x, p, y)
    W = matrix(p, 0).float().T.contiguous()
    for a in range(0, M, 8192):                # exact in fp32: whole numbers of quarters below 2^15
        assert torch.equal(y[a:a + 8192], (x[a:a + 8192].float() @ W).to(BF16))


def test_last_of_many_matrices_against_products():
    # 64 matrices of 16384 x 8192, 4.3 GB of words: first and last features of the first and last, in 64 bits.
    E, N, K = 64, 16384, 8192
    g = gen(4)
    p = packed(g, E, N, K, 128)
    x = whole(g, -3, 4, 1, K)
    ids = torch.tensor([[E - 1, 0]], dtype=I32, device="cuda")
    y = torch.full((1, 2, N), float("nan"), device="cuda")
    announce("last matrix, products")
    moe.moe_matvec_int4(x, p, y, topk_ids=ids)
    for j, e in ((0, E - 1), (1, 0)):
        for first, last in ((0, 64), (N // 2 - 8, N // 2 + 72), (N - 64, N)):
            want = matrix(p, e, first, last) @ x[0].double()
            assert torch.equal(y[0, j, first:last].double(), want)
        alone = torch.empty(1, 1, N, device="cuda")          # the same kernel on this matrix alone: the same bits
        one = moe.DeviceProjection(moe.MOE_W_INT4_AWQ, 128, *(t[e:e + 1].clone() for t in (p.q, p.scale, p.zero)))
        moe.moe_matvec_int4(x, one, alone, topk_ids=torch.zeros(1, 1, dtype=I32, device="cuda"))
        assert torch.equal(alone[0, 0], y[0, j])
