"""Offsets past 2^31 elements (rows far apart, the last of many experts' weights)
in routing, the weighted sums and the 4-bit products, and two streams at once."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _route as R

pytestmark = pytest.mark.gpu

STRIDE = 1 << 22          # the largest row stride


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


def far_rows(rows, cols, dtype):
    """[rows, cols] whose rows are STRIDE elements apart: past 2^31 elements from row 512 on."""
    return torch.empty(rows * STRIDE, dtype=dtype, device="cuda").view(rows, STRIDE)[:, :cols]


@pytest.mark.parametrize("E,k,bias", [(128, 8, False), (256, 4, True), (700, 8, False), (200, 20, True)])
def test_routing_of_rows_far_apart(E, k, bias):
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(530, E, generator=g).bfloat16().cuda()
    b = (0.1 * torch.randn(E, generator=g)).cuda() if bias else None
    far, dfar = far_rows(530, E, torch.bfloat16), far_rows(530, E, torch.bfloat16)
    far.copy_(logits)
    ids, ids2 = (torch.empty(530, k, dtype=torch.int32, device="cuda") for _ in range(2))
    w, w2 = (torch.empty(530, k, device="cuda") for _ in range(2))
    d = torch.empty_like(logits)
    announce("far route", E, k, bias)
    for score, renormalize in ((R.SOFTMAX, False), (R.SIGMOID, True)):
        moe.moe_route(logits, ids, w, bias=b, score=score, renormalize=renormalize)
        moe.moe_route(far, ids2, w2, bias=b, score=score, renormalize=renormalize)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)
        moe.moe_route_grad(logits, ids, w, d, score=score, renormalize=renormalize)
        moe.moe_route_grad(far, ids, w, dfar, score=score, renormalize=renormalize)
        assert torch.equal(d, dfar)


def test_sums_of_rows_far_apart():
    g = torch.Generator().manual_seed(2)
    M, k, H, n = 520, 2, 64, 1040
    rows, dy = torch.randn(n, H, generator=g).bfloat16().cuda(), torch.randn(M, H, generator=g).bfloat16().cuda()
    w = torch.rand(M, k, generator=g).cuda()
    pos = torch.randperm(n, generator=g).view(M, k).to(torch.int32).cuda()
    far, dfar = far_rows(n, H, torch.bfloat16), far_rows(n, H, torch.bfloat16)
    yfar = far_rows(M, H, torch.bfloat16)
    far.copy_(rows)
    y, d = torch.empty_like(dy), torch.empty_like(rows)
    dw, dw2 = torch.empty_like(w), torch.empty_like(w)
    announce("far combine")
    moe.moe_combine(rows, pos, w, y)
    moe.moe_combine(far, pos, w, yfar)
    assert torch.equal(y, yfar)
    yfar.copy_(dy)
    moe.moe_combine_grad(dy, rows, pos, w, d, dw)
    moe.moe_combine_grad(yfar, far, pos, w, dfar, dw2)
    assert torch.equal(d, dfar) and torch.equal(dw, dw2)


def test_products_of_rows_far_apart():
    g = torch.Generator().manual_seed(3)
    for M in (530, 514):
        x = torch.randn(M, 96, generator=g).bfloat16().cuda()
        q = torch.randint(-2 ** 31, 2 ** 31, (1, 40, 12), generator=g).to(torch.int32).cuda()
        s = torch.rand(1, 40, 3, generator=g).half().cuda()
        p = moe.DeviceProjection(moe.MOE_W_INT4_AWQ, 32, q, s, None)
        far, yfar = far_rows(M, 96, torch.bfloat16), far_rows(M, 40, torch.bfloat16)
        far.copy_(x)
        y = torch.empty(M, 40, dtype=torch.bfloat16, device="cuda")
        announce("far matvec", M)
        moe.moe_matvec_int4(x, p, y)
        moe.moe_matvec_int4(far, p, yfar)
        assert torch.equal(y, yfar)


def test_last_of_many_matrices():
    # 64 matrices of 16384 x 8192: 4.3 GB of words.
    E, N, K = 64, 16384, 8192
    q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), dtype=torch.int32, device="cuda")
    s = torch.rand(E, N, K // 128, device="cuda").half()
    z = torch.randint(0, 16, (E, N, K // 128), dtype=torch.uint8, device="cuda")
    x = torch.randn(1, K, device="cuda").bfloat16()
    y = torch.empty(1, 2, N, device="cuda")
    alone = torch.empty(1, 1, N, device="cuda")
    announce("last matrix")
    moe.moe_matvec_int4(x, moe.DeviceProjection(moe.MOE_W_INT4_AWQ, 128, q, s, z), y,
                        topk_ids=torch.tensor([[E - 1, 0]], dtype=torch.int32, device="cuda"))
    one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for j, e in ((0, E - 1), (1, 0)):
        w = moe.DeviceProjection(moe.MOE_W_INT4_AWQ, 128, q[e:e + 1].clone(), s[e:e + 1].clone(), z[e:e + 1].clone())
        moe.moe_matvec_int4(x, w, alone, topk_ids=one)
        # other kernels serve other numbers of tiles, in another order of sums
        assert float((y[0, j] - alone[0, 0]).norm() / alone.norm()) < 1e-5


def test_two_streams_at_once():
    # Calls share nothing: overlapping on two streams they give what each gives alone.
    g = torch.Generator().manual_seed(4)
    jobs = []
    for M, E, H in ((300, 64, 512), (2000, 128, 256)):
        logits, x = torch.randn(M, E, generator=g).cuda(), torch.randn(M, H, generator=g).bfloat16().cuda()
        q = torch.randint(-2 ** 31, 2 ** 31, (1, 200, H // 8), generator=g).to(torch.int32).cuda()
        p = moe.DeviceProjection(moe.MOE_W_INT4_AWQ, 64, q, torch.rand(1, 200, H // 64, generator=g).half().cuda(), None)
        out = dict(ids=torch.empty(M, 4, dtype=torch.int32, device="cuda"), w=torch.empty(M, 4, device="cuda"),
                   rows=torch.empty(M * 4, H, dtype=torch.bfloat16, device="cuda"),
                   y=torch.empty(M, H, device="cuda"), z=torch.empty(M, 200, device="cuda"))

        def job(stream, logits=logits, x=x, p=p, out=out):
            moe.moe_route(logits, out["ids"], out["w"], stream=stream)
            moe.moe_combine_grad(x, None, None, out["w"], out["rows"], None, stream=stream)
            moe.moe_combine(out["rows"], None, out["w"], out["y"], stream=stream)
            moe.moe_matvec_int4(x, p, out["z"], stream=stream)

        jobs.append((job, out, torch.cuda.Stream()))
    announce("two streams")
    want = []
    for job, out, _ in jobs:
        job(None)
        want.append({n: t.clone() for n, t in out.items()})
        for t in out.values():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for job, _, stream in jobs:
            job(stream)
    torch.cuda.synchronize()
    for (_, out, _), w in zip(jobs, want):
        assert all(torch.equal(out[n], w[n]) for n in w)
