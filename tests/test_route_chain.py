"""Routing, the weighted sum of routes and the 4-bit products as they are used
together: a router in front of the layer, a layer of one's own activation on
packed weights, and a training step with every gradient by hand-written calls."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
import oracle
from tests import _route as R

pytestmark = pytest.mark.gpu


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


@pytest.mark.parametrize("path", [moe.MOE_PATH_DECODE, moe.MOE_PATH_GROUPED], ids=["decode", "grouped"])
def test_router_in_front_of_the_layer(path):
    from tests import _gpu
    dw = _gpu.device_workload("tiny")
    cfg = dw.cfg
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(cfg.M, cfg.E, generator=g)
    logits[0, 1:] = -float("inf")              # one expert left: the other route is expert -1, which has no share
    bias = 0.1 * torch.randn(cfg.E, generator=g)
    router = moe.MoeRouter(cfg.k, moe.MOE_SCORE_SIGMOID, bias.cuda(), scale=1.5, groups=4, topk_groups=2, group_top=2)
    announce("router and layer", path)
    ids, w = router(logits.cuda())
    y = dw.layer.forward(dw.x, ids, w, path=path).cpu().numpy().astype(np.float64)
    want = R.choose(logits, cfg.k, R.SIGMOID, bias, 4, 2, 2)
    assert torch.equal(ids.cpu(), want) and want[0].tolist() == [0, -1]
    rw = R.weights(logits, want, R.SIGMOID, True, 1.5).float().numpy()
    ref = oracle.ffn(dw.wl.x, want.numpy(), rw, dw.wl.w13, dw.wl.w2, cfg.E)
    assert np.linalg.norm(y - ref) / np.linalg.norm(ref) <= 1e-3


def test_packed_experts_with_another_activation():
    # Gate/up and down products of a token's own experts, relu(gate) * up between them, and the sum of the
    # routes in route order; a route without an expert has no share.
    M, E, k, H, I, group = 3, 8, 3, 256, 96, 32
    g = torch.Generator().manual_seed(2)

    def packed(N, K):
        q = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=g).to(torch.int32)
        s = (0.002 + 0.008 * torch.rand(E, N, K // group, generator=g)).half()
        z = torch.randint(0, 16, s.shape, generator=g, dtype=torch.uint8)
        return moe.DeviceProjection(moe.MOE_W_INT4_AWQ, group, q.cuda(), s.cuda(), z.cuda()), R.dequantise(q, s, z, group)

    w13, W13 = packed(2 * I, H)
    w2, W2 = packed(H, I)
    x = torch.randn(M, H, generator=g).bfloat16()
    logits = torch.randn(M, E, generator=g)
    logits[1, 2:] = -float("inf")
    announce("packed experts")
    ids, w = moe.MoeRouter(k)(logits.cuda())
    h = torch.empty(M, k, 2 * I, device="cuda")
    moe.moe_matvec_int4(x.cuda(), w13, h, topk_ids=ids)
    a = (h[..., :I].relu() * h[..., I:]).bfloat16().view(M * k, I)
    rows = torch.empty(M * k, 1, H, device="cuda")
    moe.moe_matvec_int4(a, w2, rows, topk_ids=ids.view(M * k, 1))
    y = torch.empty(M, H, device="cuda")
    moe.moe_combine(rows.view(M * k, H), None, w, y)

    want = R.choose(logits, k, R.SOFTMAX)
    assert torch.equal(ids.cpu(), want) and want[1].tolist()[2] == -1
    rw = R.weights(logits, want, R.SOFTMAX, True, 1.0)
    ref, mag = torch.zeros(M, H, dtype=torch.float64), torch.zeros(M, H, dtype=torch.float64)
    for t in range(M):
        for j in range(k):
            if want[t, j] >= 0:
                v = W13[want[t, j]] @ x[t].double()
                act = v[:I].relu() * v[I:]
                ref[t] += rw[t, j] * (W2[want[t, j]] @ act)
                mag[t] += rw[t, j] * (W2[want[t, j]].abs() @ act.abs())
    # The activation is rounded to bf16 once (2^-8); the fp32 sums before it are 2^-12 of it at worst here,
    # where gate and up cancel to a few hundredths of their terms, and those after it far less.
    assert bool(((y.double().cpu() - ref).abs() <= (2.0 ** -8 + 2.0 ** -10) * mag).all())


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, router):
        ids, w = router(logits)
        ctx.save_for_backward(logits, ids)
        ctx.router = router
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, dw):
        logits, ids = ctx.saved_tensors
        return ctx.router.grad(logits, ids, dw.contiguous()), None


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, positions):
        rows = torch.zeros(positions.numel(), x.shape[1], dtype=x.dtype, device=x.device)
        moe.moe_combine_grad(x, None, positions, None, rows, None)
        ctx.save_for_backward(positions)
        return rows

    @staticmethod
    def backward(ctx, drows):
        positions, = ctx.saved_tensors
        dx = torch.empty(positions.shape[0], drows.shape[1], dtype=drows.dtype, device=drows.device)
        moe.moe_combine(drows.contiguous(), positions, None, dx)
        return dx, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w, positions):
        y = torch.empty(positions.shape[0], rows.shape[1], dtype=torch.float32, device=rows.device)
        moe.moe_combine(rows, positions, w, y)
        ctx.save_for_backward(rows, w, positions)
        return y

    @staticmethod
    def backward(ctx, dy):
        rows, w, positions = ctx.saved_tensors
        drows, dw = torch.zeros_like(rows), torch.empty_like(w)
        moe.moe_combine_grad(dy.contiguous(), rows, positions, w, drows, dw)
        return drows, dw, None


@pytest.mark.parametrize("M,E,base,held", [(40, 6, 0, 6), (60, 8, 2, 3)])
def test_training_step(M, E, base, held):
    # Router, gather, two expert products with a threshold between them, weighted sum; on a shard, routes to
    # other experts have no row. Logits are 0 or -inf: a chosen expert's sigmoid is 1/2 and its slope 1/4, so
    # with a scale of 2 every value and gradient is a multiple of 1/2 that bf16 holds exactly.
    from tests.test_ragged_chain import Product
    k, H, I = 2, 24, 16
    announce("training step", M, E, base)
    g = torch.Generator().manual_seed(3)

    def sparse(*shape):
        return (torch.randint(-1, 2, shape, generator=g) * (torch.rand(*shape, generator=g) < 0.3)).double()

    x, w1, w2, dy = sparse(M, H), sparse(held, I, H), sparse(held, H, I), sparse(M, H)
    logits = torch.where(torch.rand(M, E, generator=g) < 0.5, 0.0, -float("inf")).double()
    logits[0] = -float("inf")                 # a token without any expert
    router = moe.MoeRouter(k, moe.MOE_SCORE_SIGMOID, renormalize=False, scale=2.0)
    leaves = [t.cuda().to(d).requires_grad_() for t, d in ((x, torch.bfloat16), (w1, torch.bfloat16),
                                                           (w2, torch.bfloat16), (logits, torch.float32))]
    ids, w = Route.apply(leaves[3], router)
    i32 = dict(dtype=torch.int32, device="cuda")
    routes, blocks, n, offsets = (torch.empty(c, **i32) for c in (M * k, M * k, 1, held + 1))
    positions = torch.empty(M, k, **i32)
    moe.moe_align_ex(ids, held, base, 1, routes, blocks, n)
    moe.moe_align_offsets(blocks, n, held, 1, offsets)
    moe.moe_align_positions(routes, n, positions)
    a = Product.apply(Gather.apply(leaves[0], positions), leaves[1], offsets).relu()
    y = Combine.apply(Product.apply(a, leaves[2], offsets), w, positions)
    y.backward(dy.cuda().float())

    ref = [t.clone().requires_grad_() for t in (x, w1, w2, logits)]
    want = R.choose(logits, k, R.SIGMOID)
    out = torch.zeros(M, H, dtype=torch.float64)
    for t in range(M):
        for e in want[t].tolist():
            if base <= e < base + held:
                v = ref[2][e - base] @ (ref[1][e - base] @ ref[0][t]).relu()
                out = out.index_add(0, torch.tensor([t]), (2 * torch.sigmoid(ref[3][t, e]) * v).unsqueeze(0))
    out.backward(dy)
    assert torch.equal(ids.cpu(), want)
    largest = max(float(t.detach().abs().max()) for t in (out, *(r.grad for r in ref)))
    assert 4 < largest <= 128                # with steps of 1/2, what bf16 holds exactly
    assert torch.equal(y.detach().double().cpu(), out.detach())
    for t, r in zip(leaves, ref):
        assert torch.equal(t.grad.double().cpu(), r.grad)
