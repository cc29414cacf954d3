"""The chain from routes to ragged products where some routes have no expert
here, as on every expert-parallel shard: the README's lines, and the calls."""
import os
import re

import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _ragged as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def readme_gather():
    with open(os.path.join(ROOT, "README.md")) as f:
        return re.search(r"^x = tokens\[.*\]", f.read(), re.M).group(0)


def test_readme_gather_takes_routes_without_an_expert():
    # Positions past num_padded hold the sentinel M * k. Run on host tensors: an
    # index out of range is an exception there, and ends the process on a GPU.
    M, k = 3, 2
    tokens = torch.arange(M, dtype=torch.float32).unsqueeze(1).expand(M, 4)
    scope = dict(tokens=tokens, M=M, k=k, routes=torch.tensor([1, 2, 5, 6, 6, 6], dtype=torch.int32))
    exec(readme_gather(), scope)
    assert scope["x"].shape == (6, 4)
    assert scope["x"][:3, 0].tolist() == [0.0, 1.0, 2.0]
    no_tokens = dict(tokens=torch.empty(0, 4), M=0, k=k, routes=torch.empty(0, dtype=torch.int32))
    exec(readme_gather(), no_tokens)
    assert no_tokens["x"].shape == (0, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("M,E,shard,base", [(1, 8, 8, 0), (5, 16, 4, 12), (200, 16, 4, 8), (700, 64, 16, 0)])
def test_chain_of_a_shard(M, E, shard, base):
    # Experts base .. base + shard - 1 of E are here; IDs outside [0, E) occur too.
    # Forward, both gradients and the sums back into tokens, exact on whole numbers.
    k, N, K = 2, 72, 104
    print("[gpu-case] ragged chain of a shard", M, E, shard, base, flush=True)
    g = torch.Generator().manual_seed(M)
    ids = torch.stack([torch.randperm(E + 2, generator=g)[:k] - 1 for _ in range(M)]).to(torch.int32)
    x, w = R.whole(g, M, K), R.whole(g, shard, N, K)
    i32 = dict(dtype=torch.int32, device="cuda")
    cap = moe.moe_align_capacity(M, k, shard, 1)
    assert cap == M * k
    routes, blocks, num_padded, offsets = (torch.empty(n, **i32) for n in (cap, cap, 1, shard + 1))
    moe.moe_align_ex(ids.cuda(), shard, base, 1, routes, blocks, num_padded)
    moe.moe_align_offsets(blocks, num_padded, shard, 1, offsets)
    scope = dict(tokens=x.cuda().bfloat16(), M=M, k=k, routes=routes)
    exec(readme_gather(), scope)
    rows = scope["x"]
    wd = w.cuda().bfloat16()
    y, dx = torch.full((cap, N), 7.5, device="cuda"), torch.full((cap, K), 7.5, device="cuda")
    dw = torch.full((shard, N, K), 7.5, device="cuda")
    dy = R.whole(g, cap, N)
    dy[int((torch.isin(ids, torch.arange(base, base + shard, dtype=torch.int32))).sum()):] = float("nan")
    dyd = dy.cuda().bfloat16()
    moe.moe_grouped_matmul(rows, wd, offsets, y)
    moe.moe_grouped_matmul_dx(dyd, wd, offsets, dx)
    moe.moe_grouped_matmul_dw(dyd, rows, offsets, dw)
    torch.cuda.synchronize()

    flat = ids.flatten().long() - base
    here = ((flat >= 0) & (flat < shard)).nonzero().flatten()
    order = here[torch.sort(flat[here], stable=True).indices]
    n = order.numel()
    off = torch.cat((torch.zeros(1, dtype=torch.long), torch.bincount(flat[here], minlength=shard).cumsum(0)))
    assert torch.equal(offsets.cpu().long(), off) and torch.equal(routes[:n].cpu().long(), order)
    assert bool((routes[n:] == M * k).all())
    xr = x[order // k]
    assert torch.equal(y[:n].double().cpu(), R.forward(xr, w, off)) and bool((y[n:] == 7.5).all())
    assert torch.equal(dx[:n].double().cpu(), R.input_grad(dy[:n], w, off)) and bool((dx[n:] == 7.5).all())
    assert torch.equal(dw.double().cpu(), R.weight_grad(dy[:n], xr, off))


class Product(torch.autograd.Function):
    """What a training step writes around the raw calls."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        y = torch.zeros(x.shape[0], w.shape[1], dtype=x.dtype, device=x.device)
        moe.moe_grouped_matmul(x, w, offsets, y)
        ctx.save_for_backward(x, w, offsets)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx, dw = torch.zeros_like(x), torch.empty_like(w)
        moe.moe_grouped_matmul_dx(dy, w, offsets, dx)
        moe.moe_grouped_matmul_dw(dy, x, offsets, dw)
        return dx, dw, None


@pytest.mark.gpu
def test_training_step_of_an_expert_layer():
    # Two products with a threshold between them, gathered from and summed back into tokens, some routes
    # without an expert. Every value and gradient is a whole number up to 256, exact in bf16.
    M, k, E, H, I = 40, 2, 5, 24, 16
    print("[gpu-case] ragged training step", flush=True)
    g = torch.Generator().manual_seed(31)
    ids = torch.stack([torch.randperm(E + 1, generator=g)[:k] for _ in range(M)]).to(torch.int32)   # E is no expert

    def sparse(*shape):
        return (torch.randint(-1, 2, shape, generator=g) * (torch.rand(*shape, generator=g) < 0.3)).double()

    x, w1, w2, dy = sparse(M, H), sparse(E, I, H), sparse(E, H, I), sparse(M, H)

    i32 = dict(dtype=torch.int32, device="cuda")
    routes, blocks, num_padded, offsets = (torch.empty(n, **i32) for n in (M * k, M * k, 1, E + 1))
    moe.moe_align(ids.cuda(), E, 1, routes, blocks, num_padded)
    moe.moe_align_offsets(blocks, num_padded, E, 1, offsets)
    leaves = [t.cuda().bfloat16().requires_grad_() for t in (x, w1, w2)]
    token = (routes // k).clamp(max=M - 1).long()
    live = (routes < M * k).unsqueeze(1)
    a = Product.apply(leaves[0][token], leaves[1], offsets).relu()
    y = torch.zeros(M, H, device="cuda").index_add(0, token, Product.apply(a, leaves[2], offsets).float() * live)
    y.backward(dy.cuda().float())

    ref = [t.clone().requires_grad_() for t in (x, w1, w2)]
    out = torch.zeros(M, H, dtype=torch.float64)
    for r, e in enumerate(ids.flatten().tolist()):
        if e < E:
            out = out.index_add(0, torch.tensor([r // k]), (ref[2][e] @ (ref[1][e] @ ref[0][r // k]).relu()).unsqueeze(0))
    out.backward(dy)
    largest = max(float(t.detach().abs().max()) for t in (out, *(r.grad for r in ref)))
    assert 4 < largest <= 256                # what bf16 holds exactly
    assert torch.equal(y.detach().double().cpu(), out.detach())
    for t, r in zip(leaves, ref):
        assert torch.equal(t.grad.double().cpu(), r.grad)
