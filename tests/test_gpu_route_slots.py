"""Routing and its gradient with 9 to 16 slots, and from few groups: sixteen
lanes a row, of which each may hold several of the chosen."""
import itertools

import numpy as np
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _route as R
from tests.test_gpu_route import BF16, F16, F32, INF, announce, check, check_grad, route, shape_id

pytestmark = pytest.mark.gpu

# E, k, groups, groups kept
SHAPES = [(16, 16, 1, 1), (17, 16, 1, 1), (20, 15, 1, 1), (64, 10, 1, 1), (64, 16, 1, 1), (100, 13, 1, 1), (128, 12, 1, 1),
          (128, 16, 1, 1), (256, 11, 1, 1), (256, 14, 1, 1), (256, 16, 1, 1), (500, 15, 1, 1), (512, 16, 1, 1),
          (256, 6, 8, 1), (256, 8, 8, 1), (256, 5, 16, 2), (256, 9, 8, 2), (256, 16, 8, 2), (256, 12, 8, 4), (256, 16, 8, 4),
          (160, 12, 8, 3), (160, 16, 8, 3), (128, 16, 8, 1), (126, 13, 9, 4), (384, 16, 3, 1), (512, 4, 16, 1),
          (512, 16, 16, 1), (480, 16, 16, 3), (256, 16, 2, 1), (60, 14, 4, 2), (72, 9, 6, 2), (96, 15, 3, 2)]


@pytest.mark.parametrize("shape", SHAPES, ids=shape_id)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_random_logits(shape, score, dtype):
    # bf16 has equal logits in most rows, and without a bias (or with one of zeros) ties for the last slot.
    E, k, G, kept = shape
    g = torch.Generator().manual_seed(E * 100 + k)
    for M, bias, top in ((37, None, 1), (40, 0.2, 2), (33, None, 2), (35, 0.0, 1)):
        logits = (2 * torch.randn(M, E, generator=g)).to(dtype)
        b = None if bias is None else bias * torch.randn(E, generator=g)
        announce("route slots", shape, score, dtype, M, bias, top)
        check(logits, k, b, pad=M % 4, score=score, renormalize=M % 2 == 0, scale=1.5, groups=G, topk_groups=kept,
              group_top=top)


def in_order(ids, logits, k, score, bias, groups, topk_groups, group_top):
    """Whether ids [k] of one row is an order that 64-bit evaluations of the choice values can give.

    An evaluation is off by the exponential's last place (2^-52), by its argument's rounding (2^-53 of the argument's
    size, a summand of the exponent), by the sum's E additions and the division (2^-53 each), all relative to the
    score, and by the bias's addition (2^-53 of the result). A comparison has two values, and the reference and the
    kernel each evaluate them: values closer than `eps`, the four together, have no order of their own. Without a bias
    that is so for the groups' sums of scores alone: experts are chosen by their logits."""
    l = logits.double().numpy()
    s = R.scores(logits.unsqueeze(0), score)[0].numpy()
    b = np.zeros_like(l) if bias is None else bias.double().numpy()
    c = s + b
    live = (l > -np.inf) & (b > -np.inf)
    if not np.isfinite(c[live]).all():
        return False
    x = l.max() - l if score == R.SOFTMAX else np.abs(l)
    off = 2.0 ** -53 * (s * (4 + np.minimum(x, 1e3) + (len(l) if score == R.SOFTMAX else 0)) + np.abs(c))
    eps = 4 * float(off[live].max(initial=0.0))
    of = np.arange(len(l)) // (len(l) // groups)
    kept = [set(range(groups))]
    if topk_groups < groups:
        rank = np.array([np.sort(c[(of == g) & live])[::-1][:group_top].sum() if ((of == g) & live).any() else -np.inf
                         for g in range(groups)])
        edge = np.sort(rank)[::-1][topk_groups - 1]
        sure = {g for g in range(groups) if rank[g] > edge + 2 * eps}
        open_ = [g for g in range(groups) if abs(rank[g] - edge) <= 2 * eps or rank[g] == edge]
        kept = [sure | set(more) for more in itertools.combinations(open_, topk_groups - len(sure))]
    ids = [e for e in ids.tolist() if e >= 0]
    if bias is None:
        c, eps = l, 0.0
    for groups_kept in kept:
        mine = live & np.isin(of, list(groups_kept))
        best = np.sort(c[mine])[::-1][:k]
        if len(set(ids)) == len(ids) == len(best) and mine[ids].all() and (np.abs(c[ids] - best) <= eps).all():
            return True
    return False


def check_order(logits, k, bias, score, renormalize, groups, topk_groups, group_top):
    """check, but for rows whose order is a matter of the last places of 64-bit arithmetic."""
    kw = dict(groups=groups, topk_groups=topk_groups, group_top=group_top)
    ids, w = route(logits, k, bias, score=score, renormalize=renormalize, **kw)
    want = R.choose(logits, k, score, bias, **kw)
    other = (ids != want).any(1).nonzero().flatten().tolist()
    for t in other:
        assert in_order(ids[t], logits[t], k, score, bias, **kw), (t, ids[t], want[t])
    ref = R.weights(logits, ids, score, renormalize, 1.0)
    bad = (w.double() - ref).abs() > R.weight_bound(logits, logits.shape[1] / 16 + k) * ref.abs() + 1e-37
    assert not bool((bad | (w.isnan() != ref.isnan())).any()), (w[bad.any(1)][:4], ref[bad.any(1)][:4])


@pytest.mark.parametrize("shape", SHAPES, ids=shape_id)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
def test_ties_masks_and_close_experts(shape, score):
    E, k, G, kept = shape
    g = torch.Generator().manual_seed(E + k)
    kw = dict(score=score, groups=G, topk_groups=kept)
    few = torch.randint(0, 3, (20, E), generator=g).float()                       # equal to a third of the row
    close = 0.5 + torch.randint(0, 40, (20, E), generator=g) * 2.0 ** -24          # a few fp32 steps apart
    masked = torch.randn(24, E, generator=g)
    masked[torch.rand(24, E, generator=g) < torch.linspace(0, 1, 24).unsqueeze(1)] = -INF
    # the largest in one lane's share, and far below the rest
    run = torch.randn(18, E, generator=g)
    for t in range(18):
        first = (t * E) // 20
        run[t, first:first + 14] += 30.0
    wide = torch.randn(12, E, generator=g) * torch.logspace(-30, 30, 12).unsqueeze(1)
    announce("route slots, ties", shape, score)
    for logits in (few, close, masked, run, wide):
        for b in (None, torch.zeros(E), 0.25 * torch.randn(E, generator=g), 1e4 * torch.randn(E, generator=g)):
            check_order(logits, k, b, renormalize=True, group_top=2, **kw)


@pytest.mark.parametrize("shape", SHAPES, ids=shape_id)
def test_nan_infinite_and_lowest_values(shape):
    # Their rows are routed as any, and rows beside them (of the same wave) as without them.
    E, k, G, kept = shape
    g = torch.Generator().manual_seed(7 * E + k)
    logits = torch.randn(23, E, generator=g)
    logits[1, E // 3], logits[5, ::3], logits[6, 1::2] = float("nan"), INF, torch.finfo(F32).min
    logits[9], logits[10, E // 2:] = torch.finfo(F32).max, torch.finfo(F32).max
    bias = 0.1 * torch.randn(E, generator=g)
    bias[::5], bias[1::7], bias[2::9] = INF, -INF, torch.finfo(F32).min
    announce("route slots, extremes", shape)
    for b in (None, bias):
        for top in (1, 2):
            kw = dict(groups=G, topk_groups=kept, group_top=top)
            ids, _ = route(logits, k, b, score=R.SIGMOID, **kw)
            want = R.choose(logits, k, R.SIGMOID, b, **kw)
            assert torch.equal(ids, want), (ids[(ids != want).any(1)][:4], want[(ids != want).any(1)][:4])


@pytest.mark.parametrize("E,k", [(9, 9), (64, 10), (128, 12), (160, 16), (256, 9), (256, 16), (511, 15), (512, 16)])
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradients(E, k, score, renormalize):
    gen = torch.Generator().manual_seed(E + k)
    for M, dtype, out in ((1, F32, F32), (35, BF16, BF16), (66, F16, F32)):
        logits = (1.5 * torch.randn(M, E, generator=gen)).to(dtype)
        ids = R.choose(logits, k, score)
        g = torch.randn(M, k, generator=gen)
        announce("route grad slots", E, k, score, renormalize, M)
        check_grad(logits, ids, g, score, renormalize, 2.5, out, pad=M % 5)
        ids[:, 3], g[:, 3] = -1, float("nan")                       # a slot without an expert
        ids[:, 1] = ids[:, k - 1]                                   # an expert named twice, by the last slot
        check_grad(logits, ids, g, score, renormalize, 1.0, out)


def time_of(E, k, G, kept, bias, score):
    """us a call of 32768 tokens, over changing logits, the least of several graphs' replays."""
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = [torch.randn(32768, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
              for _ in range(2)]
    b = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
    ids, w = torch.empty(32768, k, dtype=torch.int32, device="cuda"), torch.empty(32768, k, device="cuda")

    def calls():
        for _ in range(4):
            for l in logits:
                moe.moe_route(l, ids, w, bias=b, score=score, groups=G, topk_groups=kept, group_top=2 if bias else 1)

    calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    graph.replay()
    best = float("inf")
    for _ in range(6):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        graph.replay()
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end) * 1e3 / 8)
    return best


@pytest.mark.parametrize("bias,score", [(True, R.SIGMOID), (False, R.SOFTMAX)], ids=["bias", "none"])
@pytest.mark.parametrize("E,k,G,kept", [(256, 16, 1, 1), (128, 16, 1, 1), (256, 16, 8, 4), (256, 12, 8, 2), (256, 6, 8, 1),
                                        (512, 4, 16, 1)])
def test_many_slots_take_the_same_path(E, k, G, kept, bias, score):
    # Rows whose candidates do not fit sixteen lanes go one by one, at four to ten times the cost of the rest. With
    # up to sixteen slots that is for equal and nearly equal experts alone: a call costs what its other parts do.
    announce("route cost", E, k, G, kept, bias)
    base, t = time_of(E, 2, G, kept, bias, score), time_of(E, k, G, kept, bias, score)
    print("us:", base, t, flush=True)
    assert t < 2.5 * base
