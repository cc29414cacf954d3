"""Routing to experts (moe_route) and its gradient (moe_route_grad) against
64-bit references: the choice equal, weights and gradients within the bounds of
fp32 arithmetic; ties, masks, infinities, NaN, strides, streams, graphs."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _route as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = float("inf")


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


def route(logits, k, bias=None, pad=0, **kw):
    """(ids, weights) of the kernel on the host, from a row stride of E + pad."""
    M, E = logits.shape
    wide = torch.full((M, E + pad), float("nan"), dtype=logits.dtype, device="cuda")
    wide[:, :E] = logits.cuda()
    ids = torch.full((M, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((M, k), float("nan"), device="cuda")
    moe.moe_route(wide[:, :E], ids, w, bias=None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    return ids.cpu(), w.cpu()


def check(logits, k, bias=None, pad=0, score=R.SOFTMAX, renormalize=True, scale=1.0, **groups):
    ids, w = route(logits, k, bias, pad, score=score, renormalize=renormalize, scale=scale, **groups)
    want = R.choose(logits, k, score, bias, **groups)
    assert torch.equal(ids, want), (ids[(ids != want).any(1)][:4], want[(ids != want).any(1)][:4])
    ref = R.weights(logits, want, score, renormalize, scale)
    bad = (w.double() - ref).abs() > R.weight_bound(logits, logits.shape[1] / 16 + k) * ref.abs() + 1e-37 * abs(scale)
    assert not bool((bad | (w.isnan() != ref.isnan())).any()), (w[bad.any(1)][:4], ref[bad.any(1)][:4])


# E, k, groups, topk_groups: one expert, fewer experts than lanes, odd counts, groups that lanes do not
# divide, groups of one expert, the most experts, slots and groups.
SHAPES = [(1, 1, 1, 1), (2, 1, 1, 1), (7, 7, 1, 1), (8, 2, 1, 1), (16, 4, 4, 2), (60, 4, 1, 1), (64, 6, 8, 3),
          (65, 9, 1, 1), (72, 6, 6, 2), (126, 5, 9, 4), (128, 8, 1, 1), (160, 6, 8, 3), (256, 8, 8, 4), (256, 8, 1, 1),
          (256, 17, 16, 5), (257, 8, 1, 1), (40, 12, 40, 20), (64, 20, 64, 33), (512, 22, 1, 1), (384, 8, 3, 1),
          (1000, 64, 50, 7), (2048, 10, 1, 1), (2048, 64, 64, 40)]


def shape_id(s):
    return "E%d_k%d_G%d_of%d" % s


@pytest.mark.parametrize("shape", SHAPES, ids=shape_id)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_routes_of_random_logits(shape, score, dtype):
    E, k, G, kept = shape
    g = torch.Generator().manual_seed(E * 100 + k)
    for M, renormalize, with_bias, top in ((1, True, False, 1), (37, False, True, 2), (66, True, True, 1),
                                           (5, True, False, 2)):
        logits = (2 * torch.randn(M, E, generator=g)).to(dtype)
        bias = 0.2 * torch.randn(E, generator=g) if with_bias else None
        announce("route", shape, score, dtype, M, renormalize, with_bias, top)
        check(logits, k, bias, pad=M % 7, score=score, renormalize=renormalize, scale=2.5 if with_bias else 1.0,
              groups=G, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("shape", SHAPES[3:], ids=shape_id)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(shape, score):
    E, k, G, kept = shape
    g = torch.Generator().manual_seed(2)
    for values, bias in ((1, None), (2, None), (3, torch.zeros(E)), (2, torch.randint(0, 2, (E,), generator=g) * 0.5)):
        logits = torch.randint(0, values, (33, E), generator=g).float()
        announce("route ties", shape, score, values)
        for top in (1, 2):
            check(logits, k, bias, score=score, groups=G, topk_groups=kept, group_top=top)
    # -0 is 0
    logits = torch.where(torch.rand(9, E, generator=g) < 0.5, -0.0, 0.0)
    check(logits, k, None, score=score, groups=G, topk_groups=kept, group_top=1)


@pytest.mark.parametrize("shape", SHAPES, ids=shape_id)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_experts(shape, score, renormalize):
    # From no expert masked to all of them: rows with fewer than k experts, and with none.
    E, k, G, kept = shape
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(24, E, generator=g)
    off = torch.rand(24, E, generator=g) < torch.linspace(0, 1, 24).unsqueeze(1)
    off[-1] = True
    logits[off] = -INF
    bias = 0.1 * torch.randn(E, generator=g)
    for b, top in ((None, 1), (None, 2), (bias, 2)):
        announce("route masked", shape, score, renormalize, top, b is not None)
        check(logits, k, b, score=score, renormalize=renormalize, groups=G, topk_groups=kept, group_top=top)
    bias[::2] = -INF
    check(logits, k, bias, score=score, renormalize=renormalize, groups=G, topk_groups=kept, group_top=2)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,kept", [(16, 1, 1), (128, 1, 1), (256, 8, 4), (300, 1, 1)])
def test_close_experts_keep_their_order(score, E, G, kept):
    # Logits a few fp32 steps apart: their scores round to the same fp32 values, yet have an order. Half
    # the rows are near 0, half where the sigmoid saturates in fp32 (1 - 2^-25 and above).
    g = torch.Generator().manual_seed(4)
    step = torch.randint(0, 40, (64, E), generator=g).float()
    near = 0.5 + step * 2.0 ** -24
    far = 18.0 + step * 2.0 ** -19
    logits = torch.cat((near, far))
    announce("route close", score, E, G)
    for bias in (None, torch.zeros(E), torch.full((E,), -0.25)):
        for top in (1, 2):
            check(logits, 8, bias, score=score, renormalize=True, groups=G, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
def test_extreme_logits(score, dtype):
    lowest, largest = torch.finfo(dtype).min, torch.finfo(dtype).max
    rows = torch.zeros(8, 24)
    rows[0] = lowest                                     # a mask of the type's lowest value: still an expert
    rows[1, ::3] = lowest
    rows[2] = -80.0 - torch.arange(24)                   # small scores keep their ratio
    rows[3] = torch.arange(24) * 30.0
    rows[4, 5] = largest
    rows[5] = -1000.0
    rows[5, 3] = -990.0
    rows[6] = torch.linspace(-20, 20, 24)
    rows[7, 1:] = -60000.0
    announce("route extreme", score, dtype)
    for renormalize in (True, False):
        check(rows.to(dtype), 6, score=score, renormalize=renormalize)
    check(rows.to(dtype), 3, torch.linspace(-1, 1, 24), score=score, renormalize=False, groups=4, topk_groups=2,
          group_top=2)


def test_nan_and_infinite_logits_show():
    # A NaN ranks above every number; its weights are NaN. Other rows are as without it.
    g = torch.Generator().manual_seed(5)
    for E, groups in ((40, {}), (128, dict(groups=8, topk_groups=3, group_top=2)), (256, {})):
        logits = torch.randn(6, E, generator=g)
        logits[1, E // 2] = float("nan")
        logits[3, 7] = INF
        logits[4, :] = float("nan")
        bias = 0.1 * torch.randn(E, generator=g)
        announce("route nan", E)
        for b in (None, bias):
            ids, w = route(logits, 4, b, score=R.SIGMOID, **groups)
            assert torch.equal(ids, R.choose(logits, 4, R.SIGMOID, b, **dict(dict(groups=1, topk_groups=1, group_top=1),
                                                                              **groups)))
            assert int(ids[1, 0]) == E // 2 and bool(w[1].isnan().all()) and bool(w[4].isnan().all())
            assert not bool(w[[0, 2, 3, 5]].isnan().any())
            if b is None:
                assert int(ids[3, 0]) == 7
        ids, w = route(logits, 4, None, score=R.SOFTMAX, renormalize=False)
        assert bool(w[1].isnan().all()) and not bool(w[[0, 2, 5]].isnan().any())
        bias[3], bias[5] = INF, float("nan")
        ids, w = route(logits[:1], 4, bias, score=R.SIGMOID, **groups)
        assert ids[0, :2].tolist() == [5, 3] and not bool(w.isnan().any())


@pytest.mark.parametrize("E,G,kept", [(64, 8, 3), (256, 8, 4), (512, 16, 5), (96, 32, 9)])
@pytest.mark.parametrize("bias", [False, True])
def test_softmax_of_nan_and_infinite_logits_in_groups(E, G, kept, bias):
    # One such logit makes all scores of its row NaN: groups are equal, the lowest ones kept.
    g = torch.Generator().manual_seed(6)
    logits = torch.randn(7, E, generator=g)
    logits[1, E - 2], logits[2, 3], logits[4, E // 2], logits[4, 1], logits[5, ::2] = float("nan"), INF, INF, float("nan"), -INF
    b = 0.1 * torch.randn(E, generator=g) if bias else None
    announce("route nan groups", E, G, bias)
    for top in (1, 2):
        kw = dict(groups=G, topk_groups=kept, group_top=top)
        ids, w = route(logits, 5, b, score=R.SOFTMAX, renormalize=False, **kw)
        want = R.choose(logits, 5, R.SOFTMAX, b, **kw)
        assert torch.equal(ids, want), (ids, want)
        assert bool(w[[1, 2, 4]].isnan().all()) and not bool(w[[0, 3, 5, 6]].isnan().any())


GRAD_SHAPES = [(1, 1), (2, 2), (8, 2), (60, 4), (127, 3), (128, 8), (160, 6), (256, 8), (257, 17), (1000, 64),
               (2048, 10)]


def grad(logits, ids, g, out=None, pad=0, **kw):
    M, E = logits.shape
    wide = torch.full((M, E + pad), float("nan"), dtype=logits.dtype, device="cuda")
    wide[:, :E] = logits.cuda()
    d = torch.full((M, E + 2 * pad), 77.0, dtype=out or logits.dtype, device="cuda")
    moe.moe_route_grad(wide[:, :E], ids.cuda(), g.cuda(), d[:, :E], **kw)
    torch.cuda.synchronize()
    assert bool((d[:, E:] == 77.0).all())
    return d[:, :E].cpu()


def check_grad(logits, ids, g, score, renormalize, scale, out=None, pad=0):
    got = grad(logits, ids, g, out, pad, score=score, renormalize=renormalize, scale=scale)
    valid = torch.where((ids >= 0) & (ids < logits.shape[1]), ids, -1)
    ref, mag = R.logits_grad(logits, valid, torch.nan_to_num(g), score, renormalize, scale)
    ref = torch.where((valid >= 0).any(1, keepdim=True), ref, torch.zeros_like(ref))
    mag = torch.where((valid >= 0).any(1, keepdim=True), mag, torch.zeros_like(mag))
    half = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[got.dtype]
    tiny = 2.0 ** -25 if got.dtype == F16 else 1e-37
    # The reference goes through the whole softmax: where renormalising cancels a derivative exactly it keeps
    # the rounding of its 64-bit terms, a few 2^-53 of the row's (each at most the row's magnitudes' sum).
    tiny = tiny + 8 * 2.0 ** -53 * mag.sum(1, keepdim=True)
    # the factors' errors (twice a weight's: scores and shares), then one rounding
    bound = 2 * R.weight_bound(logits, logits.shape[1] / 16 + 2 * ids.shape[1]) * mag + half * ref.abs() + tiny
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), (got[bad][:4], ref[bad][:4], bound[bad][:4])


@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=lambda s: "E%d_k%d" % s)
@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradients(shape, score, renormalize):
    E, k = shape
    gen = torch.Generator().manual_seed(E + k)
    for M, dtype, out in ((1, F32, F32), (35, BF16, BF16), (66, F16, F32), (4, F16, F16), (67, F32, F32),
                          (3, BF16, F32)):
        logits = (1.5 * torch.randn(M, E, generator=gen)).to(dtype)
        ids = R.choose(logits, k, score)
        g = torch.randn(M, k, generator=gen)
        announce("route grad", shape, score, renormalize, M, dtype)
        check_grad(logits, ids, g, score, renormalize, 2.5 if M > 40 else 1.0, out, pad=M % 5)
        # routes without an expert, in some rows all of them; their gradients are not read
        off = torch.rand(M, k, generator=gen) < torch.linspace(0, 1, M).unsqueeze(1)
        off[-1] = True
        ids = torch.where(off, torch.where(torch.rand(M, k, generator=gen) < 0.5, -1, E + 3), ids).to(torch.int32)
        g[off] = float("nan")
        check_grad(logits, ids, g, score, renormalize, 1.0, out)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_repeated_and_masked_experts(score, renormalize):
    gen = torch.Generator().manual_seed(8)
    logits = torch.randn(20, 48, generator=gen)
    ids = torch.randint(0, 6, (20, 7), generator=gen).to(torch.int32)     # repeated in every row
    announce("route grad repeated", score, renormalize)
    check_grad(logits, ids, torch.randn(20, 7, generator=gen), score, renormalize, 1.0)
    logits[:, 40:] = -INF                                                  # no gradient for masked experts
    logits[:, 30] = -120.0
    ids = R.choose(logits, 5, score)
    check_grad(logits, ids, torch.randn(20, 5, generator=gen), score, renormalize, 1.0)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(score, renormalize):
    # Central differences of the 64-bit weights with the choice held: off by h^2 / 6 times a third
    # derivative (weights and their derivatives are of order one) and 2^-52 / h.
    gen = torch.Generator().manual_seed(9)
    M, E, k, h = 3, 21, 4, 1e-5
    logits = torch.randn(M, E, generator=gen)
    ids = R.choose(logits, k, score)
    g = torch.randn(M, k, generator=gen)
    announce("route grad differences", score, renormalize)
    got = grad(logits, ids, g, score=score, renormalize=renormalize, scale=1.5).double()
    for e in range(E):
        up, down = logits.double(), logits.double()
        up[:, e] += h
        down[:, e] -= h
        d = (R.weights(up, ids, score, renormalize, 1.5) - R.weights(down, ids, score, renormalize, 1.5)) / (2 * h)
        assert bool(((d * g.double()).sum(1) - got[:, e]).abs().max() < 1e-5)


def test_no_tokens():
    logits = torch.empty(0, 16, device="cuda")
    ids, w = torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda")
    announce("route empty")
    assert moe.moe_route(logits, ids, w) == moe.MOE_OK
    assert moe.moe_route_grad(logits, ids, w, logits.clone()) == moe.MOE_OK


@pytest.mark.parametrize("E,G,kept,bias", [(128, 1, 1, False), (256, 8, 4, True)])
def test_many_tokens_match_few(E, G, kept, bias):
    # A token's routes and gradient do not depend on the batch it is in.
    g = torch.Generator().manual_seed(10)
    logits = torch.randn(9001, E, generator=g).cuda()
    b = 0.1 * torch.randn(E, generator=g).cuda() if bias else None
    kw = dict(score=R.SIGMOID if bias else R.SOFTMAX)
    ids, w = torch.empty(9001, 8, dtype=torch.int32, device="cuda"), torch.empty(9001, 8, device="cuda")
    d = torch.empty_like(logits)
    announce("route many", E)
    moe.moe_route(logits, ids, w, bias=b, groups=G, topk_groups=kept, group_top=2, **kw)
    moe.moe_route_grad(logits, ids, w, d, **kw)
    for a, z in ((0, 1), (17, 18), (4000, 4037), (8999, 9001)):
        i2, w2 = torch.empty_like(ids[a:z]), torch.empty_like(w[a:z])
        d2 = torch.empty_like(d[a:z])
        moe.moe_route(logits[a:z], i2, w2, bias=b, groups=G, topk_groups=kept, group_top=2, **kw)
        moe.moe_route_grad(logits[a:z], i2, w2, d2, **kw)
        assert torch.equal(i2, ids[a:z]) and torch.equal(w2, w[a:z]) and torch.equal(d2, d[a:z])


def test_graph_and_two_streams():
    g = torch.Generator().manual_seed(11)
    logits = torch.randn(70, 256, generator=g).cuda()
    bias = (0.1 * torch.randn(256, generator=g)).cuda()
    kw = dict(score=R.SIGMOID, scale=2.5)
    gr = dict(groups=8, topk_groups=4, group_top=2)

    def call(s=None):
        moe.moe_route(logits, ids, w, bias=bias, stream=s, **kw, **gr)
        moe.moe_route_grad(logits, ids, w, d, stream=s, **kw)

    ids, w = torch.empty(70, 8, dtype=torch.int32, device="cuda"), torch.empty(70, 8, device="cuda")
    d = torch.empty_like(logits)
    announce("route graph")
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        logits.copy_(torch.randn(70, 256, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = ids.clone(), w.clone(), d.clone()
        ids.fill_(-9), w.zero_(), d.zero_()
        call()
        assert torch.equal(got[0], ids) and torch.equal(got[1], w) and torch.equal(got[2], d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(got[0], ids) and torch.equal(got[1], w) and torch.equal(got[2], d)
