"""Host-only checks of routing, the weighted sum of routes and the products with
packed 4-bit weights: bad arguments are refused by the C ABI before anything is
enqueued; and the references the GPU tests hold the kernels to."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_align_amd import _binding as B
from tests import _route as R

FAKE = 0x10000  # aligned, non-null; never dereferenced on these paths
INV, UNS, OK = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_OK
F32, BF16, F16 = B.MOE_DTYPE_F32, B.MOE_DTYPE_BF16, B.MOE_DTYPE_F16


def rdesc(M=3, E=16, k=2, dtype=F32, score=0, renormalize=1, scale=1.0, groups=4, topk_groups=2, group_top=2):
    return B.moe_route_desc(M, E, k, dtype, score, renormalize, scale, groups, topk_groups, group_top)


def route(d, logits=FAKE, ld=None, bias=FAKE, ids=FAKE, w=FAKE):
    return B.lib().moe_route(ctypes.byref(d), logits, d.E if ld is None else ld, bias, ids, w, None)


def rgrad(d, logits=FAKE, ld=None, ids=FAKE, w=FAKE, out=F32, dl=FAKE, ldd=None):
    return B.lib().moe_route_grad(ctypes.byref(d), logits, d.E if ld is None else ld, ids, w, out, dl,
                                  d.E if ldd is None else ldd, None)


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), INV), (dict(E=0, k=0), INV), (dict(k=0), INV), (dict(k=17), INV), (dict(dtype=3), INV),
    (dict(dtype=-1), INV), (dict(score=2), INV), (dict(score=-1), INV), (dict(groups=0), INV), (dict(groups=5), INV),
    (dict(groups=-4), INV), (dict(topk_groups=0), INV), (dict(topk_groups=5), INV), (dict(group_top=0), INV),
    (dict(group_top=3), INV), (dict(k=9), INV), (dict(E=2049, groups=1, topk_groups=1), UNS),
    (dict(E=256, k=65, groups=1, topk_groups=1), UNS), (dict(E=130, groups=65, topk_groups=65), UNS),
    (dict(M=2 ** 31 - 1), UNS)], ids=str)
@pytest.mark.parametrize("call", [route, rgrad], ids=lambda c: c.__name__)
def test_routing_refuses_bad_descriptions(call, bad, status):
    assert call(rdesc(**bad)) == status


def test_routing_refuses_bad_pointers_and_strides():
    null = ctypes.POINTER(B.moe_route_desc)()
    assert B.lib().moe_route(null, FAKE, 16, FAKE, FAKE, FAKE, None) == INV
    assert B.lib().moe_route_grad(null, FAKE, 16, FAKE, FAKE, 0, FAKE, 16, None) == INV
    d = rdesc()
    for a in ("logits", "ids", "w"):
        for call in (route, rgrad):
            assert call(d, **{a: None}) == INV and call(d, **{a: FAKE + 2}) == INV, a
    assert route(d, bias=FAKE + 2) == INV and rgrad(d, dl=None) == INV and rgrad(d, dl=FAKE + 2) == INV
    for call in (route, rgrad):
        assert call(d, ld=15) == INV and call(d, ld=(1 << 22) + 1) == UNS and call(d, ld=-16) == INV
        assert call(rdesc(dtype=BF16), logits=FAKE + 1) == INV
    assert rgrad(d, ldd=15) == INV and rgrad(d, ldd=(1 << 22) + 1) == UNS
    assert rgrad(d, out=BF16) == INV and rgrad(rdesc(dtype=BF16), out=F16) == INV and rgrad(d, out=3) == INV


def test_no_tokens_is_a_no_op_without_pointers():
    assert route(rdesc(M=0), logits=None, bias=None, ids=None, w=None) == OK
    assert rgrad(rdesc(M=0), logits=None, ids=None, w=None, dl=None) == OK
    assert combine(cdesc(M=0), None, y=None) == OK and cgrad(cdesc(M=0), dy=None, drows=None) == OK
    assert matvec(mdesc(M=0), x=None, y=None) == OK and matvec(mdesc(M=0, E=4, k=2), ids=None) == OK
    assert positions(None, None, 0, 0, None) == OK


def cdesc(M=3, k=2, H=16, rows=6, dtype=BF16, y=F32):
    return B.moe_combine_desc(M, k, H, rows, dtype, y)


def combine(d, rows=FAKE, ldr=None, pos=FAKE, w=FAKE, y=FAKE, ldy=None):
    return B.lib().moe_combine(ctypes.byref(d), rows, d.H if ldr is None else ldr, pos, w, y,
                               d.H if ldy is None else ldy, None)


def cgrad(d, dy=FAKE, lddy=None, rows=FAKE, ldr=None, pos=FAKE, w=FAKE, drows=FAKE, lddr=None, dw=FAKE):
    return B.lib().moe_combine_grad(ctypes.byref(d), dy, d.H if lddy is None else lddy, rows,
                                    d.H if ldr is None else ldr, pos, w, drows, d.H if lddr is None else lddr, dw, None)


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), INV), (dict(k=0), INV), (dict(H=0), INV), (dict(H=12), INV), (dict(rows=-1), INV),
    (dict(dtype=3), INV), (dict(y=3), INV), (dict(H=(1 << 20) + 8), UNS), (dict(rows=2 ** 31 - 1), UNS),
    (dict(M=2 ** 30, k=2), UNS)], ids=str)
@pytest.mark.parametrize("call", [combine, cgrad], ids=lambda c: c.__name__)
def test_sums_refuse_bad_descriptions(call, bad, status):
    assert call(cdesc(**bad)) == status


def test_sums_refuse_bad_pointers_and_strides():
    null = ctypes.POINTER(B.moe_combine_desc)()
    assert B.lib().moe_combine(null, FAKE, 16, FAKE, FAKE, FAKE, 16, None) == INV
    assert B.lib().moe_combine_grad(null, FAKE, 16, FAKE, 16, FAKE, FAKE, FAKE, 16, FAKE, None) == INV
    d = cdesc()
    for call, names in ((combine, (("rows", "ldr"), ("y", "ldy"))),
                        (cgrad, (("dy", "lddy"), ("rows", "ldr"), ("drows", "lddr")))):
        for a, ld in names:
            assert call(d, **{a: None}) == INV and call(d, **{a: FAKE + 8}) == INV, a
            assert call(d, **{ld: 8}) == INV and call(d, **{ld: 20}) == INV and call(d, **{ld: (1 << 22) + 8}) == UNS
        assert call(d, pos=FAKE + 2) == INV and call(d, w=FAKE + 1) == INV
    assert cgrad(d, dw=FAKE + 2) == INV


def positions(routes, n, capacity, count, out):
    return B.lib().moe_align_positions(routes, n, capacity, count, out, None)


def test_positions_refuse_bad_arguments():
    assert positions(FAKE, FAKE, 4, -1, FAKE) == INV
    assert positions(None, FAKE, 4, 4, FAKE) == INV and positions(FAKE, None, 4, 4, FAKE) == INV
    assert positions(FAKE, FAKE, 4, 4, None) == INV
    assert positions(FAKE + 2, FAKE, 4, 4, FAKE) == INV and positions(FAKE, FAKE + 1, 4, 4, FAKE) == INV
    assert positions(FAKE, FAKE, 4, 4, FAKE + 2) == INV
    assert positions(FAKE, FAKE, 2 ** 31 - 1, 4, FAKE) == UNS and positions(FAKE, FAKE, 4, 2 ** 31 - 1, FAKE) == UNS
    assert positions(FAKE, FAKE, 2 ** 40, 4, FAKE) == UNS


def mdesc(M=2, k=1, E=1, N=24, K=64, dtype=BF16, out=F32, fmt=B.MOE_W_INT4_AWQ, group=32, q=FAKE, scale=FAKE, zero=FAKE):
    return B.moe_matvec_desc(M, k, E, N, K, dtype, out, B.moe_weights(fmt, group, q, scale, zero))


def matvec(d, x=FAKE, ldx=None, ids=None, y=FAKE, ldy=None):
    return B.lib().moe_matvec_int4(ctypes.byref(d), x, d.K if ldx is None else ldx, ids, y,
                                   d.N if ldy is None else ldy, None)


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), INV), (dict(k=0), INV), (dict(E=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(dtype=F32), INV),
    (dict(dtype=F16, out=BF16), INV), (dict(out=3), INV), (dict(fmt=B.MOE_W_MXFP8), UNS), (dict(fmt=7), INV),
    (dict(group=0), INV), (dict(group=16), INV), (dict(group=48, K=96), INV), (dict(group=64, K=96), INV),
    (dict(group=-32), INV), (dict(k=2), INV), (dict(E=2), INV), (dict(E=2049), UNS), (dict(N=(1 << 20) + 1), UNS),
    (dict(K=(1 << 20) + 32), UNS), (dict(M=2 ** 31 - 1), UNS), (dict(M=2 ** 24, N=1 << 20), UNS),
    (dict(q=None), INV), (dict(scale=None), INV), (dict(q=FAKE + 8), INV), (dict(scale=FAKE + 1), INV)], ids=str)
def test_matvec_refuses_bad_descriptions(bad, status):
    assert matvec(mdesc(**bad)) == status


def test_matvec_refuses_bad_pointers_and_strides():
    assert B.lib().moe_matvec_int4(ctypes.POINTER(B.moe_matvec_desc)(), FAKE, 64, None, FAKE, 24, None) == INV
    d = mdesc()
    assert matvec(d, x=None) == INV and matvec(d, x=FAKE + 8) == INV and matvec(d, ldx=56) == INV
    assert matvec(d, ldx=68) == INV and matvec(d, ldx=(1 << 22) + 8) == UNS
    assert matvec(d, y=None) == INV and matvec(d, y=FAKE + 2) == INV and matvec(d, ldy=23) == INV
    assert matvec(d, ldy=(1 << 22) + 1) == UNS and matvec(mdesc(out=BF16), y=FAKE + 1) == INV
    assert matvec(mdesc(E=4, k=2), ids=FAKE + 2) == INV


# ---- the references ----

def test_choice_by_hand():
    l = torch.tensor([[0.1, 0.9, 0.9, -0.5, 2.0, 0.3]])
    assert R.choose(l, 3, R.SOFTMAX).tolist() == [[4, 1, 2]]
    # groups {0,1,2}, {3,4,5}: the largest of each, or the two largest
    assert R.choose(l, 2, R.SOFTMAX, groups=2, topk_groups=1, group_top=1).tolist() == [[4, 5]]
    s = torch.sigmoid(l.double())[0]
    first = float(s[1] + s[2]) > float(s[4] + s[5])
    assert R.choose(l, 2, R.SIGMOID, groups=2, topk_groups=1, group_top=2).tolist() == [[1, 2] if first else [4, 5]]
    bias = torch.tensor([5.0, 0, 0, 0, 0, -float("inf")])
    assert R.choose(l, 6, R.SIGMOID, bias).tolist() == [[0, 4, 1, 2, 3, -1]]
    l[0, 4] = float("nan")
    l[0, 1] = -float("inf")
    assert R.choose(l, 6, R.SIGMOID).tolist() == [[4, 2, 5, 0, 3, -1]]


def test_weights_by_hand():
    l = torch.log(torch.tensor([[1.0, 2.0, 3.0, 4.0]]))
    ids = torch.tensor([[3, 1]], dtype=torch.int32)
    assert torch.allclose(R.weights(l, ids, R.SOFTMAX, False, 2.0), torch.tensor([[0.8, 0.4]]).double(), atol=1e-6)
    assert torch.allclose(R.weights(l, ids, R.SOFTMAX, True, 1.0), torch.tensor([[2 / 3, 1 / 3]]).double(), atol=1e-6)
    p = torch.tensor([[4 / 5, 2 / 3]]).double()
    assert torch.allclose(R.weights(l, ids, R.SIGMOID, False, 1.0), p, atol=1e-6)
    assert torch.allclose(R.weights(l, ids, R.SIGMOID, True, 1.0), p / p.sum(), atol=1e-6)


@pytest.mark.parametrize("score", [R.SOFTMAX, R.SIGMOID])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_reference_against_differences(score, renormalize):
    gen = torch.Generator().manual_seed(1)
    l = torch.randn(2, 9, generator=gen).double()
    ids = torch.tensor([[4, 0, -1], [8, 2, 3]], dtype=torch.int32)
    g = torch.randn(2, 3, generator=gen)
    d, _ = R.logits_grad(l, ids, g, score, renormalize, 1.5)
    for e in range(9):
        h = torch.zeros(2, 9, dtype=torch.float64)
        h[:, e] = 1e-6
        n = (R.weights(l + h, ids, score, renormalize, 1.5) - R.weights(l - h, ids, score, renormalize, 1.5)) / 2e-6
        assert torch.allclose((n * g.double()).sum(1), d[:, e], atol=1e-8)


def test_dequantised_words():
    q = torch.tensor([[[0x76543210, -1]]], dtype=torch.int32)       # nibble slot i holds i
    s, z = torch.tensor([[[0.5]]]), torch.tensor([[[3]]], dtype=torch.uint8)
    w = R.dequantise(q, s, z, 16)[0, 0]
    assert w[:8].tolist() == [(v - 3) / 2 for v in (0, 4, 1, 5, 2, 6, 3, 7)] and w[8:].tolist() == [6.0] * 8
