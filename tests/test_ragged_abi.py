"""Host-only checks of the ragged products, MXFP4 and the alignment's offsets:
bad arguments are refused before anything is enqueued, by the C ABI and by the
binding; and the definitions the GPU tests hold the kernels to."""
import ctypes

import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from mixture_experts_ffn_align_amd import _binding as B
from tests import _ragged as R

FAKE = 0x10000  # aligned, non-null; never dereferenced on these paths
INV, UNS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED


def desc(rows=4, E=2, N=16, K=32, dtype=B.MOE_DTYPE_BF16, out=B.MOE_DTYPE_BF16):
    return B.moe_grouped_matmul_desc(rows, E, N, K, dtype, out)


def fwd(d, x=FAKE, ldx=None, w=FAKE, off=FAKE, y=FAKE, ldy=None):
    return B.lib().moe_grouped_matmul(ctypes.byref(d), x, d.K if ldx is None else ldx, w, off, y,
                                      d.N if ldy is None else ldy, None)


def dgrad(d, dy=FAKE, lddy=None, w=FAKE, off=FAKE, dx=FAKE, lddx=None):
    return B.lib().moe_grouped_matmul_dx(ctypes.byref(d), dy, d.N if lddy is None else lddy, w, off, dx,
                                         d.K if lddx is None else lddx, None)


def wgrad(d, dy=FAKE, lddy=None, x=FAKE, ldx=None, off=FAKE, dw=FAKE):
    return B.lib().moe_grouped_matmul_dw(ctypes.byref(d), dy, d.N if lddy is None else lddy, x,
                                         d.K if ldx is None else ldx, off, dw, None)


def fp4(d, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, off=FAKE, y=FAKE, ldy=None):
    return B.lib().moe_grouped_matmul_mxfp4(ctypes.byref(d), xq, xs, wq, ws, off, y, d.N if ldy is None else ldy,
                                            None)


BAD_DESCS = [(dict(rows=-1), INV), (dict(E=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(N=12), INV),
             (dict(K=36), INV), (dict(E=4096), UNS), (dict(N=1 << 21), UNS), (dict(K=1 << 21), UNS),
             (dict(rows=2 ** 31 - 1, N=1 << 20, K=1 << 20), UNS), (dict(out=9), INV)]


@pytest.mark.parametrize("bad,status", BAD_DESCS, ids=str)
@pytest.mark.parametrize("call", [fwd, dgrad, wgrad], ids=lambda c: c.__name__)
def test_products_refuse_bad_descriptions(call, bad, status):
    assert call(desc(**bad)) == status


@pytest.mark.parametrize("call", [fwd, dgrad, wgrad], ids=lambda c: c.__name__)
def test_products_refuse_bad_types(call):
    assert call(desc(dtype=B.MOE_DTYPE_F32, out=B.MOE_DTYPE_F32)) == INV
    assert call(desc(dtype=B.MOE_DTYPE_MXFP4)) == INV
    assert call(desc(dtype=B.MOE_DTYPE_BF16, out=B.MOE_DTYPE_F16)) == INV
    assert call(desc(dtype=B.MOE_DTYPE_F16, out=B.MOE_DTYPE_BF16)) == INV


def test_products_refuse_bad_pointers_and_strides():
    d = desc()
    null = ctypes.POINTER(B.moe_grouped_matmul_desc)()
    assert B.lib().moe_grouped_matmul(null, FAKE, 32, FAKE, FAKE, FAKE, 16, None) == INV
    for call, rows_args, other in ((fwd, ("x", "y"), ("w", "off")), (dgrad, ("dy", "dx"), ("w", "off")),
                                   (wgrad, ("dy", "x"), ("off", "dw"))):
        for a in rows_args + other:
            assert call(d, **{a: None}) == INV, (call, a)
        for a in rows_args:
            assert call(d, **{a: FAKE + 2}) == INV, (call, a)
            assert call(d, **{"ld" + a: 8}) == INV, (call, a)        # shorter than a row
            assert call(d, **{"ld" + a: 36}) == INV, (call, a)       # not a multiple of 8
            assert call(d, **{"ld" + a: (1 << 22) + 8}) == UNS, (call, a)
    assert fwd(d, w=FAKE + 8) == INV and dgrad(d, w=FAKE + 8) == INV and wgrad(d, dw=FAKE + 4) == INV


def test_no_rows_is_a_no_op_without_pointers():
    d = desc(rows=0)
    assert fwd(d, x=None, w=None, off=None, y=None) == B.MOE_OK
    assert dgrad(d, dy=None, w=None, off=None, dx=None) == B.MOE_OK
    assert fp4(desc(rows=0, dtype=B.MOE_DTYPE_MXFP4), xq=None, y=None) == B.MOE_OK
    assert wgrad(d, dw=None) == INV                                  # every gradient is written


def test_fp4_product_refusals():
    good = dict(dtype=B.MOE_DTYPE_MXFP4)
    assert fp4(desc()) == INV                                        # not MXFP4
    assert fp4(desc(K=40, **good)) == INV
    assert fp4(desc(N=12, **good)) == INV
    assert fp4(desc(out=B.MOE_DTYPE_MXFP4, **good)) == INV
    for a in ("xq", "xs", "wq", "ws", "off", "y"):
        assert fp4(desc(**good), **{a: None}) == INV, a
    assert fp4(desc(**good), xq=FAKE + 8) == INV and fp4(desc(**good), wq=FAKE + 8) == INV
    assert fp4(desc(**good), y=FAKE + 8) == INV and fp4(desc(**good), ldy=8) == INV


def test_quantise_refusals():
    L = B.lib()
    for fn in (L.moe_mxfp4_quantize, ):
        assert fn(3, FAKE, 32, 1, 32, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 32, -1, 32, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 48, 1, 48, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 0, 1, 0, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 1 << 21, 1, 1 << 21, FAKE, FAKE, None) == UNS
        assert fn(0, FAKE, 32, 1 << 50, 32, FAKE, FAKE, None) == UNS
        assert fn(0, None, 32, 1, 32, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 32, 1, 32, None, FAKE, None) == INV
        assert fn(0, FAKE, 32, 1, 32, FAKE, None, None) == INV
        assert fn(0, FAKE + 8, 32, 1, 32, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 36, 1, 32, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 24, 1, 32, FAKE, FAKE, None) == INV
        assert fn(0, FAKE, 32, 1, 32, FAKE + 8, FAKE, None) == INV
        assert fn(0, None, 32, 0, 32, None, None, None) == B.MOE_OK
    fn = L.moe_mxfp4_dequantize
    assert fn(B.MOE_DTYPE_F16, FAKE, FAKE, 1, 32, FAKE, 32, None) == UNS
    assert fn(7, FAKE, FAKE, 1, 32, FAKE, 32, None) == INV
    assert fn(0, FAKE, FAKE, 1, 40, FAKE, 40, None) == INV
    assert fn(0, None, FAKE, 1, 32, FAKE, 32, None) == INV
    assert fn(0, FAKE, None, 1, 32, FAKE, 32, None) == INV
    assert fn(0, FAKE, FAKE, 1, 32, None, 32, None) == INV
    assert fn(0, FAKE, FAKE, 1, 32, FAKE, 24, None) == INV
    assert fn(0, FAKE, FAKE, 0, 32, None, 32, None) == B.MOE_OK


def test_align_offsets_refusals():
    fn = B.lib().moe_align_offsets
    assert fn(FAKE, FAKE, 4, 0, 8, FAKE, None) == INV
    assert fn(FAKE, FAKE, 4, 8, 0, FAKE, None) == INV
    assert fn(None, FAKE, 4, 8, 8, FAKE, None) == INV
    assert fn(FAKE, None, 4, 8, 8, FAKE, None) == INV
    assert fn(FAKE, FAKE, 4, 8, 8, None, None) == INV
    assert fn(FAKE, FAKE, 4, 4096, 8, FAKE, None) == UNS
    assert fn(FAKE, FAKE, 1 << 29, 8, 8, FAKE, None) == UNS


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


OFF = torch.zeros(3, dtype=torch.int32)
U8 = torch.uint8


@pytest.mark.parametrize("args,exc", [
    ((bf(4, 32), bf(2, 16, 32), OFF, bf(4, 16)), ValueError),                        # host memory
    ((bf(4, 32).float(), bf(2, 16, 32), OFF, bf(4, 16)), TypeError),
    ((bf(4, 32), bf(2, 16, 32).half(), OFF, bf(4, 16)), (TypeError, ValueError)),
    ((bf(4, 32), bf(2, 16, 32), OFF, bf(4, 16).half()), TypeError),
    ((bf(4, 32), bf(16, 32), OFF, bf(4, 16)), ValueError),
    ((bf(4, 24), bf(2, 16, 32), OFF, bf(4, 16)), ValueError),
    ((bf(4, 32), bf(2, 16, 32), OFF.long(), bf(4, 16)), (TypeError, ValueError)),
    ((bf(32, 4).t(), bf(2, 16, 32), OFF, bf(4, 16)), ValueError),                    # rows not contiguous
    ((bf(1, 4, 32), bf(2, 16, 32), OFF, bf(4, 16)), ValueError),
    (([1], bf(2, 16, 32), OFF, bf(4, 16)), TypeError),
    ((bf(4, 32), [1], OFF, bf(4, 16)), TypeError),
])
def test_binding_refuses_bad_tensors(args, exc):
    with pytest.raises(exc):
        moe.moe_grouped_matmul(*args)


def test_binding_refuses_bad_tensors_of_the_gradients_and_mxfp4():
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul_dx(bf(4, 16), bf(2, 16, 32), OFF, bf(4, 32))
    with pytest.raises(TypeError):
        moe.moe_grouped_matmul_dx(bf(4, 16), bf(2, 16, 32), OFF, bf(4, 32).half())
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul_dw(bf(4, 16), bf(4, 32), OFF, bf(2, 16, 32))
    with pytest.raises((TypeError, ValueError)):
        moe.moe_grouped_matmul_dw(bf(4, 16), bf(4, 32).half(), OFF, bf(2, 16, 32))
    with pytest.raises((TypeError, ValueError)):
        moe.moe_grouped_matmul_dw(bf(4, 16), [1], OFF, bf(2, 16, 32))
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul_mxfp4(torch.zeros(4, 16, dtype=U8), torch.zeros(4, 1, dtype=U8),
                                     torch.zeros(2, 16, 16, dtype=U8), torch.zeros(2, 16, 1, dtype=U8), OFF, bf(4, 16))
    with pytest.raises(TypeError):
        moe.moe_grouped_matmul_mxfp4(bf(4, 16), torch.zeros(4, 1, dtype=U8), torch.zeros(2, 16, 16, dtype=U8),
                                     torch.zeros(2, 16, 1, dtype=U8), OFF, bf(4, 16))
    with pytest.raises(TypeError):
        moe.moe_mxfp4_quantize(torch.zeros(4, 32, dtype=torch.float64), torch.zeros(4, 16, dtype=U8),
                               torch.zeros(4, 1, dtype=U8))
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quantize(bf(4, 32), torch.zeros(4, 16, dtype=U8), torch.zeros(4, 1, dtype=U8))
    with pytest.raises(TypeError):
        moe.moe_mxfp4_dequantize(torch.zeros(4, 16, dtype=U8), torch.zeros(4, 1, dtype=U8), bf(4, 32).half())
    with pytest.raises(ValueError):
        moe.moe_align_offsets(torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 2, 1, OFF)


def test_calls_run_with_the_tensors_device_current(monkeypatch):
    # Tensors on another device than the current one: the call is made with
    # theirs current, on its current stream.
    seen = []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(("enter", self.device.index))

        def __exit__(self, *a):
            seen.append(("exit", self.device.index))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    call = lambda *a: seen.append(a) or 7  # noqa: E731
    assert B._call_on(torch.device("cuda", 1), None, call, "x") == 7
    assert seen == [("enter", 1), ("x", 101), ("exit", 1)]
    seen.clear()
    assert B._call_on(torch.device("cuda", 0), None, call, "x") == 7
    assert B._call_on(torch.device("cuda", 0), 55, call, "x") == 7
    assert seen == [("x", 100), ("x", 55)]


def test_reference_quantiser_by_hand():
    x = torch.zeros(32, dtype=torch.float64)
    x[:8] = torch.tensor([4.0, 0.25, -0.75, 1.25, 1.75, 2.5, -3.5, 5.0])    # ties, each to the even code
    q, s = R.quantise(x)
    assert int(s[0]) == 127
    assert R.codes_to_values(q, s)[:8].tolist() == [4.0, 0.0, -1.0, 1.0, 2.0, 2.0, -4.0, 4.0]
    x[0] = 7.9
    q, s = R.quantise(x)
    assert float(R.codes_to_values(q, s)[0]) == 6.0                          # saturates
    x[0] = float("inf")
    q, s = R.quantise(x)
    assert int(s[0]) == 255 and int(q.max()) == 0
