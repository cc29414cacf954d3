"""Each operand of the routing, combine and 4-bit calls with one property broken:
the call is refused with that operand's name and nothing is enqueued. On the
host the tensors only report a GPU; with a GPU they are on it."""
import types

import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from mixture_experts_ffn_align_amd import _binding as B
from tests.test_ragged_refusals import BREAK, EXPECTED, OnGpu

M, E, K, H, ROWS, N = 3, 16, 2, 64, 6, 24
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

CALLS = {
    "moe_route": dict(logits=(BF, (M, E)), topk_ids=(I32, (M, K)), topk_w=(F32, (M, K)), bias=(F32, (E,))),
    "moe_route_grad": dict(logits=(BF, (M, E)), topk_ids=(I32, (M, K)), dtopk_w=(F32, (M, K)), dlogits=(BF, (M, E))),
    "moe_align_positions": dict(sorted_route_ids=(I32, (8,)), num_padded=(I32, (1,)), positions=(I32, (M, K))),
    "moe_combine": dict(rows=(BF, (ROWS, H)), positions=(I32, (M, K)), topk_w=(F32, (M, K)), y=(BF, (M, H))),
    "moe_combine_grad": dict(dy=(BF, (M, H)), rows=(BF, (ROWS, H)), positions=(I32, (M, K)), topk_w=(F32, (M, K)),
                             drows=(BF, (ROWS, H)), dtopk_w=(F32, (M, K))),
    "moe_matvec_int4": dict(x=(BF, (M, H)), q=(I32, (E, N, H // 8)), scale=(torch.float16, (E, N, H // 32)),
                            zero=(U8, (E, N, H // 32)), y=(BF, (M, K, N)), topk_ids=(I32, (M, K))),
}
# Operands whose shape the others are held to: a wrong size shows at another one.
DEFINES = {"moe_route": ("logits", "topk_ids"), "moe_route_grad": ("logits", "topk_ids"), "moe_align_positions": (),
           "moe_combine": ("rows", "y", "positions"), "moe_combine_grad": ("drows", "dy", "positions"),
           "moe_matvec_int4": ("x", "q", "topk_ids")}
OPTIONAL = ("bias", "positions", "topk_w", "dtopk_w", "zero", "topk_ids")
SHAPES_CHANGE = ("one shorter", "narrower", "one more dimension")


def skipped(call, name, how):
    if how == "nothing" and name in OPTIONAL and call != "moe_align_positions":
        return name not in ("topk_ids", "topk_w") or call in ("moe_combine", "moe_combine_grad", "moe_matvec_int4")
    if name == "num_padded" and how == "strided":
        return True                                   # one element
    if call == "moe_align_positions" and name != "num_padded" and how in SHAPES_CHANGE:
        # any alignment and any [M, k] is right
        return name == "sorted_route_ids" or how != "one more dimension"
    # fewer slots than routes' rows, or other rows, are the caller's business
    return (call, name, how) in (("moe_combine", "rows", "one shorter"), ("moe_combine_grad", "drows", "one shorter"))


def cases():
    for call, operands in CALLS.items():
        for name in operands:
            for how in BREAK:
                if not skipped(call, name, how):
                    yield pytest.param(call, name, how, id=f"{call}-{name}-{how}".replace(" ", "_"))


def make(call, a):
    if call == "moe_matvec_int4":
        w = types.SimpleNamespace(fmt=B.MOE_W_INT4_AWQ, group=32, q=a["q"], scale=a["scale"], zero=a["zero"])
        return moe.moe_matvec_int4(a["x"], w, a["y"], topk_ids=a["topk_ids"])
    return getattr(moe, call)(*a.values())


def refused(call, name, how, put):
    args = {n: put(torch.zeros(shape, dtype=dtype)) for n, (dtype, shape) in CALLS[call].items()}
    args[name] = BREAK[how](args[name])
    named = name
    if name in DEFINES[call] and how in SHAPES_CHANGE:
        named = r"\w+"
    with pytest.raises(EXPECTED[how], match=f"^{named}: "):
        make(call, args)


@pytest.fixture
def nothing_enqueued(monkeypatch):
    def reached(*_):
        raise AssertionError("the library was called")
    monkeypatch.setattr(B, "_call_on", reached)


@pytest.mark.parametrize("call,name,how", cases())
def test_refused_on_the_host(call, name, how, nothing_enqueued):
    refused(call, name, how, lambda t: t.as_subclass(OnGpu))


@pytest.mark.gpu
@pytest.mark.parametrize("call,name,how", cases())
def test_refused_on_a_gpu(call, name, how, nothing_enqueued):
    refused(call, name, how, lambda t: t.cuda())


def host(call, **changes):
    args = {n: torch.zeros(shape, dtype=dtype).as_subclass(OnGpu) for n, (dtype, shape) in CALLS[call].items()}
    args.update({n: None if v is None else v.as_subclass(OnGpu) for n, v in changes.items()})
    return args


def test_types_that_do_not_go_together(nothing_enqueued):
    for call, name, dtype in (("moe_route_grad", "dlogits", torch.float16), ("moe_combine_grad", "rows", F32),
                              ("moe_matvec_int4", "y", torch.float16), ("moe_matvec_int4", "x", F32)):
        shape = CALLS[call][name][1]
        with pytest.raises(TypeError, match=f"^{name}: "):
            make(call, host(call, **{name: torch.zeros(shape, dtype=dtype)}))
    with pytest.raises(TypeError, match="^rows: "):          # needed for the weights' gradient
        make("moe_combine_grad", host("moe_combine_grad", rows=None))
    with pytest.raises(TypeError, match="^w: "):
        moe.moe_matvec_int4(*(torch.zeros(M, H, dtype=BF).as_subclass(OnGpu) for _ in range(3)))


def test_rows_in_route_order_need_as_many(nothing_enqueued):
    for call in ("moe_combine", "moe_combine_grad"):
        with pytest.raises(ValueError, match="^positions: "):
            a = host(call, positions=None)
            name = "rows" if call == "moe_combine" else "drows"
            a[name] = torch.zeros(ROWS + 1, H, dtype=BF).as_subclass(OnGpu)
            make(call, a)


def test_sizes_past_32_bits(nothing_enqueued):
    a = host("moe_route")
    for name in ("score", "groups", "topk_groups", "group_top"):
        with pytest.raises(ValueError, match=f"^{name}: "):
            moe.moe_route(a["logits"], a["topk_ids"], a["topk_w"], **{name: 2 ** 32 + 1})
        with pytest.raises(ValueError, match=f"^{name}: "):
            moe.moe_route(a["logits"], a["topk_ids"], a["topk_w"], **{name: -2 ** 32 + 1})
    a = host("moe_matvec_int4")
    w = types.SimpleNamespace(fmt=B.MOE_W_INT4_AWQ, group=2 ** 32 + 32, q=a["q"],
                              scale=a["scale"][..., :0].contiguous(), zero=None)
    with pytest.raises(ValueError, match="^group: "):
        moe.moe_matvec_int4(a["x"], w, a["y"], topk_ids=a["topk_ids"])
