"""Each operand of each ragged, MXFP4 and offsets call with one property broken:
the call is refused with that operand's name and nothing is enqueued. On the
host the tensors only report a GPU; with a GPU they are on it."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from mixture_experts_ffn_align_amd import _binding as B

ROWS, E, N, K = 4, 2, 16, 64
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8

# Operands of each call: (dtype, shape), "rows" for those that may have a row stride.
CALLS = {
    "moe_grouped_matmul": dict(x=(BF, (ROWS, K), "rows"), w=(BF, (E, N, K)), offsets=(I32, (E + 1,)),
                               y=(BF, (ROWS, N), "rows")),
    "moe_grouped_matmul_dx": dict(dy=(BF, (ROWS, N), "rows"), w=(BF, (E, N, K)), offsets=(I32, (E + 1,)),
                                  dx=(BF, (ROWS, K), "rows")),
    "moe_grouped_matmul_dw": dict(dy=(BF, (ROWS, N), "rows"), x=(BF, (ROWS, K), "rows"), offsets=(I32, (E + 1,)),
                                  dw=(BF, (E, N, K))),
    "moe_grouped_matmul_mxfp4": dict(xq=(U8, (ROWS, K // 2)), x_scale=(U8, (ROWS, K // 32)),
                                     wq=(U8, (E, N, K // 2)), w_scale=(U8, (E, N, K // 32)), offsets=(I32, (E + 1,)),
                                     y=(BF, (ROWS, N), "rows")),
    "moe_mxfp4_quantize": dict(x=(BF, (ROWS, K), "rows"), q=(U8, (ROWS, K // 2)), scale=(U8, (ROWS, K // 32))),
    "moe_mxfp4_dequantize": dict(q=(U8, (ROWS, K // 2)), scale=(U8, (ROWS, K // 32)), y=(BF, (ROWS, K), "rows")),
    "moe_align_offsets": dict(expert_block_ids=(I32, (8,)), num_padded=(I32, (1,)), offsets=(I32, (E + 1,))),
}
# Operands whose shape the others are held to: a wrong size shows at another one.
DEFINES = {"moe_grouped_matmul": ("x", "w"), "moe_grouped_matmul_dx": ("dy", "w"), "moe_grouped_matmul_dw": ("dy", "dw"),
           "moe_grouped_matmul_mxfp4": ("xq", "wq"), "moe_mxfp4_quantize": ("x",), "moe_mxfp4_dequantize": ("y",),
           "moe_align_offsets": ()}


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""

    @property
    def device(self):
        return torch.device("cuda", 0)

    @property
    def is_cuda(self):
        return True


def on_host(t):
    return t.as_subclass(torch.Tensor) if isinstance(t, OnGpu) else t.cpu()


def strided(t):
    """The same values with every other element of a longer row between them."""
    return torch.stack((t, t), -1).flatten(-2)[..., ::2]


BREAK = {
    "nothing": lambda t: None,
    "a list": lambda t: [1],
    "another type": lambda t: t.to(torch.int64 if t.dtype == I32 else torch.int8 if t.dtype == U8 else torch.float64),
    "host memory": on_host,
    "strided": strided,
    "one shorter": lambda t: t[:-1],
    "narrower": lambda t: t[..., :-1].contiguous(),
    "one more dimension": lambda t: t.unsqueeze(0),
}
EXPECTED = {"nothing": TypeError, "a list": TypeError, "another type": TypeError, "host memory": ValueError,
            "strided": ValueError, "one shorter": ValueError, "narrower": ValueError, "one more dimension": ValueError}


def cases():
    for call, operands in CALLS.items():
        for name, (_, shape, *_rest) in operands.items():
            for how in BREAK:
                if call == "moe_align_offsets" and name == "expert_block_ids" and how in (
                        "one shorter", "narrower", "one more dimension"):
                    continue                      # any number of blocks is right
                if name == "num_padded" and how == "strided":
                    continue                      # one element
                if call.startswith("moe_mxfp4") and how == "one more dimension" and name in DEFINES[call]:
                    continue                      # leading dimensions are the user's
                yield pytest.param(call, name, how, id=f"{call}-{name}-{how}".replace(" ", "_"))


def operands(call, put):
    return {name: put(torch.zeros(spec[1], dtype=spec[0])) for name, spec in CALLS[call].items()}


def make_call(call, args):
    if call == "moe_align_offsets":
        blocks, num_padded, offsets = args.values()
        return moe.moe_align_offsets(blocks, num_padded, E, 1, offsets)
    return getattr(moe, call)(*args.values())


def refused(call, name, how, put):
    args = operands(call, put)
    args[name] = BREAK[how](args[name])
    named = name
    if name in DEFINES[call] and how in ("one shorter", "narrower", "one more dimension"):
        named = r"\w+"
    with pytest.raises(EXPECTED[how], match=f"^{named}: "):
        make_call(call, args)


@pytest.fixture
def made(monkeypatch):
    calls = []
    monkeypatch.setattr(B, "_call_on", lambda device, stream, fn, *args: calls.append(args) or B.MOE_OK)
    return calls


@pytest.mark.parametrize("call", CALLS)
def test_unbroken_operands_are_taken(made, call):
    make_call(call, operands(call, lambda t: t.as_subclass(OnGpu)))
    assert len(made) == 1


@pytest.mark.parametrize("call,name,how", cases())
def test_one_broken_operand(made, call, name, how):
    refused(call, name, how, lambda t: t.as_subclass(OnGpu))
    assert not made


@pytest.mark.parametrize("call,name,other", [
    ("moe_grouped_matmul", "w", torch.float16), ("moe_grouped_matmul", "y", torch.float16),
    ("moe_grouped_matmul_dx", "w", torch.float16), ("moe_grouped_matmul_dx", "dx", torch.float16),
    ("moe_grouped_matmul_dw", "x", torch.float16), ("moe_grouped_matmul_dw", "dw", torch.float16),
    ("moe_mxfp4_dequantize", "y", torch.float16)])
def test_types_that_do_not_go_together(made, call, name, other):
    args = operands(call, lambda t: t.as_subclass(OnGpu))
    args[name] = args[name].to(other)
    with pytest.raises(TypeError, match=f"^{name}: "):
        make_call(call, args)
    assert not made


@pytest.mark.gpu
@pytest.mark.parametrize("call,name,how", cases())
def test_one_broken_operand_on_a_gpu(call, name, how):
    refused(call, name, how, lambda t: t.cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("call", [c for c in CALLS if c != "moe_align_offsets"])
def test_row_strides_and_addresses_on_a_gpu(call):
    # What the library itself refuses: rows that start off 16 bytes, by their
    # first address or by a stride that is no multiple of eight elements.
    for name, (dtype, shape, *rows) in CALLS[call].items():
        if not rows:
            continue
        for wide, first in ((shape[1] + 8, 1), (shape[1] + 4, 0)):
            args = operands(call, lambda t: t.cuda())
            args[name] = torch.zeros(shape[0], wide, dtype=dtype, device="cuda")[:, first:first + shape[1]]
            with pytest.raises(moe.MoeError) as e:
                make_call(call, args)
            assert e.value.status == B.MOE_ERR_INVALID_ARG
