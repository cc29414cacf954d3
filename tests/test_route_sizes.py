"""Sizes of the routing, combine and 4-bit calls that the C ABI's int32 cannot
hold, on the host: refused by name, not truncated. (No tokens, so that such a
size takes no memory.)"""
import types

import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from mixture_experts_ffn_align_amd import _binding as B
from tests.test_ragged_refusals import OnGpu

E, H, N = 16, 64, 24
MANY = 2 ** 32 + 2                 # its lower 32 bits are a number of routes that would be taken


def on(dtype, *shape):
    return torch.empty(shape, dtype=dtype).as_subclass(OnGpu)


def calls(k):
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    w = types.SimpleNamespace(fmt=B.MOE_W_INT4_AWQ, group=32, q=on(i32, E, N, H // 8), scale=on(torch.float16, E, N, H // 32),
                              zero=None)
    return {
        "moe_route": lambda: moe.moe_route(on(f32, 0, E), on(i32, 0, k), on(f32, 0, k)),
        "moe_route_grad": lambda: moe.moe_route_grad(on(f32, 0, E), on(i32, 0, k), on(f32, 0, k), on(f32, 0, E)),
        "moe_combine": lambda: moe.moe_combine(on(bf, 0, H), on(i32, 0, k), on(f32, 0, k), on(f32, 0, H)),
        "moe_combine without weights": lambda: moe.moe_combine(on(bf, 0, H), on(i32, 0, k), None, on(f32, 0, H)),
        "moe_combine_grad": lambda: moe.moe_combine_grad(on(f32, 0, H), None, None, on(f32, 0, k), on(bf, 0, H), None),
        "moe_matvec_int4": lambda: moe.moe_matvec_int4(on(bf, 0, H), w, on(f32, 0, k, N), topk_ids=on(i32, 0, k)),
    }


@pytest.mark.parametrize("name", calls(1))
def test_routes_per_token_past_32_bits(name, monkeypatch):
    reached = []
    monkeypatch.setattr(B, "_call_on", lambda *a: reached.append(a) or 0)
    with pytest.raises(ValueError, match="^k: "):
        calls(MANY)[name]()
    assert not reached
    assert calls(2)[name]() == moe.MOE_OK and len(reached) == 1
