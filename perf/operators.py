"""Cases of the expert operators beside the routed expert FFN: matrix products grouped by expert
with ragged row counts (forward and both gradients), microscaled 4-bit floating point (quantisation,
and the grouped product of two such operands) and the row offsets of an alignment.

Rows are grouped by expert: expert e owns rows offsets[e] .. offsets[e + 1] - 1. Weights are
[E, N, K]; the forward product is y[r] = W[e] x[r], its gradients dx[r] = W[e]^T dy[r] and
dW[e] = sum over e's rows of dy[r] x[r]^T. A microscaled row holds E2M1 codes, two to a byte with
the even element in the low nibble, and one E8M0 exponent byte per 32 elements.

With `own` false, run() computes the plain forms in torch (32-bit arithmetic, rounded once).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    # Sizes of the layer this package serves: hidden 2048, per-expert intermediate 768 (gate/up
    # rows 1536), 128 experts, top-8.
    gate_up = dict(E=128, N=1536, K=2048, k=8)
    down = dict(E=128, N=2048, K=768, k=8)
    return [
        # One token's gate/up products in bf16: eight experts with one row each, weights read once.
        dict(name="forward, one token", op="forward", tokens=1, **gate_up, dtype="bf16", out="bf16", zipf=0.0),
        # A prefill or training step of 4096 tokens: every expert has a few hundred rows.
        dict(name="forward, 4096 tokens", op="forward", tokens=4096, **gate_up, dtype="bf16", out="bf16", zipf=0.5),
        # Input gradient of a small skewed batch: many experts with few rows, some with none.
        dict(name="input gradient, 256 tokens", op="dx", tokens=256, **gate_up, dtype="fp16", out="fp16", zipf=1.1),
        # Input gradient of few large experts (an expert-parallel shard), odd row count, fp32 result.
        dict(name="input gradient, 8 experts", op="dx", tokens=8191, E=8, N=2048, K=768, k=2, dtype="bf16",
             out="fp32", zipf=0.3),
        # Weight gradient of 21 tokens: bound by writing every expert's fp32 gradient.
        dict(name="weight gradient, 21 tokens", op="dw", tokens=21, **down, dtype="bf16", out="fp32", zipf=0.0),
        # Weight gradient of a training step.
        dict(name="weight gradient, 4096 tokens", op="dw", tokens=4096, **gate_up, dtype="bf16", out="bf16",
             zipf=0.5),
        # Activations of a small batch to 4 bits and back: a latency-bound call.
        dict(name="quantise, 21 rows", op="quantise", rows=21, K=2048, dtype="bf16"),
        # A whole layer's gate/up weights to 4 bits (and back: what the codes stand for).
        dict(name="quantise, layer weights", op="quantise", rows=128 * 1536, K=2048, dtype="fp32"),
        # One token's gate/up products on 4-bit operands.
        dict(name="4-bit product, one token", op="mxfp4", tokens=1, **gate_up, out="fp32", zipf=0.0),
        # A prefill step on 4-bit operands.
        dict(name="4-bit product, 4096 tokens", op="mxfp4", tokens=4096, **gate_up, out="bf16", zipf=0.5),
        # Row offsets of a small batch's alignment, and of a prefill's.
        dict(name="offsets, 21 tokens", op="offsets", tokens=21, k=8, E=128, b=8),
        dict(name="offsets, 32768 tokens", op="offsets", tokens=32768, k=8, E=128, b=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "dx", "dw", "quantise", "mxfp4", "offsets"])
    if op == "quantise":
        K = 32 * _log(rng, 1, 128)
        return dict(op=op, rows=_log(rng, 1, min(200000, (128 * 1536 * 2048) // K)), K=K,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    k = rng.choice([1, 2, 4, 6, 8])
    E = max(k, _log(rng, 1, 160))
    if op == "offsets":
        return dict(op=op, tokens=_log(rng, 1, 32768), k=k, E=E, b=rng.choice([1, 1, 8, 16, 64, 24]))
    step = 32 if op == "mxfp4" else 8
    while True:
        N, K = (step * _log(rng, 64 // step, 4096 // step) for _ in range(2))
        tokens = _log(rng, 1, 8192)
        if E * N * K <= 128 * 1536 * 2048 and tokens * k * N * K <= 32768 * 1536 * 2048:
            break
    case = dict(op=op, tokens=tokens, E=E, N=N, K=K, k=k, zipf=rng.choice([0.0, 0.3, 0.5, 1.1]))
    if op == "mxfp4":
        return dict(case, out=rng.choice(["bf16", "fp16", "fp32"]))
    dtype = rng.choice(["bf16", "fp16"])
    return dict(case, dtype=dtype, out=rng.choice([dtype, dtype, "fp32"]))


def _routing(case, g):
    """top-k expert IDs [tokens, k] int32; `zipf` is the popularity exponent."""
    rank = torch.randperm(case["E"], generator=g, device="cuda") + 1
    u = torch.rand(case["tokens"], case["E"], generator=g, device="cuda").clamp_min(1e-9)
    logits = -(-u.log()).log() - case.get("zipf", 0.0) * rank.log()
    return logits.topk(case["k"], dim=1).indices.to(torch.int32)


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * scale


def _to_mxfp4(x):
    """(codes [.., K] uint8, biased exponents [.., K / 32] uint8) of fp32 x: the shared exponent is
    floor(log2(largest magnitude)) - 2, elements round to nearest even and saturate at 6."""
    blocks = x.unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, -127)
    v = torch.ldexp(blocks, -e.unsqueeze(-1))
    m = v.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
            + 8 * torch.signbit(v))
    return code.flatten(-2).to(torch.uint8), (e + 127).to(torch.uint8)


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpacked(q):
    return torch.stack((q & 15, q >> 4), -1).flatten(-2)


def _values(code, exponent):
    lut = torch.tensor(E2M1, device=code.device)
    scale = torch.exp2(exponent.to(torch.float32) - 127.0)
    return (lut[code.to(torch.int32)].unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "quantise":
        # Rows of different magnitude, as activations after a norm and weight rows have.
        size = torch.exp(_normal(g, case["rows"], 1, scale=0.5))
        return dict(op=op, x=(_normal(g, case["rows"], case["K"]) * size).to(DTYPES[case["dtype"]]))
    ids = _routing(case, g)
    E = case["E"]
    counts = torch.bincount(ids.flatten(), minlength=E)
    if op == "offsets":
        b = case["b"]
        blocks = torch.repeat_interleave(torch.arange(E, device="cuda"), (counts + b - 1) // b)
        rows = ids.numel()
        capacity = (rows + min(E, rows) * (b - 1) + b - 1) // b
        block_ids = torch.full((capacity,), -1, dtype=torch.int32, device="cuda")
        block_ids[:blocks.numel()] = blocks.to(torch.int32)
        return dict(op=op, E=E, b=b, block_ids=block_ids,
                    num_padded=torch.full((1,), blocks.numel() * b, dtype=torch.int32, device="cuda"))
    rows, N, K = ids.numel(), case["N"], case["K"]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    # What a program that pads rows per expert keeps: the experts with rows and the largest count.
    s = dict(op=op, rows=rows, E=E, N=N, K=K, offsets=offsets, out=DTYPES[case["out"]],
             used=counts.nonzero().flatten(), most=int(counts.max()))
    if op == "mxfp4":
        code, s["xs"] = _to_mxfp4(_normal(g, rows, K))
        s["xq"] = _packed(code)
        parts = [_to_mxfp4(_normal(g, min(8, E - e), N, K, scale=0.02)) for e in range(0, E, 8)]
        s["wq"] = torch.cat([_packed(c) for c, _ in parts])
        s["ws"] = torch.cat([x for _, x in parts])
        return s
    dtype = DTYPES[case["dtype"]]
    if op != "dw":
        s["w"] = _normal(g, E, N, K, scale=0.02, dtype=dtype)
    if op != "dx":
        s["x"] = _normal(g, rows, K, dtype=dtype)
    if op != "forward":
        s["dy"] = _normal(g, rows, N, dtype=dtype)
    return s


def _places(s):
    """For each row, which of the experts with rows owns it, and its place among that expert's rows."""
    row = torch.arange(s["rows"], device="cuda")
    starts = s["offsets"][s["used"]].long()
    which = torch.searchsorted(starts, row, right=True) - 1
    return which, row - starts[which]


def _padded(s, rows, places):
    p = torch.zeros(s["used"].numel(), s["most"], rows.shape[1], device="cuda")
    p[places] = rows
    return p


def _plain(s):
    op = s["op"]
    if op == "quantise":
        code, exponent = _to_mxfp4(s["x"].float())
        return {"values": _values(code, exponent).to(torch.bfloat16), "exponent": exponent}
    if op == "offsets":
        blocks = s["block_ids"].long()
        live = torch.arange(blocks.numel(), device="cuda") * s["b"] < s["num_padded"]
        count = torch.zeros(s["E"], dtype=torch.int64, device="cuda")
        count.index_add_(0, blocks.clamp_min(0), live * s["b"])
        count = count.cumsum(0)
        return torch.cat((count.new_zeros(1), count)).to(torch.int32)
    places = _places(s)
    if op == "mxfp4":
        x = _padded(s, _values(_unpacked(s["xq"]), s["xs"]), places)
        w = _values(_unpacked(s["wq"][s["used"]]), s["ws"][s["used"]])
        return torch.matmul(x, w.transpose(1, 2))[places].to(s["out"])
    if op == "forward":
        x = _padded(s, s["x"].float(), places)
        return torch.matmul(x, s["w"][s["used"]].float().transpose(1, 2))[places].to(s["out"])
    dy = _padded(s, s["dy"].float(), places)
    if op == "dx":
        return torch.matmul(dy, s["w"][s["used"]].float())[places].to(s["out"])
    dw = torch.zeros(s["E"], s["N"], s["K"], dtype=s["out"], device="cuda")
    dw[s["used"]] = torch.matmul(dy.transpose(1, 2), _padded(s, s["x"].float(), places)).to(s["out"])
    return dw


def run(s):
    if not own:
        return _plain(s)
    import mixture_experts_ffn_align_amd as moe
    op = s["op"]
    if op == "quantise":
        rows, K = s["x"].shape
        q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
        scale = torch.empty(rows, K // 32, dtype=torch.uint8, device="cuda")
        values = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
        moe.moe_mxfp4_quantize(s["x"], q, scale)
        moe.moe_mxfp4_dequantize(q, scale, values)
        return {"values": values, "exponent": scale}
    if op == "offsets":
        offsets = torch.empty(s["E"] + 1, dtype=torch.int32, device="cuda")
        moe.moe_align_offsets(s["block_ids"], s["num_padded"], s["E"], s["b"], offsets)
        return offsets
    if op == "mxfp4":
        y = torch.empty(s["rows"], s["N"], dtype=s["out"], device="cuda")
        moe.moe_grouped_matmul_mxfp4(s["xq"], s["xs"], s["wq"], s["ws"], s["offsets"], y)
        return y
    if op == "forward":
        y = torch.empty(s["rows"], s["N"], dtype=s["out"], device="cuda")
        moe.moe_grouped_matmul(s["x"], s["w"], s["offsets"], y)
        return y
    if op == "dx":
        dx = torch.empty(s["rows"], s["K"], dtype=s["out"], device="cuda")
        moe.moe_grouped_matmul_dx(s["dy"], s["w"], s["offsets"], dx)
        return dx
    dw = torch.empty(s["E"], s["N"], s["K"], dtype=s["out"], device="cuda")
    moe.moe_grouped_matmul_dw(s["dy"], s["x"], s["offsets"], dw)
    return dw


def work(case):
    op = case["op"]
    if op == "quantise":
        n = case["rows"] * case["K"]
        return {"bytes": n * DTYPES[case["dtype"]].itemsize + n / 32 + 2 * n, "flops": 2 * n}
    rows = case["tokens"] * case["k"]
    E = case["E"]
    if op == "offsets":
        return {"bytes": 4 * (rows // case["b"]) + 4 * (E + 2), "flops": 0}
    N, K = case["N"], case["K"]
    used = min(E, rows)                     # experts whose weights a pass has to read, at most
    if op == "mxfp4":
        a, o = 17 / 32, DTYPES[case["out"]].itemsize
    else:
        a, o = 2, DTYPES[case["out"]].itemsize
    size = {"forward": a * (rows * K + used * N * K) + o * rows * N,
            "mxfp4": a * (rows * K + used * N * K) + o * rows * N,
            "dx": a * (rows * N + used * N * K) + o * rows * K,
            "dw": a * rows * (N + K) + o * E * N * K}[op]
    return {"bytes": size + 4 * (E + 1), "flops": 2 * rows * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "offsets":
        return None
    grid = torch.tensor(E2M1[:8], dtype=torch.float64, device="cuda")

    def decode(q, exponent):
        v = torch.stack((q.bitwise_and(7), q.bitwise_right_shift(4).bitwise_and(7)), -1).flatten(-2)
        sign = torch.stack((q.bitwise_and(8), q.bitwise_right_shift(4).bitwise_and(8)), -1).flatten(-2)
        return grid[v.long()] * (1.0 - sign.double() / 4) * torch.exp2(exponent.double() - 127).repeat_interleave(32, -1)

    if op == "quantise":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        even = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device="cuda")   # codes, the even ones first
        for r in range(0, out.shape[0], 4096):
            x = s["x"][r:r + 4096].double()
            top = x.abs().unflatten(-1, (-1, 32)).amax(-1)
            e = torch.where(top > 0, torch.floor(torch.log2(top)), torch.full_like(top, -200.0))
            # log2 may round up to the next whole number just below a power of two
            e = torch.where(torch.exp2(e) > top, e - 1, e) - 2
            unit = torch.exp2(e.clamp(-127, 127)).repeat_interleave(32, -1)
            m = x.abs() / unit
            best, at = torch.full_like(m, math.inf), torch.zeros_like(m)
            for c in even.tolist():        # nearest value of the grid; a tie keeps the even code
                d = (m - grid[c]).abs()
                at = torch.where(d < best, grid[c], at)
                best = torch.minimum(best, d)
            out[r:r + 4096] = torch.copysign(at * unit, x)
        return {"values": out, "exponent": None}
    ends = s["offsets"].tolist()
    if op == "dw":
        dw = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64, device="cuda")
    else:
        y = torch.zeros(s["rows"], case["K"] if op == "dx" else case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        if op == "dw":
            dw[e] = s["dy"][a:b].double().T.contiguous() @ s["x"][a:b].double()
        elif op == "dx":
            y[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
        elif op == "forward":
            y[a:b] = s["x"][a:b].double() @ s["w"][e].double().T.contiguous()
        else:
            y[a:b] = decode(s["xq"][a:b], s["xs"][a:b]) @ decode(s["wq"][e], s["ws"][e]).T.contiguous()
    return dw if op == "dw" else y
