"""Cases of the operators around the experts: routing (scores, groups, top-k, renormalised weights) and its
gradient, the weighted sum of a token's routes and its gradient, and matrix-vector products with packed
4-bit weights (dense, and routed by expert).

Routing takes logits [M, E]. The score is softmax or sigmoid, the choice value score + bias (without a
bias the logit's own order, which is the score's); experts whose logit or bias is -inf are never chosen.
With groups, the `topk_groups` groups whose `group_top` largest choice values have the largest sums keep
their experts. The k largest choice values win, ties go to the lowest index, missing ones are expert -1
with weight 0. Weights are scale * score, divided by the chosen scores' sum when renormalised.

A token's routes lie in rows grouped by expert: sorted_route_ids[p] is the route (t * k + j) of row p.
y[t] = sum_j w[t, j] rows[p(t, j)]; a route without a row contributes nothing.

4-bit weights are uint32 words of eight nibbles (slot i holds element [0, 2, 4, 6, 1, 3, 5, 7][i]) with an
fp16 scale and a zero point per group along K: w = (q - zero) * scale.

With `own` false, run() computes the plain forms in torch: 32-bit arithmetic rounded once; the choice of
experts, which a rounding could turn, in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SLOT = (0, 2, 4, 6, 1, 3, 5, 7)


def listed():
    # Sizes of the layer this package serves: hidden 2048, per-expert intermediate 768 (gate/up rows 1536),
    # 128 experts, top-8; 256 experts in 8 groups with a balancing bias is the other common router.
    softmax = dict(E=128, k=8, score="softmax", renormalize=True, scale=1.0, groups=1, topk_groups=1, group_top=1,
                   bias=False)
    grouped = dict(E=256, k=8, score="sigmoid", renormalize=True, scale=2.5, groups=8, topk_groups=4, group_top=2,
                   bias=True)
    return [
        # One generated token: a latency-bound call.
        dict(name="route, one token", op="route", M=1, **softmax, dtype="fp32"),
        # A prefill or training step on bf16 logits, where equal logits are common.
        dict(name="route, 4096 tokens", op="route", M=4096, **softmax, dtype="bf16"),
        # A long step of the grouped router.
        dict(name="route in groups, 32768 tokens", op="route", M=32768, **grouped, dtype="fp32"),
        # Gradients: renormalised weights (zero but for the chosen), and plain softmax over an odd count.
        dict(name="route gradient, 32768 tokens", op="route_grad", M=32768, **grouped, dtype="fp32"),
        dict(name="route gradient, 8191 tokens", op="route_grad", M=8191, **dict(softmax, E=160, k=6, renormalize=False),
             dtype="bf16"),
        # Weighted sums of a small batch and of a training step, with the rows' positions.
        dict(name="combine, 21 tokens", op="combine", M=21, E=128, held=128, k=8, b=8, H=2048, dtype="bf16", out="fp32"),
        dict(name="combine, 4096 tokens", op="combine", M=4096, E=128, held=128, k=8, b=1, H=2048, dtype="bf16",
             out="bf16"),
        # Its gradient in a training step: rows' and weights' gradients.
        dict(name="combine gradient, 4096 tokens", op="combine_grad", M=4096, E=128, held=128, k=8, b=1, H=2048,
             dtype="bf16", out="bf16"),
        # One token through a dense projection of the layer's hidden size, and through its eight experts' gate/up rows.
        dict(name="matvec, one token", op="matvec", M=1, k=0, E=1, N=4096, K=2048, g=128, dtype="bf16", out="bf16"),
        dict(name="matvec, one token's experts", op="matvec", M=1, k=8, E=128, N=1536, K=2048, g=128, dtype="bf16",
             out="fp32"),
        # A batch of generated tokens through a wide projection: bound by the weights.
        dict(name="matvec, 16 tokens", op="matvec", M=16, k=0, E=1, N=16384, K=8192, g=128, dtype="bf16", out="bf16"),
        # An odd batch, odd feature count, small groups, a reduction that ends inside a tile.
        dict(name="matvec, 37 tokens", op="matvec", M=37, k=0, E=1, N=5001, K=4064, g=32, dtype="fp16", out="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "combine", "combine_grad", "matvec", "matvec"])
    if op.startswith("route"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, max(2, 8 // groups), 256 // groups)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * topk_groups))
        # bf16 and fp16 logits, and fp32; a twelfth of the experts switched off in some
        return dict(op=op, M=_log(rng, 1, 32768), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), groups=groups,
                    topk_groups=topk_groups, group_top=rng.choice([1, 2]), bias=rng.random() < 0.5,
                    dtype=rng.choice(["fp32", "bf16", "fp16"]), masked=rng.random() < 0.25)
    if op == "matvec":
        g = rng.choice([32, 64, 128, 128])
        k = rng.choice([0, 0, 1, 2, 8])
        while True:
            N, K = _log(rng, 16, 16384), g * _log(rng, max(1, 256 // g), 8192 // g)
            if k == 0 and N * K <= 16384 * 8192 or k and N * K <= 4096 * 2048:
                break
        dtype = rng.choice(["bf16", "fp16"])
        return dict(op=op, M=_log(rng, 1, 64) if k == 0 else _log(rng, 1, 4), k=k,
                    E=max(k, _log(rng, 4, 64)) if k else 1, N=N, K=K, g=g, dtype=dtype,
                    out=rng.choice([dtype, "fp32"]))
    k = rng.choice([1, 2, 4, 6, 8])
    E = max(k, _log(rng, 4, 160))
    while True:
        M, H = _log(rng, 1, 16384), 8 * _log(rng, 8, 1024)
        if M * k * H <= 4096 * 8 * 2048:
            break
    # `held` of the experts' rows are here (an expert-parallel shard); b pads an expert's rows.
    return dict(op=op, M=M, E=E, held=E if rng.random() < 0.7 else max(1, E // 4), k=k, b=rng.choice([1, 1, 8, 16]),
                H=H, dtype=rng.choice(["bf16", "fp16", "fp32"]), out=rng.choice(["bf16", "fp16", "fp32"]))


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _ids(g, M, E, k):
    """k different experts per token, int32 [M, k]."""
    return torch.rand(M, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)


def _align(ids, E, b):
    """The alignment of routes to experts [0, E): (sorted_route_ids [capacity], num_padded [1])."""
    flat = ids.flatten().long()
    n = flat.numel()
    capacity = (n + min(E, n) * (b - 1) + b - 1) // b * b
    expert = torch.where((flat >= 0) & (flat < E), flat, E)
    order = expert.sort(stable=True).indices
    count = torch.bincount(expert, minlength=E + 1)
    padded = (count[:E] + b - 1) // b * b
    first = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    first[1:] = padded.cumsum(0)
    before = count.cumsum(0) - count
    e = expert[order]
    place = first[e] + torch.arange(n, device="cuda") - before[e]
    held = e < E
    rows = torch.full((capacity,), n, dtype=torch.int32, device="cuda")
    rows[place[held]] = order[held].to(torch.int32)
    return rows, first[E:].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op.startswith("route"):
        M, E, k = case["M"], case["E"], case["k"]
        # Logits of a trained router: a spread of about one, experts of different popularity.
        logits = (_normal(g, M, E) + 0.5 * _normal(g, E)).to(DTYPES[case["dtype"]])
        if case.get("masked"):
            logits[:, torch.randperm(E, generator=g, device="cuda")[:E // 12]] = -math.inf
        s["logits"] = logits
        s["offset"] = 0.1 * _normal(g, E) if case["bias"] else None
        if op == "route_grad":
            s["ids"] = _choose(s)[0]
            s["dw"] = _normal(g, M, k)
        return s
    if op == "matvec":
        M, k, E, N, K, dtype = case["M"], case["k"], case["E"], case["N"], case["K"], DTYPES[case["dtype"]]
        s["q"] = torch.randint(-2 ** 31, 2 ** 31, (E, N, K // 8), generator=g, device="cuda", dtype=torch.int32)
        scale = 0.002 + 0.008 * torch.rand(E, N, K // case["g"], generator=g, device="cuda")
        s["scales"] = scale.to(torch.float16).view(torch.int16)
        s["zeros"] = torch.randint(0, 16, scale.shape, generator=g, device="cuda", dtype=torch.uint8)
        s["x"] = _normal(g, M, K, dtype=dtype)
        s["ids"] = _ids(g, M, E, k) if k else None
        return s
    M, k, H, dtype = case["M"], case["k"], case["H"], DTYPES[case["dtype"]]
    ids = _ids(g, M, case["E"], k)
    s["routes"], s["padded"] = _align(ids, case["held"], case["b"])
    s["rows"] = _normal(g, s["routes"].numel(), H, dtype=dtype)
    s["w"] = torch.softmax(_normal(g, M, k), dim=1)
    if op == "combine_grad":
        s["dy"] = _normal(g, M, H, dtype=DTYPES[case["out"]])
        # Rows no route has keep what the buffer held.
        s["drows"] = torch.zeros_like(s["rows"])
    return s


def _choose(s):
    """(ids [M, k] int32 with -1 where none is left, live) of the experts chosen, in 64 bits."""
    logits, bias, E, k, G = s["logits"].double(), s["offset"], s["E"], s["k"], s["groups"]
    live = logits > -math.inf
    score = torch.sigmoid(logits) if s["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    value = logits if bias is None else score + bias.double()
    if G > 1:
        member = (score if bias is None else value).masked_fill(~live, -math.inf).unflatten(1, (G, E // G))
        if s["group_top"] == 1:
            # The largest score's order is the largest logit's.
            group = value.masked_fill(~live, -math.inf).unflatten(1, (G, E // G)).amax(2)
        else:
            top = member.topk(min(2, E // G), dim=2).values
            group = top[:, :, 0]
            if top.shape[2] == 2:
                group = group + torch.where(top[:, :, 1] > -math.inf, top[:, :, 1], torch.zeros_like(group))
        order = group.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, order, True)
        live = live & kept.repeat_interleave(E // G, dim=1)
    value, ids = value.masked_fill(~live, -math.inf).sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    return torch.where(value > -math.inf, ids, -1).to(torch.int32), value > -math.inf


def _positions(s):
    n = s["M"] * s["k"]
    p = torch.full((n + 1,), -1, dtype=torch.int64, device="cuda")
    at = torch.arange(s["routes"].numel(), device="cuda")
    p[torch.where(at < s["padded"], s["routes"], n).long()] = at
    return p[:n].view(s["M"], s["k"])


def _dequantised(s, e):
    """fp32 [N, K] of matrix e."""
    q = s["q"][e]
    v = torch.empty(*q.shape, 8, device="cuda")
    for slot, element in enumerate(SLOT):
        v[..., element] = (q >> (4 * slot)) & 15
    v = v.flatten(-2).unflatten(-1, (-1, s["g"]))
    return ((v - s["zeros"][e].unsqueeze(-1)) * s["scales"][e].view(torch.float16).float().unsqueeze(-1)).flatten(-2)


def _plain(s):
    op = s["op"]
    if op == "route":
        ids, live = _choose(s)
        l = s["logits"].float()
        chosen = l.gather(1, ids.clamp_min(0).long())
        if s["score"] == "sigmoid":
            score = torch.sigmoid(chosen)
        else:
            m = l.amax(1, keepdim=True)
            score = torch.exp(chosen - m) / torch.exp(l - m).sum(1, keepdim=True)
        score = torch.where(live, score, torch.zeros_like(score))
        if s["renormalize"]:
            score = score / score.sum(1, keepdim=True)
        return {"ids": ids, "w": torch.where(live, score * s["scale"], torch.zeros_like(score))}
    if op == "route_grad":
        l = s["logits"].float()
        live = s["ids"] >= 0
        at = s["ids"].clamp_min(0).long()
        g = torch.where(live, s["dw"], torch.zeros_like(s["dw"])) * s["scale"]
        if s["score"] == "sigmoid":
            p = torch.sigmoid(l.gather(1, at))
        else:
            p = torch.softmax(l, dim=1).gather(1, at)
        p = torch.where(live, p, torch.zeros_like(p))
        if s["renormalize"]:
            u = p / p.sum(1, keepdim=True)
            d = u * (g - (g * u).sum(1, keepdim=True))
            d = d * (1 - p) if s["score"] == "sigmoid" else d
        else:
            d = g * p * (1 - p) if s["score"] == "sigmoid" else g * p
        out = torch.zeros_like(l).scatter_add_(1, at, torch.where(live, d, torch.zeros_like(d)))
        if s["score"] == "softmax" and not s["renormalize"]:
            out = out - torch.softmax(l, dim=1) * (g * p).sum(1, keepdim=True)
        return out.to(s["logits"].dtype)
    if op == "matvec":
        out = DTYPES[s["out"]]
        x = s["x"].float()
        if s["ids"] is None:
            return torch.matmul(x, _dequantised(s, 0).T).to(out)
        y = torch.stack([_dequantised(s, s["ids"][t, j].long()) @ x[t]
                         for t in range(s["M"]) for j in range(s["k"])])
        return y.view(s["M"], s["k"], s["N"]).to(out)
    p = _positions(s)
    live = (p >= 0).unsqueeze(-1)
    if op == "combine":
        y = torch.zeros(s["M"], s["H"], device="cuda")
        for j in range(s["k"]):
            row = s["rows"][p[:, j].clamp_min(0)].float()
            y += torch.where(live[:, j], row, torch.zeros_like(row)) * s["w"][:, j:j + 1]
        return y.to(DTYPES[s["out"]])
    dy = s["dy"].float()
    dw = torch.zeros(s["M"], s["k"], device="cuda")
    for j in range(s["k"]):
        at, here = p[:, j], live[:, j, 0].nonzero().flatten()
        s["drows"][at[here]] = (dy[here] * s["w"][here, j:j + 1]).to(s["drows"].dtype)
        dw[here, j] = (dy[here] * s["rows"][at[here]].float()).sum(1)
    return {"drows": s["drows"], "dw": dw}


def run(s):
    if not own:
        return _plain(s)
    import mixture_experts_ffn_align_amd as moe
    op, M, k = s["op"], s["M"], s["k"]
    if op.startswith("route"):
        score = moe.MOE_SCORE_SOFTMAX if s["score"] == "softmax" else moe.MOE_SCORE_SIGMOID
        if op == "route_grad":
            dlogits = torch.empty_like(s["logits"])
            moe.moe_route_grad(s["logits"], s["ids"], s["dw"], dlogits, score=score, renormalize=s["renormalize"],
                               scale=s["scale"])
            return dlogits
        ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
        w = torch.empty(M, k, dtype=torch.float32, device="cuda")
        moe.moe_route(s["logits"], ids, w, bias=s["offset"], score=score, renormalize=s["renormalize"],
                      scale=s["scale"], groups=s["groups"], topk_groups=s["topk_groups"], group_top=s["group_top"])
        return {"ids": ids, "w": w}
    if op == "matvec":
        w = moe.DeviceProjection(moe.MOE_W_INT4_AWQ, s["g"], s["q"], s["scales"], s["zeros"])
        shape = (M, s["N"]) if s["ids"] is None else (M, k, s["N"])
        y = torch.empty(shape, dtype=DTYPES[s["out"]], device="cuda")
        moe.moe_matvec_int4(s["x"], w, y, topk_ids=s["ids"])
        return y
    positions = torch.empty(M, k, dtype=torch.int32, device="cuda")
    moe.moe_align_positions(s["routes"], s["padded"], positions)
    if op == "combine":
        y = torch.empty(M, s["H"], dtype=DTYPES[s["out"]], device="cuda")
        moe.moe_combine(s["rows"], positions, s["w"], y)
        return y
    dw = torch.empty(M, k, dtype=torch.float32, device="cuda")
    moe.moe_combine_grad(s["dy"], s["rows"], positions, s["w"], s["drows"], dw)
    return {"drows": s["drows"], "dw": dw}


def work(case):
    op, M, k = case["op"], case["M"], case["k"]
    if op == "matvec":
        N, K = case["N"], case["K"]
        used = min(case["E"], M * k) if k else 1
        rows = M * max(k, 1)
        size = used * (N * K / 2 + 3 * N * K / case["g"]) + 2 * M * K + DTYPES[case["out"]].itemsize * rows * N
        return {"bytes": size + 4 * M * k, "flops": 2 * rows * N * K}
    a = DTYPES[case["dtype"]].itemsize
    if op == "route":
        E = case["E"]
        return {"bytes": M * E * a + (4 * E if case["bias"] else 0) + 8 * M * k, "flops": 4 * M * E}
    if op == "route_grad":
        E = case["E"]
        read = E if case["score"] == "softmax" and not case["renormalize"] else k
        return {"bytes": M * (read + E) * a + 8 * M * k, "flops": 4 * M * read}
    H, live = case["H"], M * k * case["held"] / case["E"]
    size = live * H * a + DTYPES[case["out"]].itemsize * M * H + 4 * M * k + 4 * live
    if op == "combine":
        return {"bytes": size, "flops": 2 * live * H}
    return {"bytes": size + live * H * a + 4 * M * k, "flops": 3 * live * H}


def exact(case, seed):
    s = prepare(case, seed)
    op, M, k = case["op"], case["M"], case["k"]
    if op.startswith("route"):
        l = s["logits"].double()
        ids = _choose(s)[0] if op == "route" else s["ids"]
        here = torch.zeros_like(l)
        for j in range(k):                        # 1 for the experts chosen
            row = (ids[:, j] >= 0).nonzero().flatten()
            here[row, ids[row, j].long()] = 1.0
        if case["score"] == "sigmoid":
            p = 1.0 / (1.0 + torch.exp(-l))
        else:
            e = torch.exp(l - l.amax(1, keepdim=True))
            p = e / e.sum(1, keepdim=True)
        total = (p * here).sum(1, keepdim=True) if case["renormalize"] else torch.ones(M, 1, device="cuda").double()
        if op == "route":
            w = case["scale"] * (p / total).gather(1, ids.clamp_min(0).long())
            return {"ids": None, "w": torch.where(ids >= 0, w, torch.zeros_like(w))}
        g = torch.zeros_like(l)                   # the weights' gradient, by expert
        for j in range(k):
            row = (ids[:, j] >= 0).nonzero().flatten()
            g[row, ids[row, j].long()] = case["scale"] * s["dw"][row, j].double()
        # d(p / total): through p, and through total for the chosen
        dp = g / total
        if case["renormalize"]:
            dp = dp - here * (g * p).sum(1, keepdim=True) / total ** 2
        if case["score"] == "sigmoid":
            return dp * p * (1.0 - p)
        return p * (dp - (dp * p).sum(1, keepdim=True))
    if op == "matvec":
        unit = torch.empty(1, case["N"], case["K"], dtype=torch.float64, device="cuda")

        def product(e, x):
            words = s["q"][e].long() & 0xFFFFFFFF
            scale = s["scales"][e].view(torch.float16).double().repeat_interleave(case["g"], -1)
            zero = s["zeros"][e].double().repeat_interleave(case["g"], -1)
            for i in range(8):
                unit[0, :, SLOT[i]::8] = torch.bitwise_and(torch.bitwise_right_shift(words, 4 * i), 15).double()
            return x @ ((unit[0] - zero) * scale).T.contiguous()

        x = s["x"].double()
        if s["ids"] is None:
            return product(0, x)
        y = [product(int(e), x[t:t + 1]) for t, row in enumerate(s["ids"].tolist()) for e in row]
        return torch.cat(y).view(M, k, case["N"])
    n = M * k
    place = [-1] * n
    for p, r in enumerate(s["routes"].tolist()[:int(s["padded"])]):
        if r < n:
            place[r] = p
    place = torch.tensor(place, device="cuda").view(M, k)
    w, rows = s["w"].double(), s["rows"].double()
    if op == "combine":
        y = torch.zeros(M, case["H"], dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (place[:, j] >= 0).nonzero().flatten()
            y[t] += w[t, j, None] * rows[place[t, j]]
        return y
    dy = s["dy"].double()
    drows = torch.zeros_like(rows)
    dw = torch.zeros_like(w)
    for j in range(k):
        t = (place[:, j] >= 0).nonzero().flatten()
        drows[place[t, j]] = w[t, j, None] * dy[t]
        dw[t, j] = (rows[place[t, j]] * dy[t]).sum(1)
    return {"drows": drows, "dw": dw}
