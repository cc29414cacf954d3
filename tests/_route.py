"""64-bit references of routing, the weighted sum of routes and the products
with packed 4-bit weights, written from their definitions, and the bounds the
fp32 arithmetic of the kernels has to keep."""
import numpy as np
import torch

SOFTMAX, SIGMOID = 0, 1
SLOT = (0, 2, 4, 6, 1, 3, 5, 7)     # element of nibble slot i


def scores(logits, score):
    """fp64 scores [M, E] of logits (any float type)."""
    l = logits.double()
    if score == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -np.inf, torch.zeros_like(top), top))   # an infinite logit: all NaN
    return e / e.sum(1, keepdim=True)


def rank_key(v):
    """Sort key: NaN above every number."""
    return (1, 0.0) if np.isnan(v) else (0, v)


def choose(logits, k, score, bias=None, groups=1, topk_groups=1, group_top=1):
    """ids [M, k] int32: one row at a time, by sorting."""
    M, E = logits.shape
    l = logits.double().numpy()
    s = scores(logits, score).numpy()
    b = None if bias is None else bias.double().numpy()
    size = E // groups
    ids = np.full((M, k), -1, dtype=np.int32)
    for t in range(M):
        value, member = {}, {}
        for e in range(E):
            if l[t, e] == -np.inf or (b is not None and b[e] == -np.inf):
                continue
            member[e] = s[t, e] if b is None else s[t, e] + b[e]
            value[e] = l[t, e] if b is None else member[e]
        if topk_groups < groups:
            rank = []
            for g in range(groups):
                mine = [e for e in member if e // size == g]
                if not mine:
                    rank.append(((-1, 0.0), g))
                    continue
                if group_top == 1:
                    rank.append((max(rank_key(value[e]) for e in mine), g))
                else:
                    top = sorted((rank_key(member[e]) for e in mine), reverse=True)[:2]
                    rank.append(((max(x[0] for x in top), 0.0 if top[0][0] else sum(x[1] for x in top)), g))
            rank.sort(key=lambda x: (-x[0][0], -x[0][1], x[1]))
            kept = {g for _, g in rank[:topk_groups]}
            value = {e: v for e, v in value.items() if e // size in kept}
        order = sorted(value, key=lambda e: (-rank_key(value[e])[0], -rank_key(value[e])[1], e))
        ids[t, :min(k, len(order))] = order[:k]
    return torch.from_numpy(ids)


def weights(logits, ids, score, renormalize, scale):
    """fp64 weights [M, k] of the experts in ids (-1: weight 0)."""
    p = scores(logits, score)
    live = ids >= 0
    w = torch.where(live, p.gather(1, ids.clamp_min(0).long()), torch.zeros(1, dtype=torch.float64))
    if renormalize:
        if score == SIGMOID:       # a common factor, so that small scores do not vanish
            l = torch.where(live, logits.double().gather(1, ids.clamp_min(0).long()),
                            torch.full((1,), -np.inf, dtype=torch.float64))
            m = l.amax(1, keepdim=True).clamp_max(0.0)
            m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
            w = torch.where(live, torch.exp(l.clamp_max(0.0) - m) / (1.0 + torch.exp(-l.abs())), torch.zeros_like(w))
        else:
            l = torch.where(live, logits.double().gather(1, ids.clamp_min(0).long()),
                            torch.full((1,), -np.inf, dtype=torch.float64))
            m = l.amax(1, keepdim=True)
            m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
            w = torch.where(live, torch.exp(l - m), torch.zeros_like(w))
        w = w / w.sum(1, keepdim=True)
    return torch.where(live, scale * w, torch.zeros_like(w))


def logits_grad(logits, ids, g, score, renormalize, scale):
    """fp64 gradient [M, E] of sum(weights * g) by autograd of the definition in 64 bits, and the
    magnitudes of what it sums."""
    l = logits.double().clone().requires_grad_(True)
    live = ids >= 0
    at = ids.clamp_min(0).long()
    p = torch.sigmoid(l) if score == SIGMOID else torch.softmax(l, dim=1)
    chosen = torch.where(live, p.gather(1, at), torch.zeros(1, dtype=torch.float64))
    w = chosen / chosen.sum(1, keepdim=True) if renormalize else chosen
    gg = torch.where(live, g.double(), torch.zeros(1, dtype=torch.float64))
    w = torch.where(live, w, torch.zeros_like(w))
    (scale * w * gg).sum().backward()
    spread = abs(scale) * (w * gg.abs()).sum(1, keepdim=True)
    each = torch.zeros_like(p).scatter_add(1, at, torch.where(live, abs(scale) * w * (gg.abs()), torch.zeros_like(w)))
    share = torch.zeros_like(p).scatter_add(1, at, w) if renormalize or score == SIGMOID else p
    mag = each + share * spread
    return l.grad.detach(), mag.detach()


def weight_bound(logits, terms):
    """Relative error of fp32 weights: an exponential's argument is off by half a step of at most
    `spread` (differences beyond 104 vanish), the exponential, its division and each of `terms`
    additions by a few half steps."""
    l = logits.double()
    fin = torch.where(torch.isfinite(l), l, torch.zeros_like(l))
    spread = (fin.amax(1) - fin.amin(1)).clamp_max(104.0)
    return (2.0 ** -23 * (spread + terms + 16)).unsqueeze(1)


def combine(rows, positions, w, M, k):
    """(fp64 sums [M, H], magnitudes) over the slots that have a row."""
    y = torch.zeros(M, rows.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(y)
    for t in range(M):
        for j in range(k):
            p = int(positions[t, j])
            if 0 <= p < rows.shape[0]:
                v = rows[p].double() * (1.0 if w is None else float(w[t, j]))
                y[t] += v
                mag[t] += v.abs()
    return y, mag


def dequantise(q, s, z, group):
    """fp64 [E, N, K] of packed words (int32), scales and zeros [E, N, K / group]."""
    words = q.long() & 0xFFFFFFFF
    v = torch.empty(*q.shape, 8, dtype=torch.float64)
    for i in range(8):
        v[..., SLOT[i]] = ((words >> (4 * i)) & 15).double()
    v = v.flatten(-2)
    return (v - z.double().repeat_interleave(group, -1)) * s.double().repeat_interleave(group, -1)
