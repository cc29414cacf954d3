"""Inputs and 64-bit references for the products on ragged rows and MXFP4.

Most inputs are small integers: their products and sums are whole numbers
below 2^24, exact in fp32 whatever the order, so the kernels' fp32 results must
equal the reference and their 16-bit results its one rounding, bit for bit."""
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)

# counts per expert; head and tail: rows before the first and after the last expert's
SHAPES = [
    dict(counts=[1], N=8, K=8),
    dict(counts=[2], N=16, K=32, tail=3),
    dict(counts=[0, 1, 17, 0, 40], N=24, K=40, head=2, tail=5),
    dict(counts=[129, 0, 64], N=136, K=200, tail=1),
    dict(counts=[(7 * e) % 10 for e in range(70)], N=64, K=72, head=1),
    dict(counts=[300, 513], N=520, K=264),
    dict(counts=[0, 0, 0], N=40, K=48, tail=4),
    dict(counts=[3] + [0] * 128 + [2], N=96, K=64),
    dict(counts=[65, 31, 32, 33, 1], N=72, K=1032),
    dict(counts=[1100, 700, 5], N=264, K=520, head=3, tail=2),
    dict(counts=[16, 15, 17, 0, 1, 2, 4, 8], N=2048, K=768),
    # more than 256 experts, and the most
    dict(counts=[(5 * e) % 4 for e in range(300)], N=72, K=40, head=1, tail=1),
    dict(counts=[(3 * e) % 2 for e in range(2048)], N=8, K=8),
]

# Enough tasks for the larger tiles, in every direction: ends inside tiles,
# experts without rows, summed extents of one slab, of odd ones and of many.
LARGE = [
    dict(counts=[700, 20, 0, 333, 901], N=2056, K=2056, head=5, tail=3),
    dict(counts=[257, 128, 511, 64], N=2048, K=1544),
    dict(counts=[1, 1500, 3], N=3096, K=3080, tail=130),
    # whole tiles only, several to a workgroup
    dict(counts=[1024, 2048], N=4096, K=192),
    dict(counts=[1024, 2048], N=192, K=4096),
]
# Rows per expert for the largest forward tiles (a small K, and one with a tail of eight).
TALL = [dict(counts=[16500], N=2056, K=64), dict(counts=[5000, 12000], N=2048, K=200, tail=7)]


def shape_id(s):
    c = s["counts"]
    return f"E{len(c)}_rows{sum(c)}_N{s['N']}_K{s['K']}_h{s.get('head', 0)}_t{s.get('tail', 0)}"


def offsets_of(s):
    """(offsets [E + 1] int32, rows) of a shape."""
    o = [s.get("head", 0)]
    for c in s["counts"]:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32), o[-1] + s.get("tail", 0)


def whole(gen, *shape, top=4):
    """Small whole numbers as fp64."""
    return torch.randint(-top, top + 1, shape, generator=gen).double()


def owned(offsets, rows):
    m = torch.zeros(rows, dtype=torch.bool)
    m[int(offsets[0]):int(offsets[-1])] = True
    return m


def forward(x, w, offsets):
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        y[a:b] = x[a:b] @ w[e].T
    return y


def input_grad(dy, w, offsets):
    return forward(dy, w.transpose(1, 2), offsets)


def weight_grad(dy, x, offsets):
    E = offsets.numel() - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        dw[e] = dy[a:b].T @ x[a:b]
    return dw


def half_step(dtype):
    return {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]


def tolerance(ref, magnitudes, terms, dtype):
    """Largest error of a sum of `terms` exact products whose magnitudes sum to
    `magnitudes`: each fp32 addition is off by at most 2^-23 of a partial sum no
    larger than `magnitudes` (a whole step, whatever the unit's rounding), then
    one rounding to `dtype` (half a step, or half the smallest subnormal)."""
    sums = terms * 2.0 ** -23 * magnitudes
    return sums + half_step(dtype) * (ref.abs() + sums) + (2.0 ** -25 if dtype == torch.float16 else 1e-38)


def codes_to_values(q, scale):
    """fp64 values of packed MXFP4 codes and exponent bytes."""
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    unit = torch.where(scale == 255, torch.full_like(scale, 0, dtype=torch.float64) * float("nan"),
                       torch.exp2(scale.double() - 127))
    return (E2M1[c].unflatten(-1, (-1, 32)) * unit.unsqueeze(-1)).flatten(-2)


def quantise(x):
    """(packed codes, exponent bytes) of fp64 x [.., K], by the definition: the
    nearest of the eight magnitudes, a tie to the even code."""
    blocks = x.unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(blocks).all(-1)
    safe = torch.where(bad.unsqueeze(-1), torch.zeros_like(blocks), blocks)
    m = safe.abs().amax(-1)
    e = torch.frexp(m).exponent - 1 - 2
    e = torch.where(m > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    v = safe / torch.exp2(e.double()).unsqueeze(-1)
    d = (v.abs().unsqueeze(-1) - E2M1[:8]).abs()
    near = d == d.amin(-1, keepdim=True)
    even_first = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])
    code = even_first[near[..., even_first].int().argmax(-1)] + 8 * torch.signbit(v).long()
    code = torch.where(bad.unsqueeze(-1), torch.zeros_like(code), code).flatten(-2)
    q = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    return q, torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
