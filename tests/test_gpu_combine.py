"""The weighted sum of routes (moe_combine), its gradient (moe_combine_grad) and
the inverse of an alignment (moe_align_positions) against 64-bit references:
exact on whole numbers, within the bounds of fp32 sums on random ones."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe
from tests import _route as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
SENTINEL = 77.0


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


def wide(v, dtype, pad):
    """Values on the GPU with `pad` columns of NaN between rows."""
    t = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    t[:, :v.shape[1]] = v.to("cuda").to(dtype)
    return t[:, :v.shape[1]]


def out(rows, cols, dtype, pad):
    return torch.full((rows, cols + pad), SENTINEL, dtype=dtype, device="cuda")


def places(gen, M, k, rows, absent):
    """Positions [M, k]: different rows, a share of them absent (before, behind and far outside)."""
    p = torch.randperm(rows, generator=gen)[:M * k]
    p = p.view(M, k).to(torch.int32)
    off = torch.rand(M, k, generator=gen) < absent
    bad = torch.tensor([-1, rows, -2 ** 31, 2 ** 31 - 1, rows + 5], dtype=torch.int32)
    return torch.where(off, bad[torch.randint(0, 5, (M, k), generator=gen)], p), off


# M, k, H, rows beyond the routes', share of routes without a row
CASES = [(1, 1, 8, 0, 0.0), (1, 8, 2048, 3, 0.0), (3, 2, 24, 1, 0.4), (21, 8, 264, 9, 0.2), (5, 9, 520, 0, 0.1),
         (2, 17, 2056, 4, 0.5), (37, 6, 72, 0, 1.0), (300, 3, 136, 7, 0.1), (1200, 2, 40, 0, 0.3), (1030, 10, 520, 2, 0.2)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "M%d_k%d_H%d_%d_%g" % c)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("ytype", TYPES, ids=str)
def test_exact_on_whole_numbers(case, dtype, ytype):
    M, k, H, more, absent = case
    g = torch.Generator().manual_seed(M + k + H)
    n = M * k + more
    pos, off = places(g, M, k, n, absent)
    rows = torch.randint(-8, 9, (n, H), generator=g).double()
    dy = torch.randint(-8, 9, (M, H), generator=g).double()
    w = torch.randint(-8, 9, (M, k), generator=g).float() / 8
    named = torch.zeros(n, dtype=torch.bool)
    named[pos[~off].long()] = True
    src = rows.clone()
    src[~named] = float("nan")                # rows no slot names are not read
    w[off] = float("nan")                     # nor are the weights of slots without a row
    announce("combine", case, dtype, ytype)
    rd, dyd, pd, wd = wide(src, dtype, 8), wide(dy, ytype, 16), pos.cuda(), w.cuda()
    y, drows = out(M, H, ytype, 8), out(n, H, dtype, 16)
    dw = torch.full((M, k), float("nan"), device="cuda")
    moe.moe_combine(rd, pd, wd, y[:, :H])
    moe.moe_combine_grad(dyd, rd, pd, wd, drows[:, :H], dw)
    torch.cuda.synchronize()
    ref, _ = R.combine(rows, pos, torch.nan_to_num(w), M, k)
    assert torch.equal(y[:, :H].double().cpu(), ref.to(ytype).double()) and bool((y[:, H:] == SENTINEL).all())
    want = torch.full((n, H), SENTINEL, dtype=torch.float64)
    ref_dw = torch.zeros(M, k, dtype=torch.float64)
    for t in range(M):
        for j in range(k):
            if not off[t, j]:
                want[pos[t, j]] = w[t, j].double() * dy[t]
                ref_dw[t, j] = (rows[pos[t, j]] * dy[t]).sum()
    assert torch.equal(drows[:, :H].double().cpu(), want.to(dtype).double()) and bool((drows[:, H:] == SENTINEL).all())
    assert torch.equal(dw.double().cpu(), ref_dw)
    # unit weights, and the gather: no weights, no rows
    y2 = out(M, H, ytype, 0)
    moe.moe_combine(rd, pd, None, y2)
    gathered = out(n, H, dtype, 0)
    moe.moe_combine_grad(dyd, None, pd, None, gathered, None)
    torch.cuda.synchronize()
    ref, _ = R.combine(rows, pos, None, M, k)
    assert torch.equal(y2.double().cpu(), ref.to(ytype).double())
    want = torch.full((n, H), SENTINEL, dtype=torch.float64)
    for t in range(M):
        want[pos[t][~off[t]].long()] = dy[t]
    assert torch.equal(gathered.double().cpu(), want.to(dtype).double())


@pytest.mark.parametrize("M,k,H", [(7, 8, 2048), (1100, 4, 776)])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_random_values(M, k, H, dtype):
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(M * k, H, generator=g).to(dtype)
    dy = torch.randn(M, H, generator=g).to(dtype)
    w = torch.rand(M, k, generator=g)
    pos, _ = places(g, M, k, M * k, 0.0)
    y, drows = out(M, H, dtype, 0), out(M * k, H, dtype, 0)
    dw = torch.empty(M, k, device="cuda")
    announce("combine random", M, k, H, dtype)
    moe.moe_combine(rows.cuda(), pos.cuda(), w.cuda(), y)
    moe.moe_combine_grad(dy.cuda(), rows.cuda(), pos.cuda(), w.cuda(), drows, dw)
    torch.cuda.synchronize()
    ref, mag = R.combine(rows, pos, w, M, k)
    sums = 2 * k * 2.0 ** -23 * mag             # k products and k sums, a whole step each
    tiny = 2.0 ** -25 if dtype == F16 else 1e-37
    assert bool(((y.double().cpu() - ref).abs() <= sums + HALF[dtype] * (ref.abs() + sums) + tiny).all())
    at = pos.flatten().long()
    exact = (w.double().unsqueeze(-1) * dy.double().unsqueeze(1)).flatten(0, 1)
    product = 2.0 ** -24 * exact.abs()
    assert bool(((drows.double().cpu()[at] - exact).abs() <= product + HALF[dtype] * (exact.abs() + product) + tiny).all())
    prod = rows.double()[at].view(M, k, H) * dy.double().unsqueeze(1)
    # A lane sums H / 64 products at most, then lanes and waves: every addition and product a whole step at most.
    bound = (H / 64 + 8 + 16) * 2.0 ** -23 * prod.abs().sum(2)
    assert bool(((dw.double().cpu() - prod.sum(2)).abs() <= bound).all())


def test_gradient_against_differences():
    # The sum is linear in rows and in weights, so whole steps give exact differences.
    g = torch.Generator().manual_seed(6)
    M, k, H = 4, 3, 16
    rows = torch.randint(-4, 5, (M * k, H), generator=g).float().cuda()
    w = (torch.randint(-4, 5, (M, k), generator=g).float() / 4).cuda()
    dy = torch.randint(-4, 5, (M, H), generator=g).float().cuda()
    pos, _ = places(g, M, k, M * k, 0.0)
    pos = pos.cuda()
    drows, dw = torch.empty_like(rows), torch.empty_like(w)
    announce("combine differences")
    moe.moe_combine_grad(dy, rows, pos, w, drows, dw)

    def loss():
        y = torch.empty(M, H, device="cuda")
        moe.moe_combine(rows, pos, w, y)
        return float((y * dy).sum())

    base = loss()
    for p, c in ((0, 0), (5, 7), (11, 15)):
        rows[p, c] += 1
        assert loss() - base == float(drows[p, c])
        rows[p, c] -= 1
    for t, j in ((0, 0), (2, 1), (3, 2)):
        w[t, j] += 1
        assert loss() - base == float(dw[t, j])
        w[t, j] -= 1


def test_infinite_and_nan_rows_stay_in_their_tokens():
    M, k, H = 6, 2, 64
    rows = torch.ones(M * k + 1, H)
    rows[0], rows[3, 5] = float("inf"), float("nan")
    rows[M * k] = float("nan")
    pos = torch.arange(M * k, dtype=torch.int32).view(M, k)
    pos[5] = -1
    w = torch.ones(M, k)
    w[5] = float("inf")
    y = torch.empty(M, H, device="cuda")
    dw = torch.empty(M, k, device="cuda")
    dy = torch.ones(M, H)
    dy[5] = float("inf")
    drows = torch.zeros(M * k + 1, H, device="cuda")
    announce("combine inf")
    moe.moe_combine(rows.cuda(), pos.cuda(), w.cuda(), y)
    moe.moe_combine_grad(dy.cuda(), rows.cuda(), pos.cuda(), w.cuda(), drows, dw)
    y, dw = y.cpu(), dw.cpu()
    assert bool((y[0] == float("inf")).all()) and int(y[1].isnan().sum()) == 1 and bool((y[2:5] == 2).all())
    assert bool((y[5] == 0).all()) and bool((dw[5] == 0).all()) and bool((dw[2:5] == H).all())
    assert bool((drows[10:] == 0).all())


def test_rows_in_route_order_and_no_rows():
    g = torch.Generator().manual_seed(7)
    rows = torch.randint(-4, 5, (15, 40), generator=g).double()
    w = torch.randint(-4, 5, (5, 3), generator=g).float()
    y = torch.empty(5, 40, device="cuda")
    announce("combine identity")
    moe.moe_combine(rows.float().cuda(), None, w.cuda(), y)
    assert torch.equal(y.cpu().double(), (rows.view(5, 3, 40) * w.double().unsqueeze(-1)).sum(1))
    moe.moe_combine(rows.float().cuda(), None, None, y)
    assert torch.equal(y.cpu().double(), rows.view(5, 3, 40).sum(1))
    drows = torch.empty(15, 40, device="cuda")
    moe.moe_combine_grad(y, None, None, None, drows, None)
    assert torch.equal(drows.view(5, 3, 40), y.unsqueeze(1).expand(5, 3, 40))
    # no rows at all: sums are zero, weights' gradients too
    none = torch.empty(0, 40, device="cuda")
    pos = torch.zeros(5, 3, dtype=torch.int32, device="cuda")
    dw = torch.full((5, 3), float("nan"), device="cuda")
    moe.moe_combine(none, pos, w.cuda(), y)
    moe.moe_combine_grad(y, none, pos, w.cuda(), none.clone(), dw)
    assert bool((y == 0).all()) and bool((dw == 0).all())
    assert moe.moe_combine(none, torch.empty(0, 3, dtype=torch.int32, device="cuda"), None, y[:0]) == moe.MOE_OK


@pytest.mark.parametrize("M,k,E,b", [(1, 1, 1, 1), (21, 8, 128, 8), (700, 4, 60, 16), (4096, 8, 128, 1), (5000, 8, 64, 64)])
def test_positions_invert_alignments(M, k, E, b):
    # A shard's alignment too: routes of other experts have no row.
    g = torch.Generator().manual_seed(M)
    ids = torch.rand(M, E, generator=g).topk(min(k, E), dim=1).indices.to(torch.int32).cuda()
    k = ids.shape[1]
    for base, held in ((0, E), (E // 3, max(1, E // 2))):
        cap = moe.moe_align_capacity(M, k, held, b)
        routes = torch.empty(cap, dtype=torch.int32, device="cuda")
        blocks = torch.empty(cap // b, dtype=torch.int32, device="cuda")
        n = torch.empty(1, dtype=torch.int32, device="cuda")
        announce("positions", M, k, E, b, base)
        moe.moe_align_ex(ids, held, base, b, routes, blocks, n)
        pos = torch.full((M, k), -77, dtype=torch.int32, device="cuda")
        moe.moe_align_positions(routes, n, pos)
        pos = pos.cpu().flatten()
        here = ((ids >= base) & (ids < base + held)).cpu().flatten()
        assert torch.equal(pos == -1, ~here)
        assert torch.equal(routes.cpu()[pos[here].long()].long(), here.nonzero().flatten())


def test_positions_of_odd_arrays():
    # Entries past num_padded do not count; num_padded past the array, negative entries and entries that
    # are no routes do no harm.
    routes = torch.tensor([4, -5, 2, 6, 2 ** 31 - 1, 0, 1, 3], dtype=torch.int32, device="cuda")
    announce("positions odd")
    for n, want in ((0, [-1] * 6), (4, [-1, -1, 2, -1, 0, -1]), (7, [5, 6, 2, -1, 0, -1]), (-3, [-1] * 6),
                    (2 ** 31 - 1, [5, 6, 2, 7, 0, -1])):
        pos = torch.full((3, 2), -77, dtype=torch.int32, device="cuda")
        moe.moe_align_positions(routes, torch.tensor([n], dtype=torch.int32, device="cuda"), pos)
        assert pos.flatten().tolist() == want
    big = torch.full((300, 300), -77, dtype=torch.int32, device="cuda")       # two launches
    moe.moe_align_positions(routes, torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda"), big)
    assert big.flatten()[:7].tolist() == [5, 6, 2, 7, 0, -1, 3] and bool((big.flatten()[7:] == -1).all())


def test_graph():
    g = torch.Generator().manual_seed(8)
    M, k, H, E = 5000, 8, 64, 16
    ids = torch.rand(M, E, generator=g).topk(k, dim=1).indices.to(torch.int32).cuda()
    routes = torch.empty(M * k, dtype=torch.int32, device="cuda")
    blocks, n = torch.empty_like(routes), torch.empty(1, dtype=torch.int32, device="cuda")
    pos = torch.empty(M, k, dtype=torch.int32, device="cuda")
    x, w = torch.randn(M, H, device="cuda"), torch.rand(M, k, device="cuda")
    rows, y = torch.zeros(M * k, H, device="cuda"), torch.empty(M, H, device="cuda")
    drows, dw = torch.zeros_like(rows), torch.empty_like(w)

    def call():
        moe.moe_align(ids, E, 1, routes, blocks, n)
        moe.moe_align_positions(routes, n, pos)
        moe.moe_combine_grad(x, None, pos, None, rows, None)
        moe.moe_combine(rows, pos, w, y)
        moe.moe_combine_grad(y, rows, pos, w, drows, dw)

    announce("combine graph")
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(4):
        ids.copy_(torch.rand(M, E, generator=g).topk(k, dim=1).indices)
        x.normal_(), rows.zero_(), drows.zero_(), pos.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (pos, rows, y, drows, dw)]
        rows.zero_(), drows.zero_(), pos.zero_()
        call()
        assert all(torch.equal(a, b) for a, b in zip(got, (pos, rows, y, drows, dw)))
        # k products and sums with weights that add up to k at most
        assert torch.allclose(y, x * w.sum(1, keepdim=True), rtol=0, atol=float(16 * 2.0 ** -23 * k * x.abs().max()))
