"""moe_align_positions of routes that several rows name, and of more routes and
rows than its workgroups take in one turn."""
import pytest
import torch

import mixture_experts_ffn_align_amd as moe

pytestmark = pytest.mark.gpu


def announce(*parts):
    print("[gpu-case]", *parts, flush=True)


def positions(rows, n, routes):
    pos = torch.full((routes, 1), -77, dtype=torch.int32, device="cuda")
    moe.moe_align_positions(rows.to(torch.int32).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), pos)
    return pos.flatten().cpu()


# Rows, routes and rows that count: one workgroup, and several.
@pytest.mark.parametrize("rows,routes,n", [(4096, 2048, 4096), (4000, 4096, 3999), (200000, 100000, 199999)])
def test_routes_of_several_rows_get_one_of_them(rows, routes, n):
    # No alignment has them; nothing else is disturbed.
    g = torch.Generator().manual_seed(rows)
    r = torch.arange(rows) % routes
    r[torch.randperm(rows, generator=g)[:rows // 3]] = -1
    announce("positions repeated", rows, routes, n)
    got = positions(r, n, routes)
    named = torch.zeros(routes, dtype=torch.bool)
    named[r[:n][r[:n] >= 0]] = True
    assert torch.equal(got >= 0, named) and bool((got < n).all())
    assert torch.equal(r[got[named].long()], named.nonzero().flatten())


def test_more_routes_and_rows_than_one_turn():
    # The fill's workgroups take 2^20 routes a turn, the scatter's 2^22 rows.
    g = torch.Generator().manual_seed(1)
    routes, rows = 2 ** 20 + 4097, 2 ** 23 + 12345
    r = torch.full((rows,), -1, dtype=torch.int64)
    at = torch.randperm(rows, generator=g)[:routes - 100]
    r[at] = torch.arange(routes - 100)
    want = torch.full((routes,), -1, dtype=torch.int32)
    want[:routes - 100] = at.to(torch.int32)
    announce("positions turns")
    assert torch.equal(positions(r, rows, routes), want)
