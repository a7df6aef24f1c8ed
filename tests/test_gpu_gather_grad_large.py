"""The gather gradient of large batches on the GPU, where a warp takes several tokens: ragged last groups, tokens with no
local row between others, and the selections that stay at one token a warp."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt

from test_gpu_route_grads import U, routes, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,H,bs,El", [
    (40001, 24, 6, 64, 8, 6),      # four tokens a warp, most of them without a row or with one
    (40003, 24, 6, 64, 8, None),
    (40002, 160, 8, 264, 24, 20),  # four times eight slots: every lane has one
    (150001, 5, 1, 8, 1, 1),
    (20001, 64, 16, 64, 8, 16),    # two tokens a warp
    (20003, 13, 3, 520, 16, None), # two column segments a row
    (20001, 40, 17, 64, 8, 10),    # too many slots for two tokens a warp
    (20001, 32, 32, 72, 1, None),
])
def test_gather_backward(T, E, k, H, bs, El):
    _, al, status = routes(T, E, k, bs, El, seed=T + k)
    gp = torch.randn((al.capacity, H), generator=torch.Generator("cuda").manual_seed(T), device="cuda").to(torch.bfloat16)
    pad = torch.ones(al.capacity, dtype=torch.bool, device="cuda")
    pad[al.inv_perm[al.inv_perm >= 0].long()] = False
    gp[pad] = float("nan")  # pad rows are not read
    gx = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    tdt.moe_gather_backward(gp, al.inv_perm, k, gx[:T], device_status=status)
    inv = al.inv_perm.long().view(T, k)
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for j in range(k):
        row = torch.where((inv[:, j] >= 0)[:, None], gp[inv[:, j].clamp(min=0)].double(), 0.0)
        want += row
        size += row.abs()
    # sums of k terms in fp32 (1.01: their second order), rounded to bf16
    within(gx[:T], want, want.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + 1.01 * k * U * size + 2.0 ** -133, "grad")
    assert (gx[:T][(inv < 0).all(1)] == 0).all() and (gx[T] == 7).all()
    assert tdt.moe_read_status(status) == tdt.MOE_OK
    # bad rows in a group of tokens: left out, the others as they were
    bad = al.inv_perm.clone()
    bad[5 * k], bad[(T - 1) * k] = al.capacity, -7
    got = tdt.moe_gather_backward(gp, bad, k, device_status=status)
    assert tdt.moe_read_status(status) == tdt.MOE_ERR_BAD_ROW
    same = torch.ones(T, dtype=torch.bool, device="cuda")
    same[5] = same[T - 1] = False
    assert torch.equal(got[same], gx[:T][same])
