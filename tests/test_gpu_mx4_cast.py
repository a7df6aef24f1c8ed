"""Microscaled 4-bit floating point on the GPU: every code and scale byte against the format's definition in 64 bits."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def reference(x):
    """x [rows, K] bf16 (CPU) -> codes [rows, K] int, scale bytes [rows, K/32] int."""
    rows, K = x.shape
    b = x.double().view(rows, K // 32, 32)
    bad = ~torch.isfinite(b).all(-1)
    top = torch.where(bad, 1.0, b.abs().amax(-1))
    s = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 2, -127.0).clamp(-127, 127)
    a = b.abs() / torch.exp2(s)[..., None]
    dist = (a[..., None] - GRID).abs()
    best = dist.amin(-1, keepdim=True)
    near = dist == best
    even = near & (torch.arange(8) % 2 == 0)  # a tie lies between an even and an odd code
    pick = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))
    codes = pick + 8 * torch.signbit(b).int()
    codes[bad] = 0
    byte = torch.where(bad, 255, (s + 127).int())
    return codes.view(rows, K), byte


def values(codes, byte):
    v = GRID[codes & 7] * torch.where(codes >= 8, -1.0, 1.0)
    scale = torch.where(byte == 255, float("nan"), torch.exp2(byte.double() - 127))
    return v * scale.repeat_interleave(32, 1)


def unpack(q):
    c = q.codes.cpu().int()
    codes = torch.stack((c & 15, c >> 4), -1).view(q.rows, q.K)
    byte = q.scales.cpu().int().permute(1, 0, 2).reshape(q.rows, -1)
    return codes, byte[:, :q.K // 32], byte[:, q.K // 32:]


def check(x):
    q = tdt.moe_quantize_mx4(x.cuda())
    codes, byte, rest = unpack(q)
    want_codes, want_byte = reference(x)
    assert torch.equal(byte, want_byte) and torch.equal(codes, want_codes.int())
    assert (rest == 127).all()
    back = tdt.moe_dequantize_mx4(q).cpu()
    want = values(want_codes, want_byte)
    assert torch.equal(back.isnan(), want.isnan())
    assert torch.equal(back.double().nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
    return q


@pytest.mark.parametrize("rows,K", [(1, 32), (1, 64), (3, 96), (5, 128), (2, 160), (33, 256), (7, 288), (130, 2048),
                                    (9, 7168), (1, 4128), (1000, 32)])
def test_quantize_rows(rows, K):
    require_gpu()
    g = torch.Generator().manual_seed(rows + K)
    check((torch.randn((rows, K), generator=g) * 3).to(torch.bfloat16))


def test_every_bf16_value():
    """All finite bf16 values of each exponent share blocks with a leader of their own exponent and of others."""
    require_gpu()
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16)
    x = x[torch.isfinite(x)]
    check(x.view(-1, 32))  # blocks of neighbours
    g = torch.Generator().manual_seed(0)
    check(x[torch.randperm(x.numel(), generator=g)].view(-1, 32))


def test_ties_zeros_and_special_blocks():
    require_gpu()
    x = torch.zeros((6, 64))
    x[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0])
    x[0, 8:16] = -x[0, :8]
    x[1, 3], x[1, 40] = float("inf"), 2.0
    x[2, 31], x[2, 32] = float("nan"), -0.0
    x[3, :32] = 7.9  # saturates
    x[4, 0] = 2.0 ** -133  # the smallest bf16: below the smallest scale's half code
    x[5, 5], x[5, 6] = 3.3e38, 2.0 ** -100
    check(x.to(torch.bfloat16))


@pytest.mark.parametrize("byte", [0, 1, 126, 127, 128, 251, 252, 253, 254, 255])
def test_dequantize_any_scale_byte(byte):
    """Values past bf16's range become infinities, values below it round to nearest."""
    require_gpu()
    codes = torch.arange(16, dtype=torch.uint8)
    q = tdt.Mx4Tensor((codes | (codes.flip(0) << 4)).view(1, 16).cuda(),
                      torch.full((1, 1, 4), byte, dtype=torch.uint8, device="cuda"))
    got = tdt.moe_dequantize_mx4(q).cpu()
    c = torch.stack((codes, codes.flip(0)), -1).view(1, 32).long()
    want = values(c, torch.full((1, 1), byte)).to(torch.bfloat16)
    assert torch.equal(got.nan_to_num(nan=3.0), want.nan_to_num(nan=3.0))


@pytest.mark.parametrize("T,E,k,H,bs,El", [(1, 1, 1, 32, 1, None), (2, 160, 6, 4096, 8, 40), (64, 8, 2, 256, 16, None),
                                           (333, 60, 4, 288, 7, None), (50, 40, 32, 160, 24, 10),
                                           (700, 128, 8, 2048, 64, None)])
def test_gather_mx4(T, E, k, H, bs, El):
    """Each local slot's row is the quantised token row; no other row changes."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(T)
    ids = torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32).to(dev)
    emap = None
    if El is not None:
        emap = torch.full((E,), -1, dtype=torch.int32)
        emap[:El] = torch.arange(El, dtype=torch.int32)
        emap = emap.to(dev)
    al = tdt.moe_align_permute(ids, E, bs, emap, El or E)
    h = torch.randn((T, H), generator=g).to(torch.bfloat16).to(dev)
    out = tdt.alloc_mx4(al.capacity, H, dev)
    out.codes.fill_(0x5A)
    out.scales.fill_(0xA5)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    q = tdt.moe_gather_mx4(h, k, al.inv_perm, al.capacity, out=out, device_status=status)
    whole = tdt.moe_quantize_mx4(h)
    want_c, want_s = torch.full_like(out.codes, 0x5A), torch.full_like(out.scales, 0xA5)
    local = al.inv_perm >= 0
    rows, token = al.inv_perm[local].long(), torch.arange(T * k, device=dev)[local] // k
    want_c[rows], want_s[:, rows] = whole.codes[token], whole.scales[:, token]
    assert torch.equal(q.codes, want_c) and torch.equal(q.scales, want_s)
    assert tdt.moe_read_status(status) == tdt.MOE_OK
    inv = al.inv_perm.clone()
    inv[0] = al.capacity
    tdt.moe_gather_mx4(h, k, inv, al.capacity, device_status=status)
    assert tdt.moe_read_status(status) == tdt.MOE_ERR_BAD_ROW


def test_empty():
    require_gpu()
    q = tdt.moe_quantize_mx4(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert tdt.moe_dequantize_mx4(q).shape == (0, 64)


@pytest.mark.parametrize("n", [0, 1, 5, 9])
def test_rows_behind_the_last_are_left(n):
    require_gpu()
    x = torch.randn((9, 160), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    out = tdt.alloc_mx4(9, 160, "cuda")
    out.codes.fill_(0x5A)
    out.scales.fill_(0xA5)
    tdt.moe_quantize_mx4(x, out, num_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
    whole = tdt.moe_quantize_mx4(x)
    assert torch.equal(out.codes[:n], whole.codes[:n]) and torch.equal(out.scales[:, :n], whole.scales[:, :n])
    assert (out.codes[n:] == 0x5A).all() and (out.scales[:, n:] == 0xA5).all()
