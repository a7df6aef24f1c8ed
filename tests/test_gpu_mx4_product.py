"""The experts' product in microscaled 4-bit floating point on the GPU, against a product in 64 bits of the same codes
and scales."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def random_mx4(gen, rows, K, spread=3):
    """Random codes and scales of 2^-spread .. 2^spread."""
    return tdt.Mx4Tensor(torch.randint(0, 256, (rows, K // 2), generator=gen, dtype=torch.uint8).cuda(),
                         torch.randint(127 - spread, 128 + spread, (-(-K // 128), rows, 4), generator=gen,
                                       dtype=torch.uint8).cuda())


def values(q):
    c = q.codes.long()
    v = GRID.cuda()[torch.stack((c & 15, c >> 4), -1).view(q.rows, q.K)]
    byte = q.scales.permute(1, 0, 2).reshape(q.rows, -1)[:, :q.K // 32].double()
    scale = torch.where(byte == 255, float("nan"), torch.exp2(byte - 127))
    return v * scale.repeat_interleave(32, 1)


def layout(counts, bs):
    counts = torch.tensor(counts, dtype=torch.int32)
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.cumsum((counts + bs - 1) // bs * bs, 0)
    return counts, off, int(counts.sum()) + len(counts) * (bs - 1)


def reference(x, w, counts, off, N, gate):
    """Per expert: rows, values and the tolerance of the fp32 arithmetic (see below)."""
    K = x.shape[1]
    for e, n in enumerate(counts.tolist()):
        r = slice(int(off[e]), int(off[e]) + n)
        we = w[e * N:(e + 1) * N]
        y, mag = x[r] @ we.T, x[r].abs() @ we.abs().T
        # products are exact; the sum of K terms in groups of 32: a step of rounding or truncation (2^-23) each
        err = (K / 32 + 8) * 2.0 ** -23 * mag
        if gate:
            a, b, ea, eb = y[:, :N // 2], y[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
            s = a * torch.sigmoid(a)
            y = s * b
            # |silu'| <= 1.1; the exponential is off by 2 + 1.2 |a| steps, the quotient by 2, the product by 1
            err = 1.1 * ea * (b.abs() + eb) + s.abs() * eb + y.abs() * (6 + 1.2 * a.abs()) * 2.0 ** -23
        yield r, y, err + y.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -126


def run_and_check(x, w, counts, off, N, gate=False, status=None):
    cap, cols = x.rows, N // 2 if gate else N
    out = torch.full((cap, cols), 77.0, dtype=torch.bfloat16, device="cuda")
    got = tdt.moe_grouped_gemm_mx4(x, w, counts.cuda(), off.cuda(), out=out, swiglu=gate, device_status=status)
    seen = torch.zeros(cap, dtype=torch.bool)
    for r, y, tol in reference(values(x), values(w), counts, off, N, gate):
        seen[r] = True
        d = (got[r].double() - y).abs()
        ok = (d <= tol) | (y.isnan() & got[r].isnan())
        assert ok.all(), f"rows {r}: {(~ok).sum().item()} of {ok.numel()} beyond the tolerance, by {(d - tol).max().item():.3g}"
    assert (got[~seen.cuda()] == 77.0).all()
    return got


LAYOUTS = [([1], 1), ([3, 0, 17, 1], 8), ([0, 0, 5], 16), ([128, 127, 129, 0, 300], 64), ([33, 64, 1, 250], 24),
           ([7, 9, 16, 31, 32, 15], 1)]


@pytest.mark.parametrize("counts,bs", LAYOUTS)
@pytest.mark.parametrize("K,N,gate", [(32, 8, False), (64, 128, False), (256, 136, False), (288, 200, False),
                                      (1056, 384, False), (32, 16, True), (160, 128, True), (512, 272, True),
                                      (2048, 768, True)])
def test_product(counts, bs, K, N, gate):
    require_gpu()
    gen = torch.Generator().manual_seed(K + N)
    counts, off, cap = layout(counts, bs)
    x, w = random_mx4(gen, max(cap, 1), K), random_mx4(gen, len(counts) * N, K)
    x.scales[:, int(off[-1]):] = 255  # rows of no expert hold NaN
    for q in (x, w):  # and so do the bytes past K
        q.scales[-1, :, (K % 128 or 128) // 32:] = 255
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_and_check(x, w, counts, off, N, gate, status)
    assert tdt.moe_read_status(status) == tdt.MOE_OK


def test_many_experts_few_rows_and_long_k():
    """More tiles than CTAs, the largest expert count, a long K."""
    require_gpu()
    gen = torch.Generator().manual_seed(0)
    counts, off, cap = layout([(i * 7) % 5 for i in range(1024)], 8)
    run_and_check(random_mx4(gen, cap, 64), random_mx4(gen, 1024 * 40, 64), counts, off, 40)
    counts, off, cap = layout([200, 700], 128)
    run_and_check(random_mx4(gen, cap, 7168), random_mx4(gen, 2 * 1024, 7168), counts, off, 1024, True)


def test_each_scale_and_code_has_its_place():
    """One code and one scale at a time: a row's block i meets a weight row's block i, and nothing else does."""
    require_gpu()
    K, N, n = 512, 128, 130
    counts, off, cap = layout([n], 1)
    x = tdt.Mx4Tensor(torch.zeros((n, K // 2), dtype=torch.uint8, device="cuda"),
                      torch.full((4, n, 4), 127, dtype=torch.uint8, device="cuda"))
    w = tdt.Mx4Tensor(torch.full((N, K // 2), 0x22, dtype=torch.uint8, device="cuda"),
                      torch.empty((4, N, 4), dtype=torch.uint8, device="cuda"))
    block = torch.arange(16, dtype=torch.uint8).view(4, 1, 4)
    feature = torch.arange(N, dtype=torch.uint8).view(1, N, 1)
    w.scales.copy_(100 + block + feature % 13)
    for r in range(n):  # row r has a single 1.0, in column (r * 37) % K
        c = (r * 37) % K
        x.codes[r, c // 2] = 0x02 << (4 * (c % 2))
    run_and_check(x, w, counts, off, N)


def test_nan_blocks_stay_in_their_row_and_feature():
    require_gpu()
    gen = torch.Generator().manual_seed(3)
    K, N = 320, 128
    counts, off, cap = layout([40, 20], 8)
    x, w = random_mx4(gen, cap, K), random_mx4(gen, 2 * N, K)
    x.scales[1, 5, 2] = 255
    w.scales[0, 17, 0] = 255  # expert 0's feature 17
    got = run_and_check(x, w, counts, off, N)
    nan = got[:40].isnan()
    assert nan[5].all() and nan[:, 17].all() and nan.sum() == N + 40 - 1 and not got[40:60].isnan().any()


def test_bad_counts_and_offsets_are_skipped_and_recorded():
    require_gpu()
    gen = torch.Generator().manual_seed(4)
    K, N = 64, 64
    counts, off, cap = layout([10, 10, 10, 10], 16)
    x, w = random_mx4(gen, cap, K), random_mx4(gen, 4 * N, K)
    good = run_and_check(x, w, counts, off, N)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad_c, bad_o = counts.clone(), off.clone()
    bad_c[1], bad_o[2], bad_o[3] = -3, cap - 5, -8
    out = torch.full_like(good, 77.0)
    tdt.moe_grouped_gemm_mx4(x, w, bad_c.cuda(), bad_o.cuda(), out=out, device_status=status)
    assert tdt.moe_read_status(status) == tdt.MOE_ERR_BAD_ROW
    assert torch.equal(out[:10], good[:10]) and (out[10:] == 77.0).all()
    # every expert claims every row: too many to be ranges of their own
    all_c, all_o = torch.full_like(counts, cap), torch.zeros_like(off)
    tdt.moe_grouped_gemm_mx4(x, w, all_c.cuda(), all_o.cuda(), out=out.fill_(77.0), device_status=status)
    assert (out == 77.0).all() and tdt.moe_read_status(status) == tdt.MOE_ERR_BAD_ROW
    # no expert has a row
    tdt.moe_grouped_gemm_mx4(x, w, torch.zeros_like(counts).cuda(), off.cuda(), out=out.fill_(77.0), device_status=status)
    assert (out == 77.0).all() and tdt.moe_read_status(status) == tdt.MOE_OK


def test_layer_of_4_bit_experts():
    """MoeRouter.step_mx4, eager and as a replayed graph: every product against 64 bits on the rows that it was given,
    the gather and the quantisation bit for bit, and only the rows in use quantised."""
    dev = require_gpu()
    T, E, k, H, inner, bs = 70, 12, 3, 256, 160, 16
    gen = torch.Generator().manual_seed(9)
    emap = torch.full((E,), -1, dtype=torch.int32)
    emap[3:9] = torch.arange(6, dtype=torch.int32)
    r = tdt.MoeRouter(T, E, k, H, bs, True, E_local=6, expert_map=emap, device=dev)
    experts = tdt.Mx4Experts((torch.randn((6, 2 * inner, H), generator=gen) * 0.1).to(torch.bfloat16).to(dev),
                             (torch.randn((6, H, inner), generator=gen) * 0.1).to(torch.bfloat16).to(dev), r.capacity)
    x = torch.randn((T, E), generator=gen).to(torch.bfloat16).to(dev)
    h = torch.randn((T, H), generator=gen).to(torch.bfloat16).to(dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.step_mx4(x, h, experts)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.step_mx4(x, h, experts)
    for seed in range(2):
        x.copy_(torch.randn((T, E), generator=gen).to(torch.bfloat16))
        h.copy_(torch.randn((T, H), generator=gen).to(torch.bfloat16))
        experts.act_rows.codes.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        replayed = r.out.clone()
        counts, off = r.align.counts.cpu(), r.align.offsets.cpu()
        n = int(off[-1])
        want = tdt.moe_quantize_mx4(h)
        local = r.align.inv_perm >= 0
        rows, token = r.align.inv_perm[local].long(), torch.arange(T * k, device=dev)[local] // k
        assert torch.equal(experts.rows.codes[rows], want.codes[token])
        assert (experts.act_rows.codes[n:] == 0x5A).all()
        up = reference(values(experts.rows), values(experts.w_up), counts, off, 2 * inner, True)
        down = reference(values(experts.act_rows), values(experts.w_down), counts, off, H, False)
        for (ra, ya, ta), (rb, yb, tb) in zip(up, down):
            assert ((experts.act[ra].double() - ya).abs() <= ta).all()
            assert ((experts.out[rb].double() - yb).abs() <= tb).all()
            assert torch.equal(experts.act_rows.codes[ra], tdt.moe_quantize_mx4(experts.act[ra].contiguous()).codes)
        r.step_mx4(x, h, experts)
        assert torch.equal(r.out, replayed)
        assert torch.equal(r.out, tdt.moe_combine(experts.out, r.topk_weights, r.align.inv_perm))
    assert r.device_status() == tdt.MOE_OK
