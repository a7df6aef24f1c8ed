"""Gradients of the combine, the gather and the gating on the GPU, against the formulas in 64 bits and against
differences.  Tolerances count roundings: u = 2^-24 an fp32 operation, 2^-8 (bf16) or 2^-24 (fp32) the last one."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 2.0 ** -126  # results below the normal range


def routes(T, E, k, bs, El=None, seed=0, ids=None):
    """ids [T, k], an align result of them and a status word, on the GPU."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(seed)
    if ids is None:
        ids = torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32)
    emap = None
    if El is not None and El < E:
        emap = torch.full((E,), -1, dtype=torch.int32)
        emap[E - El:] = torch.arange(El, dtype=torch.int32)
        emap = emap.to(dev)
    al = tdt.moe_align_permute(ids.to(dev), E, bs, emap, El or E)
    return ids.to(dev), al, torch.zeros(1, dtype=torch.int32, device=dev)


def normal(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def within(got, want, tol, what):
    bad = (got.double() - want).abs() - tol
    assert not torch.isnan(got).any(), what
    assert bad.max().item() <= 0 if bad.numel() else True, f"{what}: beyond the tolerance by {bad.max().item():.3g}"


SIZES = [
    # T, E, k, H, bs, E_local
    (1, 1, 1, 8, 1, None),
    (1, 8, 2, 264, 16, None),
    (3, 160, 6, 4096, 8, 40),
    (64, 8, 2, 256, 16, None),
    (37, 60, 4, 7168, 64, None),
    (333, 128, 8, 520, 16, 32),
    (1000, 16, 3, 64, 7, None),
    (29, 33, 32, 1032, 24, None),
    (700, 64, 8, 2048, 64, None),
]


@pytest.mark.parametrize("T,E,k,H,bs,El", SIZES)
def test_combine_backward(T, E, k, H, bs, El):
    _, al, status = routes(T, E, k, bs, El, seed=T)
    gout, y = normal(1, T, H, dtype=torch.bfloat16), normal(2, al.capacity, H, dtype=torch.bfloat16)
    w = normal(3, T, k)
    gy = torch.full((al.capacity, H), 7.0, dtype=torch.bfloat16, device="cuda")
    gy, gw = tdt.moe_combine_backward(gout, y, w, al.inv_perm, grad_expert_out=gy, device_status=status,
                                      sorted_token_ids=al.sorted_token_ids,
                                      num_tokens_post_pad=al.num_tokens_post_pad, zero_pad=True)
    inv = al.inv_perm.long()
    local = inv >= 0
    g64 = gout.double().repeat_interleave(k, 0)
    want_y = torch.full((al.capacity, H), 7.0, dtype=torch.float64, device="cuda")
    want_y[:int(al.num_tokens_post_pad)] = 0.0
    want_y[inv[local]] = (w.double().view(-1, 1) * g64)[local]
    # w g in fp32, then to bf16
    within(gy, want_y, want_y.abs() * (2.0 ** -8 * (1 + 2.0 ** -8) + U) + 2.0 ** -133, "grad_expert_out")
    rows = y.double()[inv.clamp(min=0)]
    prod = torch.where(local[:, None], g64 * rows, 0.0)
    # products are exact in fp32; a lane adds ceil(H / 256) per sum, then 3 + 5 levels join them
    n = -(-H // 256) + 8
    within(gw.view(-1), prod.sum(1), n * U * 1.001 * prod.abs().sum(1), "grad_topk_weights")
    assert (gw.view(-1)[~local] == 0).all()
    assert tdt.moe_read_status(status) == tdt.MOE_OK


def test_combine_backward_leaves_pads_and_takes_one_output():
    T, E, k, H, bs = 50, 6, 2, 128, 16
    _, al, status = routes(T, E, k, bs)
    gout, y, w = normal(1, T, H, dtype=torch.bfloat16), normal(2, al.capacity, H, dtype=torch.bfloat16), normal(3, T, k)
    gy = torch.full_like(y, 7.0)
    _, gw = tdt.moe_combine_backward(gout, y, w, al.inv_perm, grad_expert_out=gy)
    pad = torch.ones(al.capacity, dtype=torch.bool, device="cuda")
    pad[al.inv_perm.long()] = False
    assert (gy[pad] == 7.0).all() and (gy[~pad] != 7.0).any()
    # the C entry point takes either output alone
    from token_dispatch_topk_b200 import binding as B
    lib, p = B.load_library(), lambda t: t.data_ptr()
    one_y, one_w = torch.full_like(y, 7.0), torch.zeros_like(gw)
    s = torch.cuda.current_stream().cuda_stream
    assert lib.moe_combine_backward(p(gout), None, p(w), p(al.inv_perm), None, None, T, k, H, al.capacity, 0, p(one_y),
                                    None, None, s) == 0
    assert lib.moe_combine_backward(p(gout), p(y), p(w), p(al.inv_perm), None, None, T, k, H, al.capacity, 0, None,
                                    p(one_w), None, s) == 0
    assert torch.equal(one_y, gy) and torch.equal(one_w, gw)
    # in place: the gradient rows over the expert outputs
    z = y.clone()
    _, gw2 = tdt.moe_combine_backward(gout, z, w, al.inv_perm, grad_expert_out=z)
    assert torch.equal(gw2, gw) and torch.equal(z[~pad], gy[~pad]) and torch.equal(z[pad], y[pad])


@pytest.mark.parametrize("T,E,k,H,bs,El", SIZES)
def test_gather_backward(T, E, k, H, bs, El):
    _, al, status = routes(T, E, k, bs, El, seed=T + 1)
    gp = normal(4, al.capacity, H, dtype=torch.bfloat16)
    pad = torch.ones(al.capacity, dtype=torch.bool, device="cuda")
    pad[al.inv_perm[al.inv_perm >= 0].long()] = False
    gp[pad] = float("nan")  # pad rows are not read
    gx = tdt.moe_gather_backward(gp, al.inv_perm, k, device_status=status)
    inv = al.inv_perm.long().view(T, k)
    rows = torch.where((inv >= 0)[..., None], gp.double()[inv.clamp(min=0)], 0.0)
    want = rows.sum(1)
    within(gx, want, want.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + 1.01 * k * U * rows.abs().sum(1) + 2.0 ** -133, "grad")
    assert (gx[(inv < 0).all(1)] == 0).all()
    assert tdt.moe_read_status(status) == tdt.MOE_OK


def test_all_remote_rank():
    T, k, H = 9, 3, 64
    dev = require_gpu()
    emap = torch.full((8,), -1, dtype=torch.int32, device=dev)
    ids = torch.arange(T * k, dtype=torch.int32, device=dev).view(T, k) % 8
    al = tdt.moe_align_permute(ids, 8, 16, emap, 2)
    y = torch.full((al.capacity, H), 3.0, dtype=torch.bfloat16, device=dev)
    gy = y.clone()
    gy, gw = tdt.moe_combine_backward(normal(1, T, H, dtype=torch.bfloat16), y, normal(2, T, k), al.inv_perm, gy,
                                      sorted_token_ids=al.sorted_token_ids,
                                      num_tokens_post_pad=al.num_tokens_post_pad, zero_pad=True)
    assert (gw == 0).all() and torch.equal(gy, y)
    assert (tdt.moe_gather_backward(y, al.inv_perm, k) == 0).all()


@pytest.mark.parametrize("bad", [-2, 10 ** 6])
def test_rows_out_of_range_are_skipped_and_recorded(bad):
    T, E, k, H, bs = 40, 4, 2, 64, 8
    _, al, status = routes(T, E, k, bs)
    gout, y, w = normal(1, T, H, dtype=torch.bfloat16), normal(2, al.capacity, H, dtype=torch.bfloat16), normal(3, T, k)
    want_y, want_w = tdt.moe_combine_backward(gout, y, w, al.inv_perm, torch.zeros_like(y))
    want_x = tdt.moe_gather_backward(y, al.inv_perm, k)
    inv = al.inv_perm.clone()
    lost = inv[7].item()
    inv[7] = bad
    gy, gw = tdt.moe_combine_backward(gout, y, w, inv, torch.zeros_like(y), device_status=status)
    assert tdt.moe_read_status(status) == tdt.MOE_ERR_BAD_ROW
    want_y[lost], want_w[3, 1] = 0, 0
    assert torch.equal(gy, want_y) and torch.equal(gw, want_w)
    gx = tdt.moe_gather_backward(y, inv, k, device_status=status)
    assert tdt.moe_read_status(status) == tdt.MOE_ERR_BAD_ROW
    assert torch.equal(gx[:3], want_x[:3]) and torch.equal(gx[4:], want_x[4:])


# ------------------------------------------------------------------------------------------------- gating --
def gate_reference(g, x, w, ids, renorm, scoring):
    g, x, w, ids = g.double(), x.double(), w.double(), ids.long()
    G = (g * w).sum(-1, keepdim=True)
    if scoring == "softmax" and not renorm:
        return torch.softmax(x, -1) * (torch.zeros_like(x).scatter_add_(1, ids, g) - G)
    d = w * (g - G) if renorm else w * g
    if scoring == "sigmoid":
        d = d * torch.sigmoid(-x.gather(1, ids))
    return torch.zeros_like(x).scatter_add_(1, ids, d)


def gate_tolerance(g, x, w, ids, renorm, scoring):
    """Error of the fp32 arithmetic; the output's own rounding is added by the caller."""
    g, x, w, ids = g.double().abs(), x.double(), w.double().abs(), ids.long()
    sum_gw = (g * w).sum(-1, keepdim=True)
    err_G = 7 * U * sum_gw  # products, five levels of the warp's sum, one addition
    if scoring == "softmax" and not renorm:
        span = (x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True))
        E = x.shape[1]
        # exp of a rounded difference, twice (2 ulp = 4 u each), the sum of E terms, a reciprocal and two products
        rel = (2 * span + E / 32 + 5 + 8 + 4) * U
        gf = torch.zeros_like(x).scatter_add_(1, ids, g)
        return torch.softmax(x, -1) * ((gf + sum_gw) * (rel + 2 * U) + err_G)
    e = w * (err_G + 3 * U * (g + sum_gw)) if renorm else 2 * U * w * g
    if scoring == "sigmoid":  # exp (4 u), sum, quotient
        e = e + 6 * U * w * (g + (sum_gw if renorm else 0.0))
    return torch.zeros_like(x).scatter_add_(1, ids, e)


GATES = [(1, 1, 1), (1, 8, 2), (5, 7, 7), (64, 8, 2), (33, 60, 4), (100, 128, 8), (17, 160, 6), (257, 256, 8),
         (40, 1000, 32), (9, 1024, 3), (300, 34, 5), (1025, 64, 1)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", GATES)
def test_gating_backward(T, E, k, dtype, scoring, renorm):
    require_gpu()
    x = (normal(T + E, T, E) * 2).to(dtype)
    w, ids = tdt.moe_topk_softmax(x, k, renorm, scoring=scoring)
    g = normal(5, T, k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gx = tdt.moe_topk_softmax_backward(g, x, w, ids, renorm, scoring=scoring, device_status=status)
    assert gx.dtype == dtype
    want = gate_reference(g, x, w, ids, renorm, scoring)
    tol = gate_tolerance(g, x, w, ids, renorm, scoring)
    within(gx, want, tol * (1 + 2.0 ** -7) + want.abs() * HALF[dtype] + TINY, "grad_logits")
    assert tdt.moe_read_status(status) == tdt.MOE_OK
    inplace = x.clone()
    tdt.moe_topk_softmax_backward(g, inplace, w, ids, renorm, grad_logits=inplace, scoring=scoring)
    assert torch.equal(inplace, gx)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(151001, 8, 2), (20003, 60, 4), (40001, 256, 8), (30011, 34, 1), (10007, 130, 32)])
def test_gating_backward_large_batches(T, E, k, dtype):
    """The softmax over all experts where a warp takes several groups of rows, and a ragged last warp."""
    require_gpu()
    x = torch.randn((T, E), generator=torch.Generator("cuda").manual_seed(E), device="cuda").to(dtype)
    w, ids = tdt.moe_topk_softmax(x, k, False)
    g = torch.randn((T, k), generator=torch.Generator("cuda").manual_seed(k), device="cuda")
    gx = tdt.moe_topk_softmax_backward(g, x, w, ids, False)
    want = gate_reference(g, x, w, ids, False, "softmax")
    tol = gate_tolerance(g, x, w, ids, False, "softmax")
    within(gx, want, tol * (1 + 2.0 ** -7) + want.abs() * HALF[dtype] + TINY, "grad_logits")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gating_backward_against_differences(scoring, renorm):
    """The slope of sum_j g_j w_j along a random direction, the weights of the fixed selection in 64 bits."""
    require_gpu()
    T, E, k = 20, 24, 4
    x, g, d = normal(1, T, E), normal(2, T, k), normal(3, T, E).double()
    w, ids = tdt.moe_topk_softmax(x, k, renorm, scoring=scoring)
    gx = tdt.moe_topk_softmax_backward(g, x, w, ids, renorm, scoring=scoring)

    def loss(z):
        p = torch.sigmoid(z) if scoring == "sigmoid" else torch.softmax(z, -1)
        s = p.gather(1, ids.long())
        s = s / s.sum(-1, keepdim=True) if renorm else s
        return (g.double() * s).sum(-1)
    h = 2.0 ** -13
    slope = (loss(x.double() + h * d) - loss(x.double() - h * d)) / (2 * h)
    got = (gx.double() * d).sum(-1)
    # third derivative of a softmax or logistic weight along d: at most about (2 |d|)^3; the gradient itself: 2^-16
    scale = g.double().abs().sum(-1) * (1 + d.abs().amax(-1)) ** 3
    assert ((slope - got).abs() <= scale * (8 * h * h / 6 + 2.0 ** -16)).all()


def test_gating_backward_duplicate_and_bad_ids():
    require_gpu()
    T, E, k = 4, 40, 5
    x, g, w = normal(1, T, E), normal(2, T, k), normal(3, T, k).abs()
    ids = torch.tensor([[3, 3, 3, 9, 9], [0, 1, 2, 3, 4], [39, 39, 0, 39, 0], [7, 7, 7, 7, 7]], dtype=torch.int32).cuda()
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            gx = tdt.moe_topk_softmax_backward(g, x, w, ids, renorm, scoring=scoring)
            want = gate_reference(g, x, w, ids, renorm, scoring)
            # up to four more additions
            tol = gate_tolerance(g, x, w, ids, renorm, scoring)
            mag = torch.zeros_like(want).scatter_add_(1, ids.long(), w.double() * (g.double().abs() + (g * w).double().abs().sum(-1, keepdim=True)) + g.double().abs())
            within(gx, want, tol * 1.01 + 5 * U * mag + want.abs() * U + TINY, (scoring, renorm))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = ids.clone()
    bad[1, 2], bad[1, 4] = -1, E
    gx = tdt.moe_topk_softmax_backward(g, x, w, bad, True, device_status=status)
    assert tdt.moe_read_status(status) == tdt.MOE_ERR_BAD_EXPERT_ID
    g2, w2 = g.clone(), w.clone()
    g2[1, 2] = g2[1, 4] = w2[1, 2] = w2[1, 4] = 0
    assert torch.equal(gx, tdt.moe_topk_softmax_backward(g2, x, w2, ids, True))


def test_gating_backward_far_logits():
    """Scores at the ends of the range: nothing becomes NaN, and underflowed scores give no gradient."""
    require_gpu()
    x = torch.tensor([[-200.0, -150.0, -300.0, -120.0], [200.0, 150.0, 90.0, -90.0], [0.0, -float("inf"), 1.0, 88.0]]).cuda()
    g = torch.tensor([[1.0, -2.0]] * 3).cuda()
    for renorm in (True, False):
        w, ids = tdt.moe_topk_softmax(x[:2], 2, renorm, scoring="sigmoid")
        gx = tdt.moe_topk_softmax_backward(g[:2], x[:2], w, ids, renorm, scoring="sigmoid")
        assert torch.isfinite(gx).all() and (gx[0] == 0).all()
        want = gate_reference(g[:2], x[:2], w, ids, renorm, "sigmoid")
        assert ((gx.double() - want)[1].abs() <= 1e-37).all()
    w = torch.tensor([[1.0, 0.0]]).cuda()
    ids = torch.tensor([[3, 2]], dtype=torch.int32).cuda()
    gx = tdt.moe_topk_softmax_backward(g[2:], x[2:], w, ids, False)
    assert torch.isfinite(gx).all() and gx[0, 1] == 0


# ------------------------------------------------------------------------------------------ used together --
def test_layer_gradient_against_differences():
    """Gate, dispatch, per-row experts (each row scaled by its expert's factor), combine, and the whole way back
    through the router object: the loss's slope along random directions of the hidden rows and logits."""
    T, E, k, H, bs = 48, 8, 2, 64, 16
    dev = require_gpu()
    x, h = normal(1, T, E), normal(2, T, H, dtype=torch.bfloat16)
    gout = normal(3, T, H, dtype=torch.bfloat16)
    factor = normal(4, E)
    r = tdt.MoeRouter(T, E, k, H, bs, True, logits_dtype=torch.float32, device=dev, training=True)
    r.dispatch(x, h)
    expert_of_row = r.align.expert_ids.long().repeat_interleave(bs)[:r.capacity].clamp(min=0)
    y = (r.permuted.float() * factor[expert_of_row, None]).to(torch.bfloat16)
    r.combine(y)
    gy, gw = r.combine_backward(gout, y)
    gp = (gy.float() * factor[expert_of_row, None]).to(torch.bfloat16)
    gh, gx = r.gather_backward(gp), r.gate_backward(x)
    assert r.device_status() == tdt.MOE_OK

    def loss(x64, h64):
        ids = r.topk_ids.long()
        w = torch.softmax(x64.gather(1, ids), -1)
        out = (w * factor.double()[ids]).sum(-1, keepdim=True) * h64
        return (out * gout.double()).sum(1)
    dx, dh = normal(5, T, E).double(), normal(6, T, H).double()
    e = 2.0 ** -12
    slope_x = (loss(x.double() + e * dx, h.double()) - loss(x.double() - e * dx, h.double())) / (2 * e)
    slope_h = (loss(x.double(), h.double() + e * dh) - loss(x.double(), h.double() - e * dh)) / (2 * e)
    ids = r.topk_ids.long()
    # every bf16 rounding on the way (y; gy, gp, gh) is 2^-8 of a term; differences of the loss: h^2 times its third derivative
    mag = (gout.double() * h.double()).abs().sum(1) * factor.double().abs()[ids].amax(1)
    tol_x = mag * dx.abs().amax(1) * (2 * 2.0 ** -8 * 1.1 + 8 * e * e * (1 + dx.abs().amax(1)) ** 2)
    assert ((gx.double() * dx).sum(1) - slope_x).abs().le(tol_x).all()
    tol_h = (gout.double() * dh).abs().sum(1) * factor.double().abs()[ids].amax(1) * 3 * 2.0 ** -8 * 1.1
    assert ((gh.double() * dh).sum(1) - slope_h).abs().le(tol_h).all()


def test_captured_and_replayed_on_another_stream():
    """The backward calls in a graph, replayed on new inputs, give what they give eagerly."""
    T, E, k, H, bs = 200, 32, 4, 256, 16
    dev = require_gpu()
    r = tdt.MoeRouter(T, E, k, H, bs, True, device=dev, training=True)
    x, h = normal(1, T, E, dtype=torch.bfloat16), normal(2, T, H, dtype=torch.bfloat16)
    y = normal(3, r.capacity, H, dtype=torch.bfloat16)
    gout = normal(4, T, H, dtype=torch.bfloat16)

    def step():
        r.dispatch(x, h)
        r.combine(y)
        gy, gw = r.combine_backward(gout, y)
        return r.out, gy, gw, r.gather_backward(gy), r.gate_backward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (10, 20):
        for t, s in ((x, 0), (h, 1), (y, 2), (gout, 3)):
            t.copy_(normal(seed + s, *t.shape, dtype=t.dtype))
        graph.replay()
        got = [o.clone() for o in outs]
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            want = [o.clone() for o in step()]
        side.synchronize()
        n = int(r.align.num_tokens_post_pad)
        for a, b in zip(got, want):
            m = n if a.shape[0] == r.capacity else a.shape[0]
            assert torch.equal(a[:m], b[:m])
    torch.cuda.synchronize()
    assert r.device_status() == tdt.MOE_OK


def test_repeated_calls_give_the_same_bits():
    T, E, k, H, bs = 900, 60, 4, 1024, 64
    _, al, _ = routes(T, E, k, bs)
    gout, y, w = normal(1, T, H, dtype=torch.bfloat16), normal(2, al.capacity, H, dtype=torch.bfloat16), normal(3, T, k)
    a = tdt.moe_combine_backward(gout, y, w, al.inv_perm, torch.zeros_like(y))
    for _ in range(3):
        b = tdt.moe_combine_backward(gout, y, w, al.inv_perm, torch.zeros_like(y))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
