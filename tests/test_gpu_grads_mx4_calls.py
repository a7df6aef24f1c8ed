"""How the gradients and the 4-bit entry points are called, on the GPU: outputs inside guard bands, element offsets past
32 bits, streams, two calls at once, and tensors that the wrappers turn down."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


def layer(T=130, E=12, k=3, H=288, bs=8, El=None, seed=0):
    """Inputs of every call for one small batch."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(seed)
    El = El or E
    emap = torch.full((E,), -1, dtype=I32)
    emap[E - El:] = torch.arange(El, dtype=I32)
    x = torch.randn((T, E), generator=g).to(dev)
    w, ids = tdt.moe_topk_softmax(x, k, True)
    al = tdt.moe_align_permute(ids, E, bs, emap.to(dev), El)
    rows = lambda n, c: torch.randn((n, c), generator=g).to(BF16).to(dev)  # noqa: E731
    return dict(x=x, w=w, ids=ids, al=al, k=k, h=rows(T, H), y=rows(al.capacity, H), gout=rows(T, H),
                gw=torch.randn((T, k), generator=g).to(dev), w_up=tdt.moe_quantize_mx4(rows(El * 64, H)))


def every_call(d, out, stream=None):
    """All entry points into `out`'s buffers (made where missing)."""
    al, k, C = d["al"], d["k"], d["al"].capacity
    get = out.setdefault
    T, H = d["h"].shape
    e = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    tdt.moe_combine_backward(d["gout"], d["y"], d["w"], al.inv_perm, get("gy", e(C, H)),
                             get("gwt", e(T, k, t=torch.float32)), al.sorted_token_ids, al.num_tokens_post_pad, True,
                             stream=stream)
    tdt.moe_gather_backward(d["y"], al.inv_perm, k, get("gx", e(T, H)), stream=stream)
    tdt.moe_topk_softmax_backward(d["gw"], d["x"], d["w"], d["ids"], True,
                                  get("gl", e(*d["x"].shape, t=torch.float32)), stream=stream)
    q = tdt.Mx4Tensor(get("codes", e(C, H // 2, t=torch.uint8)), get("scales", e(-(-H // 128), C, 4, t=torch.uint8)))
    tdt.moe_gather_mx4(d["h"], k, al.inv_perm, C, q, stream=stream)
    tdt.moe_grouped_gemm_mx4(q, d["w_up"], al.counts, al.offsets, get("up", e(C, 32)), True, stream=stream)
    p = tdt.Mx4Tensor(get("codes2", e(T, H // 2, t=torch.uint8)), get("scales2", e(-(-H // 128), T, 4, t=torch.uint8)))
    tdt.moe_quantize_mx4(d["h"], p, stream=stream)
    tdt.moe_dequantize_mx4(p, get("back", e(T, H)), stream=stream)
    return out


def test_no_write_outside_the_outputs():
    d = layer(El=8)
    want = every_call(d, {})
    big, views = {}, {}
    for name, t in want.items():  # each output inside a buffer of its own, 512 bytes of 0xA5 before and after
        n = t.numel() * t.element_size()
        big[name] = torch.full((n + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
        views[name] = big[name][512:512 + n].view(t.dtype).view(t.shape)
        views[name].zero_()
    got = every_call(d, dict(views))
    torch.cuda.synchronize()
    for name, t in want.items():
        assert torch.equal(got[name], t), name
        assert (big[name][:512] == 0xA5).all() and (big[name][-512:] == 0xA5).all(), name


def test_streams_and_two_calls_at_once():
    """The same results on side streams, given as objects and as handles, while another batch runs beside."""
    a, b = layer(seed=1), layer(T=500, seed=2)
    want_a, want_b = every_call(a, {}), every_call(b, {})
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [({}, {}) for _ in range(4)]
    for oa, ob in outs:
        for name in want_a:
            oa[name], ob[name] = torch.zeros_like(want_a[name]), torch.zeros_like(want_b[name])
    torch.cuda.synchronize()
    for oa, ob in outs:
        every_call(a, oa, stream=s)
        every_call(b, ob, stream=t.cuda_stream)
    torch.cuda.synchronize()
    for oa, ob in outs:
        for name in want_a:
            assert torch.equal(oa[name], want_a[name]) and torch.equal(ob[name], want_b[name]), name


def test_two_graphs_side_by_side():
    a, b = layer(seed=3), layer(T=300, seed=4)
    out_a, out_b = every_call(a, {}), every_call(b, {})
    want = [{n: t.clone() for n, t in o.items()} for o in (out_a, out_b)]
    graphs = []
    for d, o in ((a, out_a), (b, out_b)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            every_call(d, o)
        graphs.append(g)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for o in (out_a, out_b):
        for x in o.values():
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, (s, t)):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip((out_a, out_b), want):
        for n in w:
            assert torch.equal(o[n], w[n]), n


def test_element_offsets_past_32_bits():
    """A few slots whose rows lie behind 2^31 elements."""
    dev = require_gpu()
    T, k, H = 4, 2, 8192
    C = (1 << 31) // H + 40
    inv = torch.tensor([C - 1, 3, C - 30, -1, C - 7, C - 8, 0, C - 9], dtype=I32, device=dev)
    local = inv >= 0
    rows, token = inv[local].long(), torch.arange(T * k, device=dev)[local] // k
    g = torch.Generator().manual_seed(0)
    gout, w = torch.randn((T, H), generator=g).to(BF16).to(dev), torch.rand((T, k), generator=g).to(dev)
    y = torch.empty((C, H), dtype=BF16, device=dev)
    y[rows] = torch.randn((rows.numel(), H), generator=g).to(BF16).to(dev)
    small = torch.arange(T * k, dtype=I32, device=dev)  # the same rows, close together
    small[~local] = -1
    ys = torch.zeros((T * k, H), dtype=BF16, device=dev)
    ys[local] = y[rows]
    assert torch.equal(tdt.moe_gather_backward(y, inv, k), tdt.moe_gather_backward(ys, small, k))
    want_y, want_w = tdt.moe_combine_backward(gout, ys, w, small, torch.zeros_like(ys))
    got_y, got_w = tdt.moe_combine_backward(gout, y, w, inv, y)
    assert torch.equal(got_w, want_w) and torch.equal(got_y[rows], want_y[local])
    del y, got_y
    torch.cuda.empty_cache()
    # codes past 2^31 bytes, the product's rows of out past 2^31 elements
    K, N = 8192, 4096
    C = (1 << 32) // K + 300
    inv = torch.tensor([C - 1, 3, C - 30, -1, C - 7, C - 8, 0, C - 9], dtype=I32, device=dev)
    rows = inv[local].long()
    q = tdt.moe_gather_mx4(gout, k, inv, C)
    s = tdt.moe_quantize_mx4(gout)
    assert torch.equal(q.codes[rows], s.codes[token]) and torch.equal(q.scales[:, rows], s.scales[:, token])
    wq = tdt.moe_quantize_mx4(torch.randn((2 * N, K), generator=g).to(BF16).to(dev))
    n = 150
    x = torch.randn((n, K), generator=g).to(BF16).to(dev)
    xs = tdt.moe_quantize_mx4(x)
    q.codes[C - n:], q.scales[:, C - n:] = xs.codes, xs.scales
    counts = torch.tensor([0, n], dtype=I32, device=dev)
    out = torch.empty((C, N), dtype=BF16, device=dev)
    tdt.moe_grouped_gemm_mx4(q, wq, counts, torch.tensor([0, C - n, C], dtype=I32, device=dev), out=out)
    near = tdt.moe_grouped_gemm_mx4(xs, wq, counts, torch.tensor([0, 0, n], dtype=I32, device=dev))
    assert torch.equal(out[C - n:], near)


def test_what_the_wrappers_turn_down():
    d = layer()
    al, k, C = d["al"], d["k"], d["al"].capacity
    T, H = d["h"].shape
    q = tdt.moe_gather_mx4(d["h"], k, al.inv_perm, C)
    strided = torch.zeros((T, 2 * H), dtype=BF16, device="cuda")[:, :H]
    with pytest.raises(ValueError, match="contiguous"):
        tdt.moe_combine_backward(strided, d["y"], d["w"], al.inv_perm)
    with pytest.raises(ValueError, match="contiguous"):
        tdt.moe_quantize_mx4(strided)
    with pytest.raises(ValueError, match="bfloat16"):
        tdt.moe_gather_mx4(d["h"].float(), k, al.inv_perm, C)
    with pytest.raises(ValueError, match="int32"):
        tdt.moe_gather_backward(d["y"], al.inv_perm.long(), k)
    with pytest.raises(ValueError, match="shape"):
        tdt.moe_topk_softmax_backward(d["gw"][:, :2].contiguous(), d["x"], d["w"], d["ids"], True)
    with pytest.raises(ValueError, match="shape"):
        tdt.moe_grouped_gemm_mx4(q, d["w_up"], al.counts, al.offsets[:-1])
    with pytest.raises(ValueError, match="missing"):
        tdt.moe_combine_backward(d["gout"], d["y"], d["w"], al.inv_perm, zero_pad=True)
    with pytest.raises(ValueError, match="CUDA"):
        tdt.moe_gather_backward(d["y"], al.inv_perm.cpu(), k)
    with pytest.raises(tdt.MoeError):  # 4 bytes off
        tdt.moe_quantize_mx4(torch.zeros(4 * H + 2, dtype=BF16, device="cuda")[2:].view(4, H))
    with pytest.raises(tdt.MoeError):
        tdt.moe_gather_backward(torch.zeros((C, 12), dtype=BF16, device="cuda"), al.inv_perm, k)
    r = tdt.MoeRouter(T, 12, k, H, 8, True)
    with pytest.raises(RuntimeError, match="training"):
        r.combine_backward(d["gout"], d["y"])
    with pytest.raises(ValueError, match="rows"):
        tdt.Mx4Experts(torch.zeros((12, 64, H), dtype=BF16, device="cuda"),
                       torch.zeros((12, H, 32), dtype=BF16, device="cuda"), C + 1).forward(d["h"], k, al)


def test_no_tokens():
    dev = require_gpu()
    inv = torch.empty(0, dtype=I32, device=dev)
    rows, none = torch.ones((5, 64), dtype=BF16, device=dev), torch.empty((0, 64), dtype=BF16, device=dev)
    w, ids, x = torch.empty((0, 2), device=dev), torch.empty((0, 2), dtype=I32, device=dev), torch.empty((0, 8), device=dev)
    gy, gw = tdt.moe_combine_backward(none, rows, w, inv, rows.clone())
    assert (gy == 1).all() and gw.shape == (0, 2)
    assert tdt.moe_gather_backward(rows, inv, 2).shape == (0, 64)
    assert tdt.moe_topk_softmax_backward(w, x, w, ids, True).shape == (0, 8)
    q = tdt.moe_gather_mx4(none, 2, inv, 5)
    wq = tdt.moe_quantize_mx4(torch.ones((8, 64), dtype=BF16, device=dev))
    out = torch.full((5, 8), 7.0, dtype=BF16, device=dev)
    tdt.moe_grouped_gemm_mx4(q, wq, torch.zeros(1, dtype=I32, device=dev), torch.zeros(2, dtype=I32, device=dev), out)
    assert (out == 7).all()


@pytest.mark.parametrize("as_handle", [False, True])
def test_new_outputs_do_not_take_memory_in_use_on_another_stream(as_handle):
    """A tensor freed while the current stream still has to read it is not handed to a call on a side stream."""
    require_gpu()
    rows, K = 4096, 2048
    q = tdt.moe_quantize_mx4(torch.full((rows, K), 3.0, dtype=BF16, device="cuda"))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.full((rows, K), 5.0, dtype=BF16, device="cuda")
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    y.copy_(x)
    del x
    back = tdt.moe_dequantize_mx4(q, stream=side.cuda_stream if as_handle else side)
    torch.cuda.synchronize()
    assert (y == 5).all() and (back == 3).all()
