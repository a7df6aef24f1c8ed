"""The routing layer's gradients and its 4-bit expert products, as cases to measure.

Every case runs one operator once.  With ``own`` false ``run`` computes it from elementary torch operations, in
32 bits; with ``own`` true it calls the framework's entry points.  Five operators:

  combine_backward   gradient of the weighted combine: rows of the expert outputs and the combine weights
  gather_backward    gradient of the permute-gather: rows summed back to their tokens
  gating_backward    gradient of the top-k gating: combine weights to router logits
  mx4_cast           rows to microscaled 4-bit floating point (blocks of 32, one power-of-two scale each) and back
  mx4_product        the experts' product in that format, the rows quantised on the way in: "up" takes tokens
                     through the permute-gather and ends in silu(gate) * up, "down" takes expert-grouped rows
"""
import math

import torch

own = False

# Values of the sixteen 4-bit codes: sign, two exponent bits, one mantissa bit.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    route = dict(E_local=0, zipf=0.0)
    return [
        # the smallest training batch of the parity workloads: latency counts
        dict(route, name="combine_backward_T64_E8_k2", op="combine_backward", T=64, E=8, k=2, H=256, bs=16),
        # a large skewed training batch (Zipf expert popularity), long rows
        dict(route, name="combine_backward_T16384_E256_k8", op="combine_backward", T=16384, E=256, k=8, H=7168, bs=128,
             zipf=1.1),
        # an ordinary batch: every token has eight rows to sum
        dict(route, name="gather_backward_T4096_E128_k8", op="gather_backward", T=4096, E=128, k=8, H=2048, bs=64),
        # one of four expert-parallel ranks: most slots are remote, many tokens keep no row
        dict(route, name="gather_backward_T16384_local40_k6", op="gather_backward", T=16384, E=160, k=6, H=4096, bs=8,
             E_local=40),
        # gating of an ordinary batch, renormalised softmax: only the selected logits get a gradient
        dict(name="gating_backward_T4096_E128_k8", op="gating_backward", T=4096, E=128, k=8, dtype="bf16",
             scoring="softmax", renorm=True),
        # a number of experts that is no power of two, fp32 logits, softmax over all of them: a dense gradient
        dict(name="gating_backward_T16384_E60_k4", op="gating_backward", T=16384, E=60, k=4, dtype="f32",
             scoring="softmax", renorm=False),
        # the largest gating, logistic scores
        dict(name="gating_backward_T65536_E256_k8", op="gating_backward", T=65536, E=256, k=8, dtype="bf16",
             scoring="sigmoid", renorm=True),
        # odd rows whose last chunk of blocks is ragged
        dict(name="mx4_cast_333x288", op="mx4_cast", rows=333, K=288),
        # the weights of a whole layer: 128 experts, 1536 x 2048 each
        dict(name="mx4_cast_196608x2048", op="mx4_cast", rows=128 * 1536, K=2048),
        # decode on one of four expert-parallel ranks: two tokens, weights stream from memory
        dict(route, name="mx4_up_T2_local40_k6", op="mx4_product", form="up", T=2, E=160, k=6, K=4096, N=2816, bs=8,
             E_local=40),
        # the second product of an ordinary prefill: short rows in, long rows out
        dict(route, name="mx4_down_T4096_E128_k8", op="mx4_product", form="down", T=4096, E=128, k=8, K=768, N=2048,
             bs=64),
        # a large expert-parallel prefill, 32 of 256 experts: enough rows per expert to be bound by arithmetic
        dict(route, name="mx4_up_T32768_local32_k8", op="mx4_product", form="up", T=32768, E=256, k=8, K=7168, N=4096,
             bs=128, E_local=32),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["combine_backward", "gather_backward", "gating_backward", "mx4_cast", "mx4_product"])
    if op == "mx4_cast":
        K = _log_int(rng, 32, 8192, 32)
        return dict(op=op, rows=_log_int(rng, 1, 128 * 1536 * 2048 // K), K=K)
    E = _log_int(rng, 8, 256)
    k = rng.randint(1, min(8, E))
    if op == "gating_backward":
        return dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=k, dtype=rng.choice(["bf16", "f32"]),
                    scoring=rng.choice(["softmax", "sigmoid"]), renorm=rng.choice([True, False]))
    c = dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k, bs=rng.choice([1, 8, 16, 24, 64, 128]),
             E_local=rng.choice([0, 0, max(1, E // 4)]), zipf=rng.choice([0.0, 1.1]))
    if op == "mx4_product":
        form = rng.choice(["up", "down"])
        K, N = _log_int(rng, 64, 7168, 32), _log_int(rng, 64, 4096, 16)
        # at most 400 million weights and 16384 rows
        E = c["E"] = max(k, min(E, 400_000_000 // (K * N)))
        c.update(form=form, K=K, N=N, T=max(1, min(c["T"], 16384 // k)), E_local=rng.choice([0, max(1, E // 4)]))
        return c
    c["H"] = _log_int(rng, 64, 7168, 8)
    return c


# ------------------------------------------------------------------------------------------------ inputs --
def _topk(logits, k):
    """The k largest logits of each row, the lowest index first among equals."""
    return torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :k]


def _routes(c, gen):
    """Routes of a batch and their block-padded expert-grouped layout."""
    T, E, k, bs = c["T"], c["E"], c["k"], c["bs"]
    El = c["E_local"] or E
    dev = gen.device
    logits = torch.randn((T, E), generator=gen, device=dev)
    if c["zipf"]:
        rank = torch.randperm(E, generator=gen, device=dev) + 1
        logits = logits - c["zipf"] * torch.log(rank.double()).float()
    ids = _topk(logits, k)
    w = torch.softmax(logits.gather(1, ids).double(), dim=-1).float()
    lo = El if El < E else 0  # the second of the expert-parallel ranks
    lid = ids.reshape(-1) - lo
    lid = torch.where((lid >= 0) & (lid < El), lid, El)
    counts = torch.bincount(lid, minlength=El + 1)
    order = torch.sort(lid, stable=True)[1]
    start = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(lid)
    rank[order] = torch.arange(T * k, device=dev) - start[lid[order]]
    padded = (counts[:El] + bs - 1) // bs * bs
    offsets = torch.zeros(El + 1, dtype=torch.int64, device=dev)
    offsets[1:] = torch.cumsum(padded, 0)
    C = T * k + El * (bs - 1)
    local = lid < El
    inv = torch.where(local, offsets[lid.clamp(max=El - 1)] + rank, -1)
    sorted_ids = torch.full((C,), T * k, dtype=torch.int32, device=dev)
    sorted_ids[inv[local]] = torch.arange(T * k, dtype=torch.int32, device=dev)[local]
    i32 = torch.int32
    return dict(ids=ids.to(i32), w=w, counts=counts[:El].to(i32), offsets=offsets.to(i32), inv=inv.to(i32),
                sorted=sorted_ids, n_pad=offsets[-1:].to(i32), C=C, El=El, most=max(1, int(counts[:El].max())))


def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.bfloat16)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = gen.device
    s = dict(c)
    op = c["op"]
    if op == "gating_backward":
        T, E, k = c["T"], c["E"], c["k"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        x = torch.randn((T, E), generator=gen, device=dev).to(dt)
        ids = _topk(x.float(), k)
        z = x.double()
        p = torch.sigmoid(z) if c["scoring"] == "sigmoid" else torch.softmax(z, dim=-1)
        w = p.gather(1, ids)
        w = w / w.sum(-1, keepdim=True) if c["renorm"] else w
        s.update(x=x, ids=ids.to(torch.int32), w=w.float(), g=torch.randn((T, k), generator=gen, device=dev),
                 out=torch.zeros((T, E), dtype=dt, device=dev))
    elif op == "mx4_cast":
        s.update(x=_bf16(gen, c["rows"], c["K"]) * 0.02)
    else:
        r = _routes(c, gen)
        s.update(r)
        if op == "combine_backward":
            H = c["H"]
            s.update(gout=_bf16(gen, c["T"], H), y=_bf16(gen, r["C"], H),
                     gy=torch.zeros((r["C"], H), dtype=torch.bfloat16, device=dev))
        elif op == "gather_backward":
            s.update(gp=_bf16(gen, r["C"], c["H"]))
        else:
            K, N, El = c["K"], c["N"], r["El"]
            s["x"] = _bf16(gen, c["T"] if c["form"] == "up" else r["C"], K)
            # the weights, as a program keeps them: codes, and the scales of four blocks (128 elements) side by side
            qw = torch.empty((El, N, K // 2), dtype=torch.uint8, device=dev)
            sw = torch.empty((-(-K // 128), El, N, 4), dtype=torch.uint8, device=dev)
            for e in range(El):
                qw[e], sw[:, e] = _quantize(_bf16(gen, N, K) * 0.02)
            s.update(qw=qw, sw=sw.view(sw.shape[0], El * N, 4))
            s["y"] = torch.zeros((r["C"], N // 2 if c["form"] == "up" else N), dtype=torch.bfloat16, device=dev)
    return s


# -------------------------------------------------------------------------------------------- plain form --
def _quantize(x):
    """bf16 [rows, K] -> codes [rows, K/2] (the even element in the low half) and scale bytes [ceil(K/128), rows, 4]."""
    rows, K = x.shape
    b = x.float().view(rows, K // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(-127, 127)
    a = torch.ldexp(b, -e[..., None])
    m = a.abs()
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code; beyond 6 saturates
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code + 8 * torch.signbit(a)).to(torch.uint8).view(rows, K // 2, 2)
    chunks = -(-K // 128)
    scales = torch.full((rows, chunks * 4), 127, dtype=torch.uint8, device=x.device)
    scales[:, :K // 32] = (e + 127).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), scales.view(rows, chunks, 4).permute(1, 0, 2).contiguous()


def _dequantize(q, scales):
    """codes [rows, K/2] and scale bytes -> fp32 [rows, K]."""
    rows, half = q.shape
    table = torch.tensor(E2M1, device=q.device)
    v = torch.stack((table[(q & 15).int()], table[(q >> 4).int()]), -1).view(rows, half // 16, 32)
    e = scales.permute(1, 0, 2).reshape(rows, -1)[:, :half // 16].int() - 127
    return torch.ldexp(v, e[..., None]).view(rows, 2 * half)


def _plain(s):
    op = s["op"]
    if op == "gating_backward":
        x, g, w, ids = s["x"].float(), s["g"], s["w"], s["ids"].long()
        G = (g * w).sum(-1, keepdim=True)
        if s["scoring"] == "softmax" and not s["renorm"]:
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            return (p * (torch.zeros_like(x).scatter_add_(1, ids, g) - G)).to(s["x"].dtype)
        d = w * (g - G) if s["renorm"] else w * g
        if s["scoring"] == "sigmoid":
            d = d / (1 + torch.exp(x.gather(1, ids)))
        return torch.zeros_like(x).scatter_add_(1, ids, d).to(s["x"].dtype)
    if op == "mx4_cast":
        return _dequantize(*_quantize(s["x"])).to(torch.bfloat16)
    T, k, C = s["T"], s["k"], s["C"]
    inv = s["inv"].long()
    local = (inv >= 0).view(T, k, 1)
    if op == "combine_backward":
        H = s["H"]
        g = s["gout"].float().view(T, 1, H)
        gw = torch.where(local, s["y"][inv.clamp(min=0)].float().view(T, k, H) * g, 0.0).sum(-1)
        gy = torch.zeros((C + 1, H), dtype=torch.bfloat16, device=g.device)
        gy[torch.where(inv >= 0, inv, C)] = (s["w"].view(T, k, 1) * g).to(torch.bfloat16).view(T * k, H)
        return gy[:C], gw
    if op == "gather_backward":
        rows = s["gp"][inv.clamp(min=0)].float().view(T, k, s["H"])
        return torch.where(local, rows, 0.0).sum(1).to(torch.bfloat16)
    # mx4_product: rows of expert e at offsets[e], padded to the longest expert so that one batched product does
    K, N, El, most = s["K"], s["N"], s["El"], s["most"]
    x = s["x"]
    at = torch.arange(most, device=x.device)
    rows = s["offsets"][:El, None].long() + at
    valid = at < s["counts"][:, None]
    xq = _dequantize(*_quantize(x))
    if s["form"] == "up":
        token = torch.where(s["sorted"] < T * k, s["sorted"] // k, 0).long()
        src = token[rows.clamp(max=C - 1)]
    else:
        src = rows.clamp(max=C - 1)
    w = _dequantize(s["qw"].view(El * N, K // 2), s["sw"]).view(El, N, K)
    y = torch.bmm(xq[src], w.transpose(1, 2))
    if s["form"] == "up":
        gate, up = y[..., :N // 2], y[..., N // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    out = torch.zeros((C + 1, y.shape[-1]), dtype=torch.bfloat16, device=x.device)
    out[torch.where(valid, rows, C)] = y.to(torch.bfloat16)
    return out[:C]


# ---------------------------------------------------------------------------------------- framework's form --
def _own(s):
    import token_dispatch_topk_b200 as tdt
    op = s["op"]
    if op == "gating_backward":
        return tdt.moe_topk_softmax_backward(s["g"], s["x"], s["w"], s["ids"], s["renorm"], grad_logits=s["out"],
                                             scoring=s["scoring"])
    if op == "mx4_cast":
        return tdt.moe_dequantize_mx4(tdt.moe_quantize_mx4(s["x"]))
    if op == "combine_backward":
        return tdt.moe_combine_backward(s["gout"], s["y"], s["w"], s["inv"], grad_expert_out=s["gy"],
                                        sorted_token_ids=s["sorted"], num_tokens_post_pad=s["n_pad"], zero_pad=True)
    if op == "gather_backward":
        return tdt.moe_gather_backward(s["gp"], s["inv"], s["k"])
    K, N, El = s["K"], s["N"], s["El"]
    if s["form"] == "up":
        x = tdt.moe_gather_mx4(s["x"], s["k"], s["inv"], s["C"])
    else:
        x = tdt.moe_quantize_mx4(s["x"], num_rows=s["n_pad"])
    w = tdt.Mx4Tensor(s["qw"].view(El * N, K // 2), s["sw"])
    return tdt.moe_grouped_gemm_mx4(x, w, s["counts"], s["offsets"], out=s["y"], swiglu=s["form"] == "up")


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------ work and exact --
def work(case):
    c = case
    op = c["op"]
    if op == "gating_backward":
        T, E, k = c["T"], c["E"], c["k"]
        b = 2 if c["dtype"] == "bf16" else 4
        dense = c["scoring"] == "softmax" and not c["renorm"]
        read = T * E * b if dense else T * k * b if c["scoring"] == "sigmoid" else 0
        return {"bytes": read + T * E * b + 12 * T * k, "flops": T * (6 * E if dense else 6 * k)}
    if op == "mx4_cast":
        n = c["rows"] * c["K"]
        return {"bytes": 4 * n + 2 * n * 17 / 32, "flops": 4 * n}
    T, k, E = c["T"], c["k"], c["E"]
    El = c["E_local"] or E
    share = El / E
    P = T * k * share                        # rows on this rank
    tokens = T * (1 - (1 - share) ** k)      # tokens with such a row
    pads = El * (c["bs"] - 1) / 2            # pad rows, about
    if op == "combine_backward":
        H = c["H"]
        return {"bytes": 2 * H * (tokens + 2 * P + pads) + 12 * T * k, "flops": 3 * P * H}
    if op == "gather_backward":
        H = c["H"]
        return {"bytes": 2 * H * (P + T) + 4 * T * k, "flops": P * H}
    K, N = c["K"], c["N"]
    active = El * (1 - (1 - 1 / E) ** (T * k))  # experts with a row, about
    up = c["form"] == "up"
    return {"bytes": 2 * K * (tokens if up else P) + active * N * K * 17 / 32 + 2 * P * (N // 2 if up else N),
            "flops": 2 * P * N * K}


def _exact_mx4(x):
    """The 64-bit values that x (bf16 [rows, K]) has in the format."""
    rows, K = x.shape
    b = x.double().view(rows, K // 32, 32)
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -200))) - 2).clamp(-127, 127))
    a = (b / scale).abs().clamp(max=6.0)
    # spacing of the format at a: 0.5 below 2, then 1, then 2; torch.round takes a tie to the even multiple
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    return (torch.sign(b) * torch.round(a / step) * step * scale).view(rows, K)


def _exact_values(q, scales):
    """The 64-bit values of codes and scale bytes, by arithmetic on the fields of a code."""
    rows, half = q.shape
    v = torch.empty((rows, 2 * half), dtype=torch.float64, device=q.device)
    for i, c in enumerate((q & 15, q >> 4)):
        e, m = ((c >> 1) & 3).double(), (c & 1).double()
        v[:, i::2] = torch.where(c >= 8, -1.0, 1.0) * torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    for j in range(half // 16):
        v[:, 32 * j:32 * j + 32] *= torch.exp2(scales[j // 4, :, j % 4].double() - 127)[:, None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "gating_backward":
        # the weights' Jacobian, from the logits alone
        x, g, ids = s["x"].double(), s["g"].double(), s["ids"].long()
        sig = s["scoring"] == "sigmoid"
        f = torch.sigmoid(x) if sig else torch.softmax(x, -1)
        df = f.gather(1, ids)
        if s["renorm"]:
            total = df.sum(-1, keepdim=True)
            g = g / total - (g * df).sum(-1, keepdim=True) / total ** 2
        gf = torch.zeros_like(x).scatter_add_(1, ids, g)
        return gf * f * torch.sigmoid(-x) if sig else f * (gf - (gf * f).sum(-1, keepdim=True))
    if op == "mx4_cast":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device)
        for r in range(0, s["rows"], 1 << 15):
            out[r:r + (1 << 15)] = _exact_mx4(s["x"][r:r + (1 << 15)])
        return out
    T, k, C = s["T"], s["k"], s["C"]
    inv = s["inv"].long().view(T, k)
    if op == "combine_backward":
        gy = torch.zeros((C, s["H"]), dtype=torch.float64, device=inv.device)
        gw = torch.zeros((T, k), dtype=torch.float64, device=inv.device)
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            g = s["gout"][t].double()
            gy[inv[t, j]] = g * s["w"][t, j, None].double()
            gw[t, j] = torch.einsum("th,th->t", g, s["y"][inv[t, j]].double())
        return gy, gw
    if op == "gather_backward":
        gx = torch.zeros((T, s["H"]), dtype=torch.float64, device=inv.device)
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            gx[t] += s["gp"][inv[t, j]].double()
        return gx
    N, K = s["N"], s["K"]
    out = torch.zeros((C, N // 2 if s["form"] == "up" else N), dtype=torch.float64, device=inv.device)
    first, count = s["offsets"].tolist(), s["counts"].tolist()
    for e in range(s["El"]):
        r = slice(first[e], first[e] + count[e])
        x = s["x"][s["sorted"][r].long() // k] if s["form"] == "up" else s["x"][r]
        y = _exact_mx4(x) @ _exact_values(s["qw"][e], s["sw"][:, e * N:(e + 1) * N]).T
        if s["form"] == "up":
            y = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:]
        out[r] = y
    return out
