"""What the gradients and the 4-bit entry points refuse, on the CPU: every call here is turned down (or has nothing to
do) before a launch."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt
from token_dispatch_topk_b200 import binding as B

OK, INVALID, UNSUPPORTED = tdt.MOE_OK, tdt.MOE_ERR_INVALID_ARG, tdt.MOE_ERR_UNSUPPORTED
P = 1 << 20   # a 16-byte aligned address that is never read
ODD = P + 8   # one that is not

COMBINE = dict(grad_out=P, expert_out=P, topk_weights=P, inv_perm=P, sorted_ids=None, n_pad=None, T=4, k=2, H=64,
               capacity=64, flags=0, gy=P, gw=P, status=None, stream=None)
GATHER = dict(gp=P, inv_perm=P, T=4, k=2, H=64, capacity=64, gx=P, status=None, stream=None)
GATING = dict(gw=P, logits=P, dtype=1, w=P, ids=P, T=4, E=8, k=2, flags=0, gx=P, status=None, stream=None)
QUANT = dict(x=P, rows=4, K=64, num_rows=None, codes=P, scales=P, stream=None)
DEQUANT = dict(codes=P, scales=P, rows=4, K=64, out=P, stream=None)
GATHER4 = dict(hidden=P, T=4, H=64, k=2, inv_perm=P, capacity=64, codes=P, scales=P, status=None, stream=None)
GEMM = dict(x=P, xs=P, w=P, ws=P, counts=P, offsets=P, E=4, capacity=64, N=64, K=64, flags=0, out=P, status=None,
            stream=None)

REFUSED = [
    ("moe_combine_backward", COMBINE, INVALID, [dict(T=-1), dict(k=0), dict(H=0), dict(H=60), dict(capacity=-1),
     dict(flags=1), dict(flags=2), dict(gy=None, gw=None), dict(grad_out=None), dict(topk_weights=None),
     dict(inv_perm=None), dict(expert_out=None), dict(grad_out=ODD), dict(expert_out=ODD), dict(gy=ODD),
     dict(T=1 << 30), dict(capacity=1 << 31), dict(flags=2, sorted_ids=P, n_pad=P, gy=None)]),
    ("moe_combine_backward", COMBINE, UNSUPPORTED, [dict(k=33)]),
    ("moe_combine_backward", COMBINE, OK, [dict(T=0), dict(T=0, grad_out=None, topk_weights=None, inv_perm=None, gw=None),
     dict(T=0, capacity=0, gy=None, gw=None, expert_out=None)]),
    ("moe_gather_backward", GATHER, INVALID, [dict(T=-1), dict(k=0), dict(H=0), dict(H=12), dict(capacity=-1),
     dict(gp=None), dict(inv_perm=None), dict(gx=None), dict(gp=ODD), dict(gx=ODD), dict(T=1 << 30)]),
    ("moe_gather_backward", GATHER, UNSUPPORTED, [dict(k=33)]),
    ("moe_gather_backward", GATHER, OK, [dict(T=0)]),
    ("moe_topk_softmax_backward", GATING, INVALID, [dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(dtype=2),
     dict(flags=2), dict(gw=None), dict(logits=None), dict(w=None), dict(ids=None), dict(gx=None), dict(gx=P + 1),
     dict(logits=P + 1), dict(dtype=0, gx=P + 2), dict(T=1 << 41), dict(flags=16, logits=None),
     dict(flags=17, logits=None)]),
    ("moe_topk_softmax_backward", GATING, UNSUPPORTED, [dict(E=1025), dict(E=64, k=33)]),
    ("moe_topk_softmax_backward", GATING, OK, [dict(T=0)]),
    ("moe_quantize_mx4", QUANT, INVALID, [dict(rows=-1), dict(K=0), dict(K=48), dict(K=1 << 21), dict(rows=1 << 31),
     dict(x=None), dict(codes=None), dict(scales=None), dict(x=ODD), dict(codes=ODD), dict(scales=ODD)]),
    ("moe_quantize_mx4", QUANT, OK, [dict(rows=0)]),
    ("moe_dequantize_mx4", DEQUANT, INVALID, [dict(rows=-1), dict(K=0), dict(K=48), dict(out=None), dict(codes=None),
     dict(scales=None), dict(out=ODD), dict(codes=ODD), dict(scales=ODD)]),
    ("moe_dequantize_mx4", DEQUANT, OK, [dict(rows=0)]),
    ("moe_gather_mx4", GATHER4, INVALID, [dict(T=-1), dict(k=0), dict(H=40), dict(H=0), dict(capacity=-1),
     dict(hidden=None), dict(inv_perm=None), dict(codes=None), dict(scales=None), dict(hidden=ODD), dict(codes=ODD),
     dict(T=1 << 30)]),
    ("moe_gather_mx4", GATHER4, UNSUPPORTED, [dict(k=33)]),
    ("moe_gather_mx4", GATHER4, OK, [dict(T=0)]),
    ("moe_grouped_gemm_mx4", GEMM, INVALID, [dict(E=0), dict(capacity=-1), dict(N=0), dict(N=12), dict(K=0),
     dict(K=48), dict(flags=1), dict(flags=32, N=24), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None),
     dict(counts=None), dict(offsets=None), dict(out=None), dict(x=ODD), dict(xs=ODD), dict(w=ODD), dict(ws=ODD),
     dict(out=ODD), dict(capacity=1 << 31), dict(K=1 << 21), dict(N=1 << 21)]),
    ("moe_grouped_gemm_mx4", GEMM, UNSUPPORTED, [dict(E=1025)]),
    ("moe_grouped_gemm_mx4", GEMM, OK, [dict(capacity=0)]),
]


@pytest.mark.parametrize("name,base,want,change", [(n, b, w, c) for n, b, w, cs in REFUSED for c in cs])
def test_entry_points_refuse(name, base, want, change):
    assert set(change) <= set(base)
    assert getattr(B.load_library(), name)(*{**base, **change}.values()) == want


def test_cpu_tensors_are_refused():
    bf16, i32 = torch.bfloat16, torch.int32
    rows, w, inv = torch.zeros((8, 64), dtype=bf16), torch.zeros((4, 2)), torch.zeros(8, dtype=i32)
    q = tdt.alloc_mx4(8, 64, "cpu")
    for call in (lambda: tdt.moe_combine_backward(rows[:4], rows, w, inv),
                 lambda: tdt.moe_gather_backward(rows, inv, 2),
                 lambda: tdt.moe_topk_softmax_backward(w, torch.zeros((4, 8)), w, torch.zeros((4, 2), dtype=i32), True),
                 lambda: tdt.moe_quantize_mx4(rows), lambda: tdt.moe_dequantize_mx4(q),
                 lambda: tdt.moe_gather_mx4(rows[:4], 2, inv, 8),
                 lambda: tdt.moe_grouped_gemm_mx4(q, q, torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_shapes_are_checked_before_anything_else():
    bf16, i32 = torch.bfloat16, torch.int32
    q = tdt.alloc_mx4(8, 64, "cpu")
    for call in (lambda: tdt.alloc_mx4(4, 40, "cpu"), lambda: tdt.alloc_mx4(4, 0, "cpu"),
                 lambda: tdt.moe_quantize_mx4(torch.zeros(64, dtype=bf16)),
                 lambda: tdt.moe_quantize_mx4(torch.zeros((8, 64), dtype=bf16), out=tdt.alloc_mx4(8, 32, "cpu")),
                 lambda: tdt.moe_gather_backward(torch.zeros((8, 64), dtype=bf16), torch.zeros(7, dtype=i32), 2),
                 lambda: tdt.moe_gather_backward(torch.zeros((8, 64), dtype=bf16), torch.zeros(8, dtype=i32), 0),
                 lambda: tdt.moe_topk_softmax_backward(torch.zeros((4, 2)), torch.zeros((4, 8), dtype=torch.float16),
                                                       torch.zeros((4, 2)), torch.zeros((4, 2), dtype=i32), True),
                 lambda: tdt.moe_grouped_gemm_mx4(q, q, torch.zeros(3, dtype=i32), torch.zeros(4, dtype=i32)),
                 lambda: tdt.moe_grouped_gemm_mx4(q, tdt.alloc_mx4(8, 32, "cpu"), torch.zeros(2, dtype=i32),
                                                  torch.zeros(3, dtype=i32)),
                 lambda: tdt.moe_grouped_gemm_mx4(q, q, torch.zeros(8, dtype=i32), torch.zeros(9, dtype=i32), swiglu=True),
                 lambda: tdt.Mx4Experts(torch.zeros((2, 6, 64), dtype=bf16), torch.zeros((2, 64, 4), dtype=bf16), 8)):
        with pytest.raises(ValueError):
            call()
