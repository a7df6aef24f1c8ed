"""New outputs of the calls that are given a stream's handle, on the GPU."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


def test_handle_0_takes_the_default_streams_memory():
    """A tensor that a side stream freed and still has to read is not handed to calls on the default stream, however
    often they are made, and those calls use one piece of memory again and again."""
    require_gpu()
    rows, K = 4096, 2048
    q = tdt.moe_quantize_mx4(torch.full((rows, K), 3.0, dtype=torch.bfloat16, device="cuda"), stream=0)
    sides = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ys = []
    for side in sides:
        with torch.cuda.stream(side):
            x = torch.full((rows, K), 5.0, dtype=torch.bfloat16, device="cuda")
            ys.append(torch.empty_like(x))
            torch.cuda._sleep(200_000_000)  # about 0.1 s
            ys[-1].copy_(x)
            del x
    used, last = set(), torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    for _ in range(40):  # more calls than torch keeps streams in its pool
        back = tdt.moe_dequantize_mx4(q, stream=0)
        used.add(back.data_ptr())
        last.copy_(back)
        del back
    torch.cuda.synchronize()
    assert all((y == 5).all() for y in ys) and (last == 3).all()
    assert len(used) == 1
