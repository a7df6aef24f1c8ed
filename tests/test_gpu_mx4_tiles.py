"""The tiles of the 4-bit product on the GPU: rings of stages filled to every level, many launches in a row, and (from
test_gpu_mx4_product) every output against 64 bits."""
import pytest
import torch

import token_dispatch_topk_b200 as tdt

from gpu_helpers import require_gpu
from test_gpu_mx4_product import layout, random_mx4, run_and_check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("stages", [1, 2, 4, 5, 6, 7, 8])
def test_launches_in_a_row(stages, pair, gate):
    """Products of one tile a CTA or pair, some of them without one, each launched as the one before ends."""
    require_gpu()
    gen = torch.Generator().manual_seed(stages)
    K, N = 256 * stages, 512
    counts, off, cap = layout([3, 130, 0] if pair else [3, 60, 0], 64 if pair else 1)
    assert (cap >= 64 * 3) == pair  # which form a capacity gets
    x, w = random_mx4(gen, cap, K), random_mx4(gen, 3 * N, K)
    want = run_and_check(x, w, counts, off, N, gate)
    outs = [torch.full_like(want, 77.0) for _ in range(40)]
    c, o = counts.cuda(), off.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out in outs:
        tdt.moe_grouped_gemm_mx4(x, w, c, o, out=out, swiglu=gate, device_status=status)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)
    assert tdt.moe_read_status(status) == tdt.MOE_OK
