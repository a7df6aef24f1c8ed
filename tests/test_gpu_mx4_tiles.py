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


@pytest.mark.parametrize("bs", [1, 8])
@pytest.mark.parametrize("K,N,gate", [(64, 136, False), (288, 200, False), (544, 272, True)])
def test_one_expert_of_several_tiles_among_small_ones(K, N, gate, bs):
    """Skewed routes: few rows an expert on the whole, so that single CTAs take the tiles, and a few experts with more
    rows than a tile."""
    require_gpu()
    gen = torch.Generator().manual_seed(K + bs)
    counts, off, cap = layout([200, 65, 129, 1, 0, 64, 17] + [0, 1] * 7, bs)
    assert cap < 64 * 21
    x, w = random_mx4(gen, cap, K), random_mx4(gen, 21 * N, K)
    x.scales[:, int(off[-1]):] = 255  # rows of no expert hold NaN
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_and_check(x, w, counts, off, N, gate, status)
    assert tdt.moe_read_status(status) == tdt.MOE_OK


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("pair", [False, True])
def test_more_than_32_tiles_a_cta(pair, gate):
    """The tiles are worked out 32 at a time: several such batches a CTA or pair, the last of them ragged."""
    require_gpu()
    gen = torch.Generator().manual_seed(7)
    E, K, N = 50, 32, 16384 if not gate else 16416
    counts, off, cap = layout([1 + i % 7 for i in range(E)], 64 if pair else 1)
    tiles = E * (-(-(N // 2 if gate else N) // ((128 if pair else 64) * (1 if gate else 2))))
    ctas = torch.cuda.get_device_properties(0).multi_processor_count // (2 if pair else 1)
    assert (cap >= 64 * E) == pair and tiles > 32 * ctas
    run_and_check(random_mx4(gen, cap, K), random_mx4(gen, E * N, K), counts, off, N, gate)
