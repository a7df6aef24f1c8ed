"""The size limits that the header states for the gradients and the 4-bit casts, on the CPU: refused before a launch."""
import pytest

import token_dispatch_topk_b200 as tdt
from token_dispatch_topk_b200 import binding as B

P = 1 << 20  # a 16-byte aligned address that is never read


@pytest.mark.parametrize("name,args", [
    # T * H = 2^40 + 2^27, with 2^29 slots
    ("moe_gather_backward", (P, P, 1 << 27, 4, 8200, 64, P, None, None)),
    ("moe_gather_backward", (P, P, 1 << 29, 1, 1 << 20, 64, P, None, None)),
    # rows * K = 2^42, 2^41 + 2^31
    ("moe_quantize_mx4", (P, 1 << 30, 4096, None, P, P, None)),
    ("moe_quantize_mx4", ((P, (1 << 21) + (1 << 11), 1 << 20, None, P, P, None))),
    ("moe_dequantize_mx4", (P, P, 1 << 30, 4096, P, None)),
    # of the tokens, of the gathered rows
    ("moe_gather_mx4", (P, 1 << 29, 8192, 1, P, 64, P, P, None, None)),
    ("moe_gather_mx4", (P, 64, 1 << 20, 1, P, (1 << 21) + 1, P, P, None, None)),
])
def test_more_elements_than_stated_are_refused(name, args):
    assert getattr(B.load_library(), name)(*args) == tdt.MOE_ERR_UNSUPPORTED
