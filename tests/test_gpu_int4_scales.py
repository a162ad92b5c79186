"""int4_matvec takes no part in autograd: scales that want a gradient are refused too."""
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import normal

pytestmark = pytest.mark.gpu


def test_scales_that_want_a_gradient():
    q = amr.int4_quantize(normal((3, 8, 64), torch.bfloat16, 1), 32)
    x, ids = normal((2, 64), torch.bfloat16, 2), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    want = amr.int4_matvec(x, q, ids)
    q = amr.Int4(q.codes, q.scales.requires_grad_())
    with pytest.raises(ValueError, match="autograd"):
        amr.int4_matvec(x, q, ids)
    with torch.no_grad():
        assert torch.equal(amr.int4_matvec(x, q, ids), want)
