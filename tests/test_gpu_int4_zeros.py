"""int4_matvec where the weights are zero (codes of 8), or nearly all of them: codes enter a
chunk of 32 columns as 16 + c and 24 sum x is taken off, which is exact for small integers.
Otherwise a chunk is a chain of 16 pair products, two roundings each, and one more, of
partial sums of at most 55 sum |x|, each by 2^-24; sum x is such a chain of 32 roundings of
at most sum |x|, times 24: 33 + 32 * 24 / 55 < 48 of 55 * 2^-24 scale sum |x|, and the scale and
the sum over the chunks less than two more where the weights are zero.  The result is
rounded to x's type."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import HALF, STEP, f64, normal

pytestmark = pytest.mark.gpu


def zeros(E, N, K, group, t):
    Kp = -(-K // 128) * 128
    return amr.Int4(torch.full((E, N, Kp // 2), 0x88, dtype=torch.uint8, device="cuda"),
                    torch.ones(E, N, Kp // group, dtype=t, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", [128, 1001, 2176])
def test_whole_numbers_are_exact(K, dtype):
    t, g = HALF[dtype], torch.Generator().manual_seed(1)
    q = zeros(3, 10, K, 32, t)
    x = torch.randint(-40, 41, (5, K), generator=g).to(t).cuda()
    ids = torch.tensor([[0, 1], [2, 0], [1, 1], [2, 2], [0, 2]], dtype=torch.int32, device="cuda")
    v = torch.rand(5, 2, generator=g).cuda()
    assert not amr.int4_matvec(x, q, ids).any()
    assert not amr.int4_matvec(x, q, ids, gated=True).any()
    assert not amr.int4_matvec(x, q, ids, weights=v).any()
    q.codes[:, 3, 7] = 0x9F  # weights 7 and 1 at columns 14 and 15
    y = amr.int4_matvec(x, q, ids)
    assert torch.equal(y[:, :, 3], (7 * x[:, 14].float() + x[:, 15].float()).to(t)[:, None].expand(-1, 2))
    y[:, :, 3] = 0
    assert not y.any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", [32, 128, 1001, 3584])
def test_other_values_leave_little(K, dtype):
    t = HALF[dtype]
    x = normal((64, K), t, 2)
    ids = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    y = f64(amr.int4_matvec(x, zeros(1, 4, K, 128, t), ids))
    bound = 50 * 55 * 2.0 ** -24 * np.abs(f64(x)).sum(1)
    rel, tiny = STEP[t]
    assert (np.abs(y) <= (bound * (1 + rel) + tiny)[:, None, None]).all()


def test_subnormal_inputs():
    """FP16 below 2^-14 counts in full: 2^-24 to 60 * 2^-24 times weights of about 64."""
    E, N, K = 3, 12, 256
    g = torch.Generator().manual_seed(3)
    q = amr.int4_quantize(normal((E, N, K), torch.float16, 4, 64.0), 64)
    m = torch.randint(-60, 61, (4, K), generator=g)
    x = (m.double() * 2.0 ** -24).to(torch.float16).cuda()
    ids = torch.tensor([[0], [2], [1], [0]], dtype=torch.int32, device="cuda")
    code = q.codes.cpu().numpy()
    w = np.empty((E, N, K))
    w[..., 0::2], w[..., 1::2] = code & 15, code >> 4
    scale = np.repeat(f64(q.scales), 64, axis=-1)
    w = (w - 8) * scale
    want = np.stack([w[int(e)] @ f64(x[i]) for i, e in enumerate(ids[:, 0])])
    size = np.stack([scale[int(e)] @ np.abs(f64(x[i])) for i, e in enumerate(ids[:, 0])])
    rel, tiny = STEP[torch.float16]
    slack = (50 * 55 + 7 * K / 32) * 2.0 ** -24 * size  # the chunks' sums: |w| is up to 7 scales
    got = f64(amr.int4_matvec(x, q, ids))[:, 0]
    assert (np.abs(got - want) <= rel * (np.abs(want) + slack) + slack + tiny).all() and np.abs(want).max() > 0.001
