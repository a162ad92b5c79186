"""Rows at the border of what the router's gradient and the trained weights are
defined for: NaN beside -infinity, and logits so low that FP32 scores vanish."""
import numpy as np
import pytest

from test_gpu_balance import DT, check_backward

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k", [(64, 1), (64, 2), (64, 16), (64, 20), (700, 4), (700, 30), (2000, 3)])
def test_nan_pick_reaches_every_pick_of_its_row(E, k, dtype):
    """The weights share their sum, so one NaN logit makes each of them NaN, also
    where the other picks have the score zero."""
    rng = np.random.default_rng(E + k)
    x = torch.from_numpy(rng.standard_normal((7, E))).to(DT[dtype])
    ids = np.stack([np.sort(rng.choice(E, k, replace=False)) for _ in range(7)]).astype(np.int32)
    nan, inf = float("nan"), float("inf")
    for t, other in ((0, -inf), (1, nan), (2, None), (3, -1000.0), (4, inf)):
        if other is not None:
            x[t, ids[t]] = other
        x[t, ids[t, k // 2]] = nan
    x[5, ids[5]] = -inf  # no NaN: every weight zero
    check_backward(x, ids, None, None, balance=False)
