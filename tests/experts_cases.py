"""Shared by the tests of the experts' operators: routings, 16-bit inputs and the
float64 view of what the GPU was given."""
import numpy as np
import torch

import align_moe_route_amd as amr

HALF = {"bf16": torch.bfloat16, "f16": torch.float16}
# half a step of a type, relative to the value, and absolute below its normal range
STEP = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float16: (2.0 ** -11, 2.0 ** -25),
        torch.float32: (2.0 ** -24, 2.0 ** -150)}


def ids_of(M, E, k, seed, dropped=0.0, only=None):
    """[M, k] ids, ascending in a row and distinct where E allows, some dropped (-1);
    `only` keeps the routes to the first experts."""
    rng = np.random.default_rng(seed)
    n = E if only is None else only
    ids = np.stack([np.sort(rng.permutation(n)[:k] if n >= k else rng.integers(0, n, k)) for _ in range(M)]) \
        if M else np.zeros((0, k))
    ids = ids.astype(np.int32)
    ids[rng.random(ids.shape) < dropped] = -1
    return ids


class Routed:
    """Metadata of given ids on the GPU and on the host."""

    def __init__(self, ids, E, block):
        self.M, self.k = ids.shape
        self.E, self.block = E, block
        self.ids = torch.from_numpy(ids).cuda()
        out = amr.sort_from_ids(self.ids, E, block)
        self.meta = (out.sorted_ids, out.expert_of_block, out.num_post_pad)
        self.cap = amr.max_rows(self.M, E, self.k, block)
        self.npp = int(out.num_post_pad.item())
        self.sid = out.sorted_ids.cpu().numpy()
        self.eob = out.expert_of_block.cpu().numpy()
        s = self.sid[:self.npp]
        self.live = (s >= 0) & (s < self.M * self.k)


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, want, mag, steps, dtype):
    """|got - want| within half a step of the output's type, plus `steps` FP32 roundings
    (each at most 2^-23 of the magnitudes' sum, which bounds every partial sum)."""
    rel, tiny = STEP[dtype]
    got = f64(got)
    assert np.isfinite(got).all() or not np.isfinite(want).all()
    slack = steps * 2.0 ** -23 * mag
    bound = rel * (np.abs(want) + slack) + tiny + slack
    bad = np.abs(got - want) > bound
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - want) / (bound + 1e-300))))
