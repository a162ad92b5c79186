"""Refusals of moe_route_far_weights; no call here reaches a launch."""
import pytest

import align_moe_route_amd as amr

P = 0x10000  # aligned fake device address: never dereferenced, validation fails first


def far(logits=P, dt=0, ids=P, M=4, E=8, k=2, weights=P):
    return amr.lib().moe_route_far_weights(logits, dt, ids, M, E, k, weights, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(dt=2), -1),
    (dict(logits=None), -2), (dict(ids=None), -2), (dict(weights=None), -2), (dict(logits=P + 2), -3),
    (dict(logits=P + 1, dt=1), -3), (dict(ids=P + 2), -3), (dict(weights=P + 2), -3), (dict(M=(1 << 30) + 1, k=1), -5),
    (dict(M=1 << 28, k=8), -5), (dict(M=0, logits=None), 0),
])
def test_codes(kw, code):
    assert far(**kw) == code
