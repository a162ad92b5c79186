"""What experts_train knows of the route that it is given: its experts and its block."""
import pytest

import align_moe_route_amd as amr

torch = pytest.importorskip("torch")
from align_moe_route_amd.experts import _holds_experts  # noqa: E402


def route(M, E, k, block, rows=0, blocks=0):
    i32 = torch.int32
    return amr.RouteSortOutput(torch.zeros(M, k, dtype=i32), torch.zeros(M, k),
                               torch.zeros(amr.max_rows(M, E, k, block) + rows, dtype=i32),
                               torch.zeros(amr.max_blocks(M, E, k, block) + blocks, dtype=i32), torch.zeros(1, dtype=i32))


@pytest.mark.parametrize("M,k", [(64, 4), (1, 2)])  # more routes than experts, and fewer
def test_known_route(M, k):
    r = amr._routed(route(M, 16, k, 32), 16, 32)
    assert _holds_experts(r, 16, 32) and _holds_experts(r, 17, 32)
    for E, block in ((15, 32), (8, 32), (16, 64), (16, 16)):
        with pytest.raises(ValueError):
            _holds_experts(r, E, block)


def test_route_made_by_hand():
    assert _holds_experts(route(64, 16, 4, 32), 16, 32)
    for r in (route(64, 17, 4, 32), route(64, 16, 4, 64), route(64, 16, 4, 32, rows=32), route(64, 16, 4, 32, blocks=1)):
        assert not _holds_experts(r, 16, 32)
    assert not _holds_experts(route(4, 16, 4, 32), 16, 32)  # as long as one of 1000 experts


def test_knowledge_follows_the_metadata():
    r = amr._routed(route(2, 8, 2, 16), 8, 16)
    assert (r._replace(weights=r.weights + 1).experts, r._replace(ids=r.ids).block) == (8, 16)
    assert r._replace(sorted_ids=r.sorted_ids).experts is None and amr.RouteSortOutput(*r).block is None
    ids, weights, *meta = r  # five parts, as ever
    assert len(meta) == 3 and amr.RouteSortOutput(ids, weights, *meta) == r
    assert amr._routed(("another", "tuple"), 8, 16) == ("another", "tuple")
