"""The block-scaled product's barriers between the two CTAs of a pair.  A wait that
orders too little shows only now and then, as a stale scale, so the source is read:
a wait whose acquire is the CTA's alone is for barriers at which only this CTA's
threads arrive; what the peer has written to shared memory is acquired at the
cluster's scope, and memory is given back to the peer by a release at that scope."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_routing_count_prefix_gb300", "csrc")
# at which this CTA's threads alone arrive; kScaleFull: of the scales, from the sums' first barrier on
LOCAL = ("plan_full", "plan_empty", "scale_full", "scale_empty", "kScaleFull", "amax_read", "row_full")
TENSOR = ("acc_full", "acc_empty")  # tensor memory of both CTAs


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def names(call):
    """(function, identifiers of its first argument) of every such call."""
    return [(f, re.findall(r"[A-Za-z_]\w*", arg)) for f, arg in re.findall(rf"\b({call})\(([^,;]*)", code("block_scaled.cu"))]


def test_waits():
    seen = set()
    for f, ids in names(r"mbar_(?:wait|test|try_wait)\w*"):
        local = [i for i in ids if i in LOCAL]
        if f in ("mbar_wait", "mbar_wait_warp"):  # they acquire the cluster's writes: right for any barrier
            seen.update(ids)
        elif local:
            assert "_cta" in f, (f, ids)
        else:
            assert any(i in TENSOR for i in ids) and f in ("mbar_wait_tensor", "mbar_test_tensor"), (f, ids)
    assert {"full", "swapped", "amax_empty"} <= seen


def test_shared_memory_goes_back_by_a_release():
    to_peer = [(f, ids) for f, ids in names(r"mbar_arrive\w*") if "map_rank" in ids or "leader_empty" in ids]
    assert to_peer
    for f, ids in to_peer:
        if "leader_empty" in ids:
            assert f == "mbar_arrive_tensor"
        else:
            assert f == "mbar_arrive_peer_release", (f, ids)


@pytest.mark.parametrize("f,has", [("mbar_try_wait", "try_wait.parity.acquire.cluster"),
                                   ("mbar_arrive_peer_release", "arrive.release.cluster.shared::cluster"),
                                   ("mbar_try_wait_tensor", "try_wait.parity.relaxed.cluster"),
                                   ("mbar_test_tensor", "test_wait.parity.relaxed.cluster"),
                                   ("mbar_arrive_tensor", "arrive.relaxed.cluster.shared::cluster")])
def test_scopes(f, has):
    s = code("block_tensor.cuh")
    body = s[re.search(rf"\b{f}\(uint32_t bar", s).start():]
    assert has in body[:body.index("\n}\n")]
