"""Failure detection in the tree attention with copies in flight, without a GPU fault.

attn_debug_inject(3): every CTA begins as if one of its waits had run out.  The load-issuing warp issues the copies that
need no wait and leaves, as all others do, the one that the values of a tree's keys go through on their way to the products
among them.  On its way out it waits for its own copies, by the barriers that the copies themselves complete.  They land
within microseconds, so the call ends far within one wait's budget and records nothing."""
import time

import pytest
import torch

import exact_attention_forward_06_gb300 as A
from tree_ref import Batch

pytestmark = pytest.mark.gpu

BUDGET = 0.5    # seconds


@pytest.mark.parametrize("sizes,contexts,pad", [
    ([200], [50], 0),                       # both tiles of each unit are the tree's; no unit is cut
    ([30, 256, 5], [700, 300, 0], 20),      # cut units; values of keys before the tree go to the products at once
])
def test_copies_in_flight_are_waited_for_by_their_own_barriers(sizes, contexts, pad):
    b = Batch(70, sizes, contexts, 4, 2, pad=pad)
    dev = [x.cuda() for x in (b.q, b.k, b.v, b.table, b.lens, b.cu, b.parents)]
    ws = torch.full((A.fwd_tree_paged_workspace_bytes(len(sizes), 4, 2, 128, max(sizes)),), 0x7f, dtype=torch.uint8,
                    device="cuda")

    def run():
        return A.fwd_tree_paged(*dev, max_seqlen_q=max(sizes), workspace=ws)

    good = [x.clone() for x in run()]
    assert A.device_status()[0] == 0
    A.set_wait_budget_ns(int(BUDGET * 1e9))
    try:
        for _ in range(5):
            A.debug_inject(3)
            t = time.perf_counter()
            run()
            status = A.device_status()       # synchronises
            t = time.perf_counter() - t
            assert status[0] == 0, status
            assert t < BUDGET / 2, t
    finally:
        A.debug_inject(0)
        A.set_wait_budget_ns(0)
    again = run()
    assert A.device_status()[0] == 0
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])
