"""Outputs of the tree operators that lie over their inputs are refused before any launch (CPU): blocks read the inputs in
any order with other blocks' writes.  Only calls that have to be refused are made: addresses are made up."""
import pytest

import exact_attention_forward_06_gb300 as A
from exact_attention_forward_06_gb300 import _binding


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_binding.LIBRARY_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return A.load()


MB = 1 << 20
B, LAYERS, HKV, WIDTH, PAGES, MAXB = 3, 2, 2, 8, 10, 4
POOL = LAYERS * PAGES * 16 * HKV * 128 * 2
COMPACT = dict(k=MB, v=2 * MB, bt=3 * MB, sl=4 * MB, cu=5 * MB, path=6 * MB, counts=7 * MB, out=8 * MB, B=B, layers=LAYERS,
               Hkv=HKV, total=9, width=WIDTH, d=128, page=16, npages=PAGES, maxb=MAXB)
COMPACT_BYTES = dict(k=POOL, v=POOL, bt=B * MAXB * 4, sl=B * 4, cu=(B + 1) * 4, path=B * WIDTH * 4, counts=B * 4)


@pytest.mark.parametrize("name", COMPACT_BYTES)
@pytest.mark.parametrize("place", ["first", "last", "before"])
def test_compact_refuses_lengths_over_an_input(lib, name, place):
    at = {"first": COMPACT[name], "last": COMPACT[name] + COMPACT_BYTES[name] - 4, "before": COMPACT[name] - (B - 1) * 4}[place]
    assert lib.attn_compact_paged(*dict(COMPACT, out=at).values(), None) == 1


@pytest.mark.parametrize("v", [MB + 256, MB + POOL - 256, MB - POOL + 256])
def test_compact_refuses_pools_over_parts_of_one_another(lib, v):
    assert lib.attn_compact_paged(*dict(COMPACT, v=v, k=MB).values(), None) == 1
