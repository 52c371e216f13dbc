"""Outputs of the tree operators that lie over their inputs are refused before any launch (CPU): blocks read the inputs in
any order with other blocks' writes.  Only calls that have to be refused are made: addresses are made up."""
import pytest
import torch

import exact_attention_forward_06_gb300 as A
from exact_attention_forward_06_gb300 import _binding


@pytest.fixture(scope="module")
def lib():
    import os
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: a call that was not refused would launch")
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


BV, TOTAL, V = 3, 9, 100
VERIFY = dict(logits=MB, draft=2 * MB, dtype=0, tok=3 * MB, par=4 * MB, cu=5 * MB, temp=6 * MB, u=7 * MB, noise=8 * MB,
              path=9 * MB, out=10 * MB, counts=11 * MB, B=BV, total=TOTAL, V=V, width=WIDTH, ls=V, ds=V + 20, ns=V + 4,
              ws=12 * MB, wsb=MB)
VERIFY_READS = dict(logits=((TOTAL - 1) * V + V) * 2, draft=((TOTAL - 1) * (V + 20) + V) * 2, tok=TOTAL * 4, par=TOTAL * 4,
                    cu=(BV + 1) * 4, temp=BV * 4, u=TOTAL * 4, noise=((BV - 1) * (V + 4) + V) * 4)
VERIFY_WRITES = dict(path=BV * WIDTH * 4, out=BV * WIDTH * 4, counts=BV * 4)


def _verify(lib, **kw):
    return lib.attn_verify_tree(*dict(VERIFY, **kw).values(), None)


@pytest.mark.parametrize("read", VERIFY_READS)
@pytest.mark.parametrize("written", VERIFY_WRITES)
def test_verify_refuses_outputs_over_an_input(lib, read, written):
    for at in (VERIFY[read], VERIFY[read] + VERIFY_READS[read] - 4, VERIFY[read] - VERIFY_WRITES[written] + 4):
        assert _verify(lib, **{written: at}) == 1


def test_verify_refuses_outputs_over_one_another(lib):
    for a, b in (("path", "out"), ("path", "counts"), ("out", "counts")):
        for at in (VERIFY[a], VERIFY[a] + VERIFY_WRITES[a] - 4, VERIFY[a] - VERIFY_WRITES[b] + 4):
            assert _verify(lib, **{b: at}) == 1


def test_verify_refuses_a_workspace_over_anything(lib):
    need = A.verify_tree_workspace_bytes(BV, TOTAL, V, WIDTH, with_draft=True)
    for name in list(VERIFY_READS) + list(VERIFY_WRITES):
        assert _verify(lib, ws=VERIFY[name]) == 1
        assert _verify(lib, ws=VERIFY[name] - need // 256 * 256) == 1


BT, HQ, TQ = 3, 4, 9
TREE = dict(q=MB, k=2 * MB, v=3 * MB, bt=4 * MB, sl=5 * MB, cu=6 * MB, par=7 * MB, out=8 * MB, lse=9 * MB, B=BT, Hq=HQ, Hkv=HKV,
            total=TQ, longest=5, d=128, page=16, npages=PAGES, maxb=MAXB, scale=0.1, mode=0, ws=64 * MB, wsb=64 * MB)
TREE_READS = dict(q=TQ * HQ * 256, k=PAGES * 16 * HKV * 256, v=PAGES * 16 * HKV * 256, bt=BT * MAXB * 4, sl=BT * 4,
                  cu=(BT + 1) * 4, par=TQ * 4)
TREE_WRITES = dict(out=TQ * HQ * 256, lse=TQ * HQ * 4)


def _tree(lib, **kw):
    return lib.attn_fwd_tree_paged(*dict(TREE, **kw).values(), None)


@pytest.mark.parametrize("read", TREE_READS)
def test_tree_attention_refuses_outputs_over_an_input(lib, read):
    a, n = TREE[read], TREE_READS[read]
    for at in (a, a + (n - 1) // 16 * 16, a - TREE_WRITES["out"] + 16):
        assert _tree(lib, out=at) == 1
    for at in (a, a + n - 4, a - TREE_WRITES["lse"] + 4):
        assert _tree(lib, lse=at) == 1


def test_tree_attention_refuses_outputs_over_one_another(lib):
    for at in (TREE["out"], TREE["out"] + TREE_WRITES["out"] - 4, TREE["out"] - TREE_WRITES["lse"] + 4):
        assert _tree(lib, lse=at) == 1


def test_tree_attention_refuses_a_workspace_over_anything(lib):
    need = A.fwd_tree_paged_workspace_bytes(BT, HQ, HKV, 128, 5)
    for name in list(TREE_READS) + list(TREE_WRITES):
        for at in (0, need // 2 // 256 * 256, (need - 1) // 256 * 256):
            assert _tree(lib, **{name: TREE["ws"] + at}) == 1
