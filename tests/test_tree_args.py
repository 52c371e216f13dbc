"""Refusals of the operators around a tree of drafted tokens, before any launch (CPU): the C ABI's argument checks, the
workspace's size, and the binding's checks."""
import pytest
import torch

import exact_attention_forward_06_gb300 as A
from exact_attention_forward_06_gb300 import _binding


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_binding.LIBRARY_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return A.load()


TREE = dict(q=256, k=512, v=1024, bt=4, sl=8, cu=12, par=4, out=1 << 20, lse=4, B=2, Hq=8, Hkv=2, total=9, longest=16, d=128,
            page=16, npages=10, maxb=4, scale=0.1, mode=0, ws=256, wsb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(q=264), 1), (dict(k=None), 1), (dict(k=520), 1), (dict(v=None), 1), (dict(v=1032), 1),
    (dict(bt=None), 1), (dict(bt=6), 1), (dict(sl=None), 1), (dict(sl=7), 1), (dict(cu=None), 1), (dict(cu=2), 1),
    (dict(par=None), 1), (dict(par=6), 1), (dict(out=None), 1), (dict(out=2056), 1), (dict(out=256), 1), (dict(lse=6), 1), (dict(B=0), 1),
    (dict(out=240 + 9 * 8 * 256), 1), (dict(q=(1 << 20) + 16), 1), (dict(q=(1 << 20) - 16), 1),  # out over q
    (dict(B=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=9), 1), (dict(total=0), 1), (dict(longest=0), 1),
    (dict(longest=257), 1), (dict(d=64), 2), (dict(page=32), 2), (dict(npages=0), 1), (dict(npages=1 << 28), 1),
    (dict(maxb=0), 1), (dict(maxb=1 << 27), 1), (dict(maxb=(1 << 27) - 16, B=1 << 8), 1),
    (dict(Hq=258, Hkv=2), 2),                        # 129 query heads to a KV head
    (dict(B=1 << 26, Hq=1 << 4), 1),                 # rows of the merge past 2^31
    (dict(scale=float("nan")), 1), (dict(scale=-1.0), 1), (dict(mode=3), 1), (dict(mode=-1), 1), (dict(ws=None), 5),
    (dict(ws=272), 5), (dict(wsb=1000), 5),
])
def test_tree_attention_rejects_before_any_launch(lib, kw, code):
    a = dict(TREE, **kw)
    assert lib.attn_fwd_tree_paged(*a.values(), None) == code


def test_tree_workspace_bytes(lib):
    need = A.fwd_tree_paged_workspace_bytes
    align = lambda x: (x + 255) // 256 * 256  # noqa: E731
    for B, Hq, Hkv, N, rows in ((1, 32, 8, 5, 20), (3, 32, 8, 64, 256), (7, 20, 4, 37, 128 + 12 * 5), (2, 32, 1, 61, 256),
                                (2, 128, 1, 1, 128), (5, 3, 3, 256, 256), (5, 7, 1, 20, 128 + 2 * 7)):
        parts = 152 * 2 * rows
        assert need(B, Hq, Hkv, 128, N) == align(4 * (B + 1)) + align(parts * 512) + align(parts * 4)
        a = dict(TREE, B=B, Hq=Hq, Hkv=Hkv, longest=N, wsb=need(B, Hq, Hkv, 128, N) - 1)
        assert lib.attn_fwd_tree_paged(*a.values(), None) == 5
    for bad in ((0, 8, 2, 128, 4), (1, 0, 2, 128, 4), (1, 8, 0, 128, 4), (1, 9, 2, 128, 4), (1, 8, 2, 64, 4),
                (1, 8, 2, 128, 0), (1, 8, 2, 128, 257), (1, 258, 2, 128, 4)):
        assert need(*bad) == 0


VERIFY = dict(logits=16, draft=32, dtype=0, tok=4, par=4, cu=4, temp=4, u=4, noise=4, path=4, out=4, counts=4, B=2, total=9,
              V=100, width=8, ls=100, ds=100, ns=100, ws=256, wsb=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), 1), (dict(logits=17), 1), (dict(dtype=1, logits=18), 1), (dict(draft=33), 1), (dict(dtype=2), 1),
    (dict(dtype=-1), 1), (dict(tok=None), 1), (dict(tok=2), 1), (dict(par=None), 1), (dict(cu=None), 1), (dict(cu=5), 1),
    (dict(temp=6), 1), (dict(temp=None), 1),         # random numbers and a draft without a temperature
    (dict(temp=None, u=None, noise=None), 1), (dict(temp=None, draft=None, u=None), 1), (dict(u=None), 1),
    (dict(noise=None), 1), (dict(noise=6), 1), (dict(path=None), 1), (dict(out=None), 1), (dict(counts=None), 1),
    (dict(counts=3), 1), (dict(B=0), 1), (dict(B=1 << 29), 1), (dict(total=0), 1), (dict(V=0), 1),
    (dict(V=(1 << 28) + 1, ls=1 << 31, ds=1 << 31, ns=1 << 31), 1), (dict(width=0), 1), (dict(width=257), 1),
    (dict(ls=99), 1), (dict(ds=99), 1), (dict(ns=99), 1), (dict(ls=1 << 41), 1), (dict(ds=1 << 41), 1),
    (dict(ns=1 << 41), 1), (dict(ws=None), 5), (dict(ws=260), 5), (dict(wsb=100), 5),
])
def test_verify_rejects_before_any_launch(lib, kw, code):
    assert lib.attn_verify_tree(*dict(VERIFY, **kw).values(), None) == code


COMPACT = dict(k=256, v=512, bt=4, sl=1024, cu=4, path=4, counts=2048, out=4096, B=2, layers=3, Hkv=2, total=9, width=8,
               d=128, page=16, npages=10, maxb=4)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(k=264), 1), (dict(v=None), 1), (dict(v=520), 1), (dict(bt=None), 1), (dict(sl=None), 1),
    (dict(cu=None), 1), (dict(path=None), 1), (dict(path=6), 1), (dict(counts=None), 1), (dict(out=None), 1),
    (dict(out=1024), 1), (dict(out=1028), 1), (dict(out=1020), 1), (dict(out=2052), 1),   # over the lengths or counts
    (dict(B=0), 1), (dict(layers=0), 1), (dict(Hkv=0), 1), (dict(total=0), 1), (dict(width=0), 1), (dict(width=257), 1),
    (dict(npages=0), 1), (dict(npages=1 << 27), 1), (dict(maxb=0), 1), (dict(maxb=1 << 27), 1), (dict(d=64), 2),
    (dict(page=8), 2), (dict(layers=1 << 20, Hkv=1 << 10), 1), (dict(B=1 << 24, layers=1 << 10), 1),
])
def test_compact_rejects_before_any_launch(lib, kw, code):
    assert lib.attn_compact_paged(*dict(COMPACT, **kw).values(), None) == code


def test_binding_rejects_cpu_tensors(lib):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(TypeError, match="q must be"):
        A.fwd_tree_paged(bf(4, 8, 128), bf(4, 16, 2, 128), bf(4, 16, 2, 128), i(1, 4), i(1), i(2), i(4), max_seqlen_q=4)
    with pytest.raises(ValueError, match="rounding"):
        A.fwd_tree_paged(bf(4, 8, 128), bf(4, 16, 2, 128), bf(4, 16, 2, 128), i(1, 4), i(1), i(2), i(4), rounding="up")
    with pytest.raises(TypeError, match="logits must be"):
        A.verify_tree(bf(4, 50), i(4), i(4), i(2), max_seqlen=4)
    with pytest.raises(TypeError, match="logits must be"):
        A.verify_tree([1.0], i(4), i(4), i(2))
    with pytest.raises(TypeError, match="k_pages must be"):
        A.compact_paged(bf(4, 16, 2, 128), bf(4, 16, 2, 128), i(1, 4), i(1), i(2), i(1, 4), i(1))


def test_verify_workspace_bytes(lib):
    need = A.verify_tree_workspace_bytes
    align = lambda x: (x + 255) // 256 * 256  # noqa: E731
    bf, fp = torch.bfloat16, torch.float32
    # up to 16 rows a sequence (and 64 MB, without draft), the rows' sums come first: slices of 4096 to 16384 tokens
    assert need(2, 9, 100, 8, bf) == align(2 * (64 + 32)) + 9 * 8
    assert need(64, 320, 131072, 5, bf, True) == align(64 * (64 + 20)) + 320 * 2 * 8 * 8
    assert need(1, 5, 32768, 5, fp) == align(64 + 20) + 5 * 8 * 8
    assert need(4, 65, 131072, 40, bf) == align(4 * (64 + 160))
    assert need(1, 16, 1 << 28, 16, bf, True) == align(64 + 64) + 16 * 2 * 64 * 8
    assert need(1, 16, 1 << 28, 16, bf) == align(64 + 64)
    for bad in ((0, 9, 100, 8), (2, 0, 100, 8), (2, 9, 0, 8), (2, 9, (1 << 28) + 1, 8), (2, 9, 100, 0), (2, 9, 100, 257)):
        assert need(*bad) == 0
    assert lib.attn_verify_tree_workspace_bytes(2, 9, 100, 8, 2, 0) == 0
    a = dict(VERIFY, wsb=need(2, 9, 100, 8, bf, True) - 1)
    assert lib.attn_verify_tree(*a.values(), None) == 5
