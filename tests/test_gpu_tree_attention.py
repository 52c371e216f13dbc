"""Attention of trees of drafted tokens over the paged cache (fwd_tree_paged) against the definition in 64 bits.

Bounds.  Keys, values and queries are bf16 and exact.  Each probability goes into the P V product rounded to bf16 (2^-8
of itself), so the output is off by at most 2^-8 sum p |v| before its own rounding (2^-8 of itself).  All else is fp32:
a score's dot product of 128 terms is off by at most 128 * 2^-24 * sum |q k| * scale, below 1e-4 here (sum |q k| * scale
stays below 13 for these inputs), which moves a probability by less than 1e-4 of itself and the log-sum-exp by as much.
"""
import math

import pytest
import torch

import exact_attention_forward_06_gb300 as A
from tree_ref import Batch, ancestors

pytestmark = pytest.mark.gpu


def call(b, **kw):
    dev = "cuda"
    kw.setdefault("max_seqlen_q", max(1, max(b.sizes)))
    return A.fwd_tree_paged(b.q.to(dev), b.k.to(dev), b.v.to(dev), b.table.to(dev), b.lens.to(dev), b.cu.to(dev),
                            b.parents.to(dev), **kw)


def check(b, got, scale=None):
    out, lse = got
    ref, ref_lse, mass = b.attention(scale)
    out, lse = out.double().cpu(), lse.double().cpu()
    bound = (2.0 ** -8 + 2e-4) * mass + 2.0 ** -8 * ref.abs() + 1e-30
    assert ((out - ref).abs() <= bound).all(), float(((out - ref).abs() / bound).max())
    off = (lse - ref_lse).abs()
    assert (off <= 2e-4).all(), float(off.max())
    assert A.device_status()[0] == 0


SHAPES = [
    # sizes, contexts, Hq, Hkv, kind
    ([1], [0], 8, 2, "chain"),
    ([1], [1], 1, 1, "chain"),
    ([5], [200], 32, 8, "chain"),
    ([33], [95], 8, 2, "tree"),                     # ends with the first tile
    ([33], [96], 8, 2, "tree"),                     # one key into the second
    ([64], [1000], 32, 8, "tree"),
    ([64], [130], 64, 8, "bush"),                   # two tiles of eight heads each, several row blocks
    ([17, 1, 40, 3], [0, 300, 77, 15], 20, 4, "tree"),       # five heads: tiles of 125 rows
    ([7, 0, 9], [500, 33, 0], 12, 4, "tree"),       # an idle sequence among them
    ([19], [40], 6, 1, "roots"),
    ([3, 50], [128, 256], 7, 1, "tree"),            # seven heads
    ([9], [64], 32, 1, "tree"),                     # four positions a tile
    ([6], [200], 128, 1, "tree"),                   # one position a tile
    ([256], [100], 4, 2, "tree"),                   # the largest tree, over three tiles
    ([256], [383], 3, 3, "chain"),
    ([129, 200], [1, 127], 8, 4, ["bush", "tree"]),
    ([2] * 40, list(range(0, 400, 10)), 4, 1, "chain"),
    ([5, 31, 12], [3000, 2500, 9], 16, 2, "tree"),  # cut over many CTAs
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_shapes(i):
    sizes, ctx, Hq, Hkv, kind = SHAPES[i]
    b = Batch(100 + i, sizes, ctx, Hq, Hkv, kind)
    check(b, call(b))


def test_long_context_one_head():
    b = Batch(7, [11, 4], [40000, 33333], 8, 1)
    check(b, call(b))


def test_consecutive_pages():
    b = Batch(8, [20, 30], [700, 900], 8, 2, consecutive=True)
    check(b, call(b))


def test_more_sequences_than_a_warp():
    b = Batch(9, [(i % 4) for i in range(75)], [(i * 37) % 200 + 1 for i in range(75)], 4, 2)
    check(b, call(b))


@pytest.mark.parametrize("scale", [0.0, 0.5])
def test_scale(scale):
    b = Batch(10, [21], [300], 8, 2)
    b.q = (b.q.float() * 0.1).to(torch.bfloat16)
    check(b, call(b, scale=scale), scale)


def test_chain_is_the_causal_chunk():
    b = Batch(11, [30, 9], [450, 128], 32, 8, "chain")
    dev = "cuda"
    got = call(b)
    want = A.fwd_paged(b.q.to(dev), b.k.to(dev), b.v.to(dev), b.table.to(dev), b.lens.to(dev), b.cu.to(dev),
                       max_seqlen_q=30, causal=True)
    _, _, mass = b.attention()
    diff = (got[0].double() - want[0].double()).abs().cpu()
    assert (diff <= (2 * 2.0 ** -8 + 4e-4) * mass + 2 * 2.0 ** -8 * want[0].double().abs().cpu()).all()


def test_single_token_is_the_decode():
    b = Batch(12, [1, 1, 1], [450, 128, 0], 32, 8, "chain")
    dev = "cuda"
    out, lse = call(b)
    ref, ref_lse = A.decode_paged(b.q.to(dev), b.k.to(dev), b.v.to(dev), b.table.to(dev), b.lens.to(dev))
    _, _, mass = b.attention()
    assert ((out.double() - ref.double()).abs().cpu() <= (2.0 ** -7 + 4e-4) * mass + 2.0 ** -7 * ref.double().abs().cpu()).all()
    assert (lse.t() - ref_lse).abs().max() <= 4e-4


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_hidden_keys_may_hold_anything(bad, which):
    """A token is only touched by keys that it sees: a branch's NaN or infinity stays in the branch."""
    b = Batch(13, [60, 25], [150, 700], 8, 2)
    clean = call(b)
    hurt = 9
    for seq in (0, 1):
        t = b.lens_list[seq] - b.sizes[seq] + hurt
        page, slot = int(b.table[seq, t // 16]), t % 16
        if which != "v":
            b.k[page, slot, :, 5] = bad
        if which != "k":
            b.v[page, slot, 1, 3] = bad
            b.v[page, slot, 0, 127] = bad
    out, lse = call(b)
    for seq in (0, 1):
        for i, _ in enumerate(b.trees[seq]):
            t = int(b.cu[seq]) + i
            sees = hurt in ancestors(b.trees[seq], i)
            same = torch.equal(out[t], clean[0][t]) and torch.equal(lse[:, t], clean[1][:, t])
            if not sees:
                assert same, (seq, i)
            elif which == "v":
                assert torch.equal(lse[:, t], clean[1][:, t])
                o = out[t].float().cpu()
                want = torch.zeros(8, 128, dtype=torch.bool)
                want[:4, 127] = True
                want[4:, 3] = True
                assert ((~o.isfinite()) == want).all(), (seq, i)
                if bad != bad:
                    assert o[want].isnan().all()
                else:
                    assert (o[want] == bad).all()
                # what is taken out of the product and added one key at a time is not rounded to bf16 on the way
                ok = ~want
                assert (o[ok] - clean[0][t].float().cpu()[ok]).abs().max() <= 2.0 ** -6
            else:
                assert not same
    assert A.device_status()[0] == 0


def test_seen_nan_scores_give_nan():
    b = Batch(14, [4], [600], 8, 2, "chain")
    page = int(b.table[0, 3])
    b.k[page, 2, :, 0] = math.nan
    out, lse = call(b)
    assert out.isnan().all() and lse.isnan().all()


def test_rows_of_no_sequence_stay():
    b = Batch(15, [6, 11], [40, 90], 8, 2)
    dev = "cuda"
    q = torch.cat([b.q, b.q[:5]])
    out = torch.full_like(q, 7.0, device=dev)
    lse = torch.full((8, q.shape[0]), 3.0, device=dev)
    parents = torch.cat([b.parents, torch.zeros(5, dtype=torch.int32)]).to(dev)
    A.fwd_tree_paged(q.to(dev), b.k.to(dev), b.v.to(dev), b.table.to(dev), b.lens.to(dev), b.cu.to(dev), parents,
                     max_seqlen_q=11, out=out, lse=lse)
    check(b, (out[:17], lse[:, :17]))
    assert (out[17:] == 7).all() and (lse[:, 17:] == 3).all()


def test_no_lse_and_roundings():
    b = Batch(16, [12, 30], [2000, 100], 8, 2)
    out, lse = call(b, lse=False)
    assert lse is None
    ref = call(b)[0]
    assert torch.equal(out, ref)
    zero = call(b, rounding="rtz")[0]
    assert (zero.float().abs() <= ref.float().abs() + 0).all()
    away = call(b, rounding="rtna")[0]
    assert ((away.float() - ref.float()).abs() <= 2.0 ** -7 * ref.float().abs()).all()


def test_deterministic_whatever_the_workspace_holds():
    b = Batch(17, [40, 40, 40], [900, 5000, 70], 32, 8)
    need = A.fwd_tree_paged_workspace_bytes(3, 32, 8, 128, 40)
    one = call(b, workspace=torch.full((need,), 0xff, dtype=torch.uint8, device="cuda"))
    two = call(b, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_bad_entries_are_reported_and_skipped():
    b = Batch(18, [6, 11, 8], [40, 90, 700], 8, 2)
    out = torch.full(b.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    # a cache shorter than its tree, and one longer than its table
    for length in (10, b.table.shape[1] * 16 + 1, -1):
        lens = b.lens.clone()
        lens[1] = length
        keep = b.lens
        b.lens = lens
        got, lse = call(b, out=out.clone())
        b.lens = keep
        assert A.device_status() == (6, 27)
        assert (got[6:17] == 7).all()
        ref = call(b)[0]
        assert torch.equal(got[:6], ref[:6]) and torch.equal(got[17:], ref[17:])
    # a tree larger than max_seqlen_q
    got, _ = call(b, max_seqlen_q=8, out=out.clone())
    assert A.device_status() == (6, 27) and (got[6:17] == 7).all()
    # a parent at or behind its child counts as none
    good = b.parents.clone()
    for i, p in ((3, 3), (4, 200), (5, -2)):
        b.parents = good.clone()
        b.parents[i] = p
        got = call(b)
        assert A.device_status() == (6, 28)
        b.parents[i] = -1
        kept = b.trees[0]
        b.trees[0] = b.parents[:6].tolist()
        check(b, got)
        b.trees[0] = kept
    b.parents = good
    # a page outside the pool reads as zeros
    b.table[2, 1] = b.k.shape[0]
    got = call(b)
    assert A.device_status() == (6, 13)
    check(b, got)


def test_captured_and_replayed():
    b = Batch(19, [16, 16], [1500, 300], 32, 8)
    dev = "cuda"
    args = [x.to(dev) for x in (b.q, b.k, b.v, b.table, b.lens, b.cu, b.parents)]
    ws = torch.empty(A.fwd_tree_paged_workspace_bytes(2, 32, 8, 128, 16), dtype=torch.uint8, device=dev)
    out, lse = A.fwd_tree_paged(*args, max_seqlen_q=16, workspace=ws)
    want = out.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.fwd_tree_paged(*args, max_seqlen_q=16, workspace=ws, out=out, lse=lse)
    for _ in range(3):
        out.zero_(), lse.zero_()
        g.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # other lengths and another tree in the same buffers
    c = Batch(20, [16, 16], [200, 1400], 32, 8)
    w = args[3].shape[1]
    c.table = (torch.arange(2 * w).view(2, w) % b.k.shape[0]).to(torch.int32)
    c.k, c.v = (x.nan_to_num(0.5) for x in (b.k, b.v))
    for i, x in ((0, c.q), (1, c.k), (2, c.v), (3, c.table), (4, c.lens), (6, c.parents)):
        args[i].copy_(x)
    g.replay()
    check(c, (out, lse))


def test_another_stream():
    b = Batch(21, [30, 2], [800, 50], 16, 4)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(b, stream=s)
    s.synchronize()
    check(b, got)
    with torch.cuda.stream(s):
        got = call(b)
    s.synchronize()
    check(b, got)


def test_pool_past_32_bit_offsets():
    """The same batch with its pages at the end of a pool of more than 2^32 elements, a key with infinite values too."""
    b = Batch(30, [30, 64], [400, 1500], 16, 8)
    t = b.lens_list[0] - 5
    b.v[int(b.table[0, t // 16]), t % 16, 3, 7] = math.inf
    want = call(b)
    few, pages = b.k.shape[0], (1 << 18) + b.k.shape[0]
    dev = []
    for pool in (b.k, b.v):
        big = torch.empty((pages, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
        big[-few:] = pool.cuda()
        dev.append(big)
    table = torch.where(b.table >= 0, b.table + (pages - few), b.table).cuda()
    got = A.fwd_tree_paged(b.q.cuda(), *dev, table, b.lens.cuda(), b.cu.cuda(), b.parents.cuda(), max_seqlen_q=64)
    assert torch.equal(got[0].nan_to_num(9.0), want[0].nan_to_num(9.0)) and torch.equal(got[1], want[1])
    assert A.device_status()[0] == 0
    del dev, big
    torch.cuda.empty_cache()


def test_out_that_is_16_byte_aligned_only():
    b = Batch(31, [9, 5], [100, 700], 4, 2)
    want = call(b)
    flat = torch.empty(14 * 4 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    out = flat[8:].view(14, 4, 128)
    got = call(b, out=out)
    assert got[0] is out and torch.equal(out, want[0])


def test_calls_at_the_same_time_with_a_workspace_each():
    cases = [Batch(40 + i, [16, 40, 1], [900, 2000, 77], 16, 4) for i in range(2)]
    dev = [[x.cuda() for x in (b.q, b.k, b.v, b.table, b.lens, b.cu, b.parents)] for b in cases]
    want = [A.fwd_tree_paged(*d, max_seqlen_q=40) for d in dev]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(A.fwd_tree_paged(*dev[i], max_seqlen_q=40))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1]) for g in got[i])


def test_expired_wait_is_reported_and_the_next_call_is_right():
    """The load-issuing warps issue nothing: the other warps' bounded waits run out, nothing is left in flight."""
    b = Batch(50, [16, 40, 1], [900, 2000, 77], 16, 4)
    good = call(b)
    ws = torch.full((A.fwd_tree_paged_workspace_bytes(3, 16, 4, 128, 40),), 0x7f, dtype=torch.uint8, device="cuda")
    A.set_wait_budget_ns(20_000_000)          # 20 ms
    try:
        A.debug_inject(1)
        call(b, workspace=ws)
        code, site = A.device_status()
        assert code == 4 and site == 19, (code, site)   # a work item that never came
        assert A.device_status()[0] == 0
    finally:
        A.debug_inject(0)
        A.set_wait_budget_ns(0)
    again = call(b, workspace=ws)
    assert A.device_status()[0] == 0
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


def test_many_idle_rows_between_trees():
    sizes = [0] * 500
    ctx = [0] * 500
    for at, n, c in ((0, 4, 900), (130, 7, 3000), (131, 1, 20), (499, 12, 700)):
        sizes[at], ctx[at] = n, c
    b = Batch(60, sizes, ctx, 8, 2)
    check(b, call(b, max_seqlen_q=200))


def test_bound_far_above_the_trees():
    b = Batch(61, [3, 9, 5], [2000, 777, 130], 32, 8)
    want = call(b)
    got = call(b, max_seqlen_q=256)
    check(b, got)
    _, _, mass = b.attention()
    assert ((got[0].double() - want[0].double()).abs().cpu() <= (2.0 ** -7 + 4e-4) * mass + 2.0 ** -7 * want[0].double().abs().cpu()).all()
