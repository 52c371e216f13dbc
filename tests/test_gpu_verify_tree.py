"""Verification of drafted tokens (verify_tree) against the walk in 64 bits, one step at a time.

Nodes and tokens have to be equal.  A decision u q(x) < p(x), or between the two best tokens of a race, could only differ
where the two sides lie within the rounding of 32-bit probabilities (about 2^-20 of each other), which no seed here meets.
"""
import math

import pytest
import torch

import exact_attention_forward_06_gb300 as A
from tree_ref import make_tree, verify

import random

pytestmark = pytest.mark.gpu


def make(seed, sizes, V, kind, dtype=torch.bfloat16, temps=None, tree="tree", sharp=3.0):
    """Inputs of one call (CPU): kind 'greedy', 'top' (chosen tokens) or 'draft' (drawn ones)."""
    rng = random.Random(seed)
    gen = torch.Generator().manual_seed(seed)
    B, T = len(sizes), sum(sizes)
    trees = [make_tree(rng, n, tree) for n in sizes]
    parents = torch.tensor(sum(trees, []), dtype=torch.int32)
    cu = torch.tensor([0] + sizes).cumsum(0).to(torch.int32)
    base = torch.randn(max(T, 1), V, generator=gen) * sharp
    other = base + torch.randn(max(T, 1), V, generator=gen)
    logits, draft = base.to(dtype), other.to(dtype)
    tokens = torch.zeros(max(T, 1), dtype=torch.int32)
    for b, tree_b in enumerate(trees):
        seen = {}
        for i, up in enumerate(tree_b):
            if up < 0:
                tokens[int(cu[b]) + i] = rng.randrange(V)
                continue
            row = other[int(cu[b]) + up].to(dtype).float()
            if kind == "draft":
                x = int(torch.multinomial(torch.softmax(row, -1), 1, generator=gen))
            else:
                r = seen.get(up, 0)
                x = int(row.argsort(descending=True)[min(r, V - 1)])
                seen[up] = r + 1
            tokens[int(cu[b]) + i] = x
    d = dict(logits=logits, tokens=tokens, parents=parents, cu=cu, draft=None, temperature=None, uniforms=None, noise=None)
    if kind != "greedy":
        d["temperature"] = torch.tensor([(temps or [1.0])[b % len(temps or [1.0])] for b in range(B)])
        d["uniforms"] = torch.rand(max(T, 1), generator=gen)
        d["noise"] = torch.empty(B, V).exponential_(generator=gen)
        if kind == "draft":
            d["draft"] = draft
    d["width"] = max(1, max(sizes))
    return d


def call(d, **kw):
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    kw.setdefault("max_seqlen", d["width"])
    return A.verify_tree(dev["logits"], dev["tokens"], dev["parents"], dev["cu"], draft_logits=dev["draft"],
                         temperature=dev["temperature"], uniforms=dev["uniforms"], noise=dev["noise"], **kw)


def want(d):
    return verify(d["logits"], d["tokens"], d["parents"], d["cu"], d["draft"], d["temperature"], d["uniforms"], d["noise"],
                  d["width"])


def check(d, got=None, status=(0, 0)):
    got = call(d) if got is None else got
    for g, w, name in zip(got, want(d), ("path", "tokens", "counts")):
        assert torch.equal(g.cpu(), w), (name, g.cpu(), w)
    assert A.device_status()[0] == status[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["greedy", "top", "draft"])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 1000, 4097, 12345])
def test_sizes(V, kind, dtype):
    sizes = [1, 9, 4, 0, 23] if V < 4000 else [5, 12]
    check(make(1000 + V, sizes, V, kind, dtype, temps=[1.0, 0.6, 1.4]))


@pytest.mark.parametrize("kind", ["greedy", "top", "draft"])
@pytest.mark.parametrize("tree", ["chain", "bush", "roots"])
def test_trees(tree, kind):
    check(make(20, [14, 3, 40], 200, kind, tree=tree, temps=[1.0, 0.0, 0.8], sharp=1.0))


def test_many_sequences_of_mixed_temperatures():
    for seed, kind in ((31, "top"), (32, "draft")):
        check(make(seed, [i % 6 for i in range(90)], 77, kind, temps=[1.0, 0.0, 0.5, -1.0, 2.0, math.nan], sharp=1.5))


def test_largest_tree():
    check(make(33, [256, 256], 50, "draft", tree="chain", sharp=0.3))
    check(make(34, [256], 300, "top", tree="bush", sharp=0.1))
    check(make(35, [256], 300, "draft", tree="bush", sharp=4.0))     # a sum for every sibling that is rejected
    check(make(36, [16, 9], 9000, "draft", tree="bush", sharp=4.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["greedy", "top", "draft"])
def test_strided_and_unaligned_rows(kind, dtype):
    d = make(40, [7, 12], 4611, kind, dtype)
    ref = want(d)
    for pad, off in ((13, 1), (5, 3), (8, 0)):
        wide = {}
        for name in ("logits", "draft", "noise"):
            if d[name] is None:
                wide[name] = None
                continue
            x = torch.full((d[name].shape[0], 4611 + pad), math.nan, dtype=d[name].dtype, device="cuda")
            x[:, off:off + 4611] = d[name].cuda()
            wide[name] = x[:, off:off + 4611]
        got = call({**d, **wide})
        for g, w in zip(got, ref):
            assert torch.equal(g.cpu(), w)


def test_masked_logits():
    """-inf leaves a token out, NaN counts as -inf, +inf as the largest number there is."""
    for seed, kind in ((50, "greedy"), (51, "top"), (52, "draft")):
        d = make(seed, [6, 11, 5, 3], 333, kind, sharp=2.0)
        gen = torch.Generator().manual_seed(seed)
        for name in ("logits", "draft"):
            if d[name] is not None:
                hide = torch.rand(d[name].shape, generator=gen)
                d[name][hide < 0.5] = -math.inf
                d[name][hide > 0.9] = math.nan
        d["logits"][0, 17] = math.inf
        d["logits"][0, 200] = math.inf
        d["logits"][6] = -math.inf           # the second sequence's root: no token left
        d["logits"][17] = math.nan           # the third's
        d["logits"][22] = torch.finfo(torch.bfloat16).min
        check(d)


def test_largest_logits_tie_to_the_lowest_index():
    d = make(60, [4, 4], 9000, "greedy", tree="chain")
    d["logits"][:] = 1.0
    d["logits"][0, [8191, 4100, 77]] = 5.0
    d["tokens"][1] = 77
    d["logits"][1, [8999, 4096]] = 5.0
    d["tokens"][2] = 8999
    check(d)


def test_race_ties_to_the_lowest_index():
    d = make(61, [1, 1], 9000, "top", tree="chain")
    d["logits"][:] = 0.0
    d["noise"][:] = 2.0
    d["noise"][0, [8500, 4300]] = 0.5
    got = call(d)
    assert got[1].flatten().tolist() == [4300, 0]


def test_noise_that_is_not_positive_is_never_drawn():
    d = make(62, [1, 1, 1], 40, "top")
    d["logits"][:] = 0.0
    d["noise"][0, :39] = -1.0
    d["noise"][1, 1:] = math.nan
    d["noise"][2, :] = -3.0
    assert call(d)[1].flatten().tolist() == [39, 0, -1]
    assert A.device_status()[0] == 0


@pytest.mark.parametrize("bad", [0.0, -0.0, -1e-3, -math.inf])
def test_noise_that_is_not_positive_where_a_drawn_child_was_rejected(bad):
    # p: three quarters on token 4; q: on token 7, which is rejected and has p - q below 0
    d = make(65, [2, 1], 16, "draft", tree="chain")
    d["logits"][:] = 0.0
    d["draft"][:] = 0.0
    d["logits"][0, 4] = d["draft"][0, 7] = math.log(45.0)
    d["tokens"][1] = 7
    d["uniforms"][1] = 0.5
    d["noise"][:] = bad
    d["noise"][0, 4] = 1.0
    d["noise"][1, 11] = 1.0
    path, tokens, counts = call(d)
    assert counts.tolist() == [1, 1] and tokens[:, 0].tolist() == [4, 11]
    d["noise"][:] = bad
    assert call(d)[1][:, 0].tolist() == [-1, -1]


@pytest.mark.parametrize("V", [24569, 24576, 24577, 49145, 49152, 49153, 50001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_siblings_drawn_from_one_row_in_long_slices(V, dtype):
    # so many sequences that each has one CTA or two, whose slices are as long as shared memory keeps, or longer
    sizes = [0] * 80
    sizes[3], sizes[41], sizes[79] = 9, 17, 6
    d = make(90 + V % 7, sizes, V, "draft", dtype=dtype, tree="bush", sharp=2.0)
    d["uniforms"][:] = 0.5 + d["uniforms"] / 2
    check(d)
    # with rows that begin anywhere, and numbers that are not plain
    d["logits"][9, ::3] = math.nan
    d["draft"][9, ::2] = -math.inf
    d["logits"][0, 5] = math.inf
    check(d)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tree", ["tree", "bush"])
@pytest.mark.parametrize("kind", ["greedy", "top", "draft"])
def test_large_trees_of_long_rows(kind, tree, dtype):
    # more rows, and more bytes, than are summed up ahead: the walk sums up the rows that it comes to
    d = make(98, [70, 3, 65], 131077, kind, dtype, tree=tree, temps=[1.0, 0.0, 0.7], sharp=8.0)
    check(d)
    gen = torch.Generator().manual_seed(99)
    for name in ("logits", "draft"):
        if d[name] is not None:
            d[name][:, 7::3] = -math.inf
            d[name][torch.randint(138, (40,), generator=gen), torch.randint(131077, (40,), generator=gen)] = math.nan
    d["logits"][73, 99] = math.inf
    check(d)


def test_large_drawn_trees_in_long_slices():
    sizes = [0] * 80
    for b in (0, 8, 30, 31, 70, 79):
        sizes[b] = 220
    d = make(97, sizes, 73729, "draft", sharp=2.0)
    d["uniforms"][:] = 0.5 + d["uniforms"] / 2
    check(d)


def test_equal_siblings_and_nothing_left():
    # the only two tokens are both children, and rejected although they have all the mass
    d = make(63, [4], 8, "top", tree="bush")
    d["logits"][:] = -math.inf
    d["logits"][0, 2] = d["logits"][0, 5] = 0.0
    d["tokens"][1:] = torch.tensor([2, 2, 5])
    d["uniforms"][:] = torch.tensor([0.0, 0.75, 0.0, 1.5])
    path, tokens, counts = call(d)
    # 2 is rejected, 2 again has nothing left, 5 is rejected only by a number that is not below 1: then of all tokens
    race = 1.0 / d["noise"][0]
    assert counts.tolist() == [1] and tokens[0, 0] == (2 if race[2] >= race[5] else 5)
    d["uniforms"][3] = 0.999
    assert call(d)[0][0, :2].tolist() == [0, 3]


def test_draft_that_equals_the_target_is_accepted():
    d = make(64, [9, 9, 9], 5000, "draft", tree="chain")
    d["draft"] = d["logits"].clone()
    d["uniforms"][:] = 1.0 - 2.0 ** -24
    path, tokens, counts = call(d)
    ref = want(d)
    assert torch.equal(counts.cpu(), ref[2]) or counts.min() >= 1
    d["uniforms"][:] = 0.99
    assert call(d)[2].tolist() == [9, 9, 9]


def test_bad_entries_are_reported():
    d = make(70, [5, 8, 3], 100, "top", sharp=1.0)
    ref = call(d)
    cu = d["cu"].clone()
    d["cu"] = torch.tensor([0, 5, 20, 16], dtype=torch.int32)
    got = call(d)
    assert A.device_status() == (6, 29)
    assert got[2].tolist()[1:] == [0, 0] and (got[0][1:] == -1).all() and (got[1][1:] == -1).all()
    assert all(torch.equal(g[0], r[0]) for g, r in zip(got, ref))
    d["cu"] = cu
    got = call(d, max_seqlen=6)       # the second tree is larger than that
    assert A.device_status() == (6, 29) and got[2][1] == 0
    for tok in (-1, 100, 2 ** 31 - 1):
        e = {**d, "tokens": d["tokens"].clone()}
        e["tokens"][7] = tok
        check(e, status=(6, 30))
    for i, up in ((7, 3), (7, 200), (9, -5)):
        e = {**d, "parents": d["parents"].clone()}
        e["parents"][i] = up
        got = call(e)
        assert A.device_status() == (6, 28)
        e["parents"][i] = -1
        check(e, got)


def test_outputs_given_captured_and_on_another_stream():
    d = make(80, [9, 4, 6], 6000, "draft")
    ref = want(d)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    path, tokens = (torch.full((3, 9), 5, dtype=torch.int32, device="cuda") for _ in range(2))
    counts = torch.zeros(3, dtype=torch.int32, device="cuda")

    def run(**kw):
        return A.verify_tree(dev["logits"], dev["tokens"], dev["parents"], dev["cu"], draft_logits=dev["draft"],
                             temperature=dev["temperature"], uniforms=dev["uniforms"], noise=dev["noise"], max_seqlen=9,
                             path=path, out_tokens=tokens, counts=counts, **kw)

    got = run()
    assert got[0] is path and got[1] is tokens and got[2] is counts
    check(d, got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in (81, 82):
        e = make(seed, [9, 4, 6], 6000, "draft")
        for name in ("logits", "draft", "tokens", "parents", "uniforms", "noise"):
            dev[name].copy_(e[name])
        g.replay()
        check(e, got)
    for name in ("logits", "draft", "tokens", "parents", "uniforms", "noise"):
        dev[name].copy_(d[name])
    path.zero_()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    run(stream=s)
    s.synchronize()
    for x, w in zip(got, ref):
        assert torch.equal(x.cpu(), w)


@pytest.mark.parametrize("kind", ["top", "draft"])
def test_first_token_is_distributed_as_the_target(kind):
    """Whatever is drafted: 40000 steps of one distribution, three siblings each, within five standard deviations."""
    B, V, n = 40000, 6, 4
    gen = torch.Generator(device="cuda").manual_seed(90)
    p = torch.tensor([0.4, 0.25, 0.15, 0.12, 0.05, 0.03], device="cuda")
    q = torch.tensor([0.1, 0.1, 0.5, 0.1, 0.1, 0.1], device="cuda")
    logits = p.log().repeat(B * n, 1).contiguous()
    parents = torch.tensor([-1, 0, 0, 0] * B, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    if kind == "draft":
        tokens = torch.multinomial(q, B * n, replacement=True, generator=gen).to(torch.int32)
        draft = q.log().repeat(B * n, 1).contiguous()
    else:
        tokens, draft = torch.tensor([0, 2, 0, 5] * B, dtype=torch.int32, device="cuda"), None
    _, out, counts = A.verify_tree(logits, tokens, parents, cu, draft_logits=draft, temperature=torch.ones(B, device="cuda"),
                                   uniforms=torch.rand(B * n, generator=gen, device="cuda"),
                                   noise=torch.empty(B, V, device="cuda").exponential_(generator=gen), max_seqlen=n)
    first = out[:, 0].long()
    share = torch.bincount(first, minlength=V).double() / B
    sigma = (p * (1 - p) / B).sqrt().double()
    assert ((share - p.double()).abs() <= 5 * sigma).all(), share
    # and the second one, where a token was accepted, as well: its row is the same distribution
    more = counts > 1
    share = torch.bincount(out[more, 1].long(), minlength=V).double() / int(more.sum())
    assert ((share - p.double()).abs() <= 5 * (p * (1 - p) / int(more.sum())).sqrt().double()).all(), share


def test_rows_past_32_bit_offsets():
    d = make(100, [6, 9], 1000, "draft")
    stride = (1 << 28) + 24
    ref = want(d)
    wide = {}
    for name in ("logits", "draft"):
        big = torch.empty(14 * stride + 1000, dtype=torch.bfloat16, device="cuda")
        view = big.as_strided((15, 1000), (stride, 1))
        view.copy_(d[name])
        wide[name] = view
    got = call({**d, **wide})
    for g, w in zip(got, ref):
        assert torch.equal(g.cpu(), w)
    del wide, view, big
    torch.cuda.empty_cache()


def test_more_sequences_than_sms():
    check(make(101, [1 + i % 3 for i in range(400)], 5000, "draft", tree="chain", temps=[1.0, 0.0, 0.7]))


@pytest.mark.parametrize("kind", ["greedy", "top", "draft"])
def test_short_and_long_trees_alike(kind):
    """Rows summed up ahead (few a sequence, or few bytes) or one by one: the same sequences alone and beside a long tree."""
    d = make(102, [12, 200, 3], 90001, kind, tree="chain" if kind == "greedy" else "tree", temps=[1.0, 0.8])
    whole = call(d)
    check(d, whole)
    for b in (0, 2):
        rows = slice(int(d["cu"][b]), int(d["cu"][b + 1]))
        one = {k: (v[rows] if k in ("logits", "draft", "tokens", "parents", "uniforms") else
                   v[b:b + 1] if k in ("temperature", "noise") else v) if v is not None and k != "width" else v
               for k, v in d.items()}
        n = rows.stop - rows.start
        one["cu"] = torch.tensor([0, n], dtype=torch.int32)
        got = call(one, max_seqlen=n)
        for g, w in zip(got, whole):
            assert torch.equal(g[0], w[b, :n] if w.dim() == 2 else w[b])


def test_calls_at_the_same_time_with_a_workspace_each():
    cases = [make(110 + i, [5, 9, 3], 9000, "draft") for i in range(2)]
    refs = [want(d) for d in cases]
    dev = [{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()} for d in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(A.verify_tree(dev[i]["logits"], dev[i]["tokens"], dev[i]["parents"], dev[i]["cu"],
                                            draft_logits=dev[i]["draft"], temperature=dev[i]["temperature"],
                                            uniforms=dev[i]["uniforms"], noise=dev[i]["noise"], max_seqlen=9))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x.cpu(), w) for x, w in zip(g, refs[i]))


@pytest.mark.parametrize("kind", ["greedy", "top", "draft"])
def test_one_long_tree_among_short_ones(kind):
    """Few rows a sequence on average, so all are summed up ahead, the long tree's one after another."""
    check(make(120, [3, 1, 150, 2, 4, 1, 5, 2, 0, 1, 3, 2], 700, kind, temps=[1.0, 0.8, 0.0 if kind == "greedy" else 1.2]))
