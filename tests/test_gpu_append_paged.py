"""GPU tests of the appends into the paged cache (attn_append_paged) and the
4-bit cache (attn_append_paged_q4): ragged chunks around the page edge, single
tokens, nothing new, strided inputs, every untouched byte, bad arguments on the
device, and the run of append and attention as a user makes it."""
import pytest
import torch

import cache_ref as R
import oracle
from parity_util import check_lse, check_out

pytestmark = pytest.mark.gpu
NEW = (1, 0, 16, 17, 3, 40, 0, 33)
CTX = (0, 5, 16, 15, 29, 100, 0, 7)


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_06_gb300 as attn
    attn.load()
    return attn


def _case(new, ctx, Hq, Hkv, seed, pad=0, max_blocks=None, spare=3):
    """Ragged new tokens on contexts; the pool has spare pages, the rows `pad` more tokens than sequences own."""
    g = torch.Generator().manual_seed(seed)
    lens = [n + c for n, c in zip(new, ctx)]
    pages = [(x + 15) // 16 for x in lens]
    P = sum(pages) + spare
    width = max_blocks or max(pages) + 1
    perm = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((len(new), width), -1, dtype=torch.int32)
    off = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[off:off + n]
        off += n
    total = sum(new) + pad
    qkv = torch.randn(total, (Hq + 2 * Hkv) * 128, generator=g).to(torch.bfloat16)
    q = qkv[:, :Hq * 128].unflatten(-1, (Hq, 128))
    k = qkv[:, Hq * 128:(Hq + Hkv) * 128].unflatten(-1, (Hkv, 128))
    v = qkv[:, (Hq + Hkv) * 128:].unflatten(-1, (Hkv, 128))
    kp, vp = (torch.randn(P, 16, Hkv, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
    return qkv, q, k, v, kp, vp, table, torch.tensor(lens, dtype=torch.int32), cu


def _slots(table, lens, cu):
    """(token, page, row, position) of every new token."""
    tok, page, row, pos = [], [], [], []
    for b in range(len(lens)):
        for i in range(int(cu[b]), int(cu[b + 1])):
            p = int(lens[b]) - int(cu[b + 1]) + i
            tok.append(i), page.append(int(table[b, p // 16])), row.append(p % 16), pos.append(p)
    return [torch.tensor(x, dtype=torch.long) for x in (tok, page, row, pos)]


def _split(dqkv, Hq, Hkv):
    return (dqkv[:, :Hq * 128].unflatten(-1, (Hq, 128)), dqkv[:, Hq * 128:(Hq + Hkv) * 128].unflatten(-1, (Hkv, 128)),
            dqkv[:, (Hq + Hkv) * 128:].unflatten(-1, (Hkv, 128)))


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16)


@pytest.mark.parametrize("inter,rdim,norm", [(False, 128, True), (True, 64, True), (False, 96, False), (True, 0, False)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 1), (5, 5), (32, 8)])
def test_appends_every_byte(A, Hq, Hkv, inter, rdim, norm):
    qkv, q, k, v, kp, vp, table, lens, cu = _case(NEW, CTX, Hq, Hkv, seed=Hq + rdim, pad=2)
    g = torch.Generator().manual_seed(1)
    wq, wk = ((torch.rand(128, generator=g) + 0.5).to(torch.bfloat16) if norm else None for _ in range(2))
    freq = R.inv_freq(rdim) if rdim else []
    kw = dict(rope=A.rope_table(freq) if rdim else None, q_weight=None if wq is None else wq.cuda(),
              k_weight=None if wk is None else wk.cuda(), interleaved=inter)
    tok, page, row, pos = _slots(table, lens, cu)
    dq, dk, dv = _split(qkv.cuda(), Hq, Hkv)
    dkp, dvp = kp.cuda(), vp.cuda()
    q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    r = A.append_paged(dq, dk, dv, dkp, dvp, table.cuda(), lens.cuda(), cu.cuda(), q_out=q_out, **kw)
    torch.cuda.synchronize()
    assert r is q_out and A.device_status()[0] == 0
    # q: against 64 bits; the rows behind the last sequence as they were
    ref = R.norm_rope(q[tok], wq, 1e-6, pos[None], freq, [0] * len(freq), inter)
    R.check_norm_rope(q_out.cpu()[tok], ref, "q")
    assert (q_out.cpu()[sum(NEW):] == 7.0).all()
    # k: the bits of qk_norm_rope at the slots, v its own bits, the rest untouched
    dpos = torch.zeros(q.shape[0], dtype=torch.int32)
    dpos[tok] = pos.to(torch.int32)
    kk = A.qk_norm_rope(dq, dk, positions=dpos.cuda(), **kw)[1].cpu()
    want_k, want_v = kp.clone(), vp.clone()
    want_k[page, row], want_v[page, row] = kk[tok], v[tok]
    assert torch.equal(_bits(dkp), _bits(want_k)) and torch.equal(_bits(dvp), _bits(want_v))
    # the 4-bit cache: the bytes of the quantised bf16 values, the rest untouched
    cache = torch.randint(0, 256, (kp.shape[0], Hkv, R.BLOCK), generator=g, dtype=torch.uint8)
    dcache = cache.cuda()
    q2 = A.append_paged_q4(dq, dk, dv, dcache, table.cuda(), lens.cuda(), cu.cuda(), **kw)
    torch.cuda.synchronize()
    assert A.device_status()[0] == 0 and torch.equal(q2.cpu()[tok], q_out.cpu()[tok])
    for h in range(Hkv):
        R.write_tokens(cache, page, row, torch.full_like(page, h), kk[tok, h], v[tok, h])
    assert torch.equal(dcache.cpu(), cache)


def test_single_tokens_without_offsets_and_without_q(A):
    new, ctx = (1,) * 9, (0, 1, 15, 16, 17, 31, 32, 500, 8)
    qkv, q, k, v, kp, vp, table, lens, cu = _case(new, ctx, 4, 4, seed=20)
    dq, dk, dv = _split(qkv.cuda(), 4, 4)
    rope = A.rope_table(R.inv_freq(128))
    pools = [(kp.cuda(), vp.cuda()) for _ in range(2)]
    A.append_paged(dq, dk, dv, *pools[0], table.cuda(), lens.cuda(), cu.cuda(), rope=rope)
    assert A.append_paged(None, dk, dv, *pools[1], table.cuda(), lens.cuda(), rope=rope) is None
    torch.cuda.synchronize()
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    assert not torch.equal(pools[0][0].cpu(), kp) and A.device_status()[0] == 0


def test_many_sequences_are_found(A):
    # more sequences than one round of the search's probes, empty ones between
    g = torch.Generator().manual_seed(3)
    new = [int(x) for x in torch.randint(0, 4, (700,), generator=g)]
    ctx = [int(x) for x in torch.randint(0, 20, (700,), generator=g)]
    qkv, q, k, v, kp, vp, table, lens, cu = _case(new, ctx, 1, 1, seed=21)
    tok, page, row, _ = _slots(table, lens, cu)
    dq, dk, dv = _split(qkv.cuda(), 1, 1)
    dkp, dvp = kp.cuda(), vp.cuda()
    A.append_paged(dq, dk, dv, dkp, dvp, table.cuda(), lens.cuda(), cu.cuda())
    torch.cuda.synchronize()
    want_k, want_v = kp.clone(), vp.clone()
    want_k[page, row], want_v[page, row] = k[tok], v[tok]
    assert torch.equal(_bits(dkp), _bits(want_k)) and torch.equal(_bits(dvp), _bits(want_v))
    assert A.device_status()[0] == 0


def test_positions_given_on_axes(A):
    new, ctx = (5, 20), (3, 0)
    qkv, q, k, v, kp, vp, table, lens, cu = _case(new, ctx, 2, 1, seed=22)
    tok, page, row, _ = _slots(table, lens, cu)
    freq, axes = R.inv_freq(128), [i % 3 for i in range(64)]
    pos = torch.randint(-100, 100000, (3, 25), dtype=torch.int32)
    dq, dk, dv = _split(qkv.cuda(), 2, 1)
    dkp, dvp = kp.cuda(), vp.cuda()
    q_out = A.append_paged(dq, dk, dv, dkp, dvp, table.cuda(), lens.cuda(), cu.cuda(),
                           rope=A.rope_table(freq, axes), positions=pos.cuda())
    torch.cuda.synchronize()
    R.check_norm_rope(q_out.cpu(), R.norm_rope(q, None, 0, pos, freq, axes, False), "q")
    R.check_norm_rope(dkp.cpu()[page, row], R.norm_rope(k, None, 0, pos, freq, axes, False), "k")


@pytest.mark.parametrize("group,code", [
    ([1.0] * 32, 0), ([0.0] * 32, 0), ([float("inf")] + [1.0] * 31, "nan"), ([1.0] * 31 + [float("nan")], "nan"),
    ([2.0 ** -126] * 16 + [-2.0 ** -126] * 16, None), ([1e38, -1e38] * 16, None), ([100.0 + i / 2 for i in range(32)], None),
    ([-float(i) for i in range(32)], None), ([1e-38, 1e-39] * 16, None)])
def test_quantisation_of_odd_groups(A, group, code):
    """Constant, zero, non-finite, subnormal, huge and offset groups: the definition's bytes, and what is read back."""
    x = torch.randn(1, 1, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[0, 0, 32:64] = torch.tensor(group, dtype=torch.float32).to(torch.bfloat16)
    cache = torch.zeros(1, 1, R.BLOCK, dtype=torch.uint8)
    one = torch.ones(1, dtype=torch.int32)
    table = torch.zeros(1, 1, dtype=torch.int32)
    d = cache.cuda()
    A.append_paged_q4(None, x.cuda(), x.cuda(), d, table.cuda(), one.cuda())
    z = torch.zeros(1, dtype=torch.long)
    R.write_tokens(cache, z, z, z, x[0], x[0])
    k, v = A.gather_paged_q4(d, table.cuda(), one.cuda(), torch.tensor([0, 1], dtype=torch.int32).cuda(), total_k=1)
    torch.cuda.synchronize()
    kp, vp = R.read_tokens(cache, table[0], 1)
    got = d.cpu()
    for name, parts, back in (("k", kp, k), ("v", vp, v)):
        g_parts = R.read_tokens(got, table[0], 1)[0 if name == "k" else 1]
        for a, b in zip(g_parts, parts):
            assert torch.equal(torch.nan_to_num(a, nan=-1.0), torch.nan_to_num(b, nan=-1.0)), name
        want = R.values_bf16(parts)
        assert torch.equal(torch.isnan(back.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(back.cpu()), torch.nan_to_num(want))
        if code == "nan":
            assert torch.isnan(back[0, 0, 32:64]).all() and not torch.isnan(back[0, 0, 64:]).any()
        if code == 0:
            assert torch.equal(back.cpu()[0, 0, 32:64], x[0, 0, 32:64])


def test_bad_device_arguments_are_reported_and_skipped(A):
    qkv, q, k, v, kp, vp, table, lens, cu = _case((3, 4, 5), (20, 30, 0), 2, 2, seed=23)
    dq, dk, dv = _split(qkv.cuda(), 2, 2)

    def run(table=table, lens=lens, cu=cu, q4=False):
        q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pools = [kp.cuda(), vp.cuda()]
        cache = torch.zeros(kp.shape[0], 2, R.BLOCK, dtype=torch.uint8, device="cuda")
        args = (table.cuda(), lens.cuda(), cu.cuda())
        if q4:
            A.append_paged_q4(dq, dk, dv, cache, *args, q_out=q_out)
        else:
            A.append_paged(dq, dk, dv, *pools, *args, q_out=q_out)
        code = A.device_status()[0]
        return code, q_out.cpu(), pools[0].cpu(), cache.cpu()

    for q4 in (False, True):
        assert run(q4=q4)[0] == 0
        bad = table.clone()
        bad[1, 30 // 16] = kp.shape[0]                         # tokens 30, 31 of sequence 1
        code, q_out, pool, cache = run(table=bad, q4=q4)
        assert code == 6 and not (q_out == 7.0).any()          # the queries are written all the same
        for short in (2, 16 * table.shape[1] + 1, -1):         # fewer keys than new ones; past the table; negative
            bad = lens.clone()
            bad[0] = short
            code, q_out, pool, cache = run(lens=bad, q4=q4)
            assert code == 6 and (q_out[:3] == 7.0).all() and not (q_out[3:] == 7.0).any()
        bad = cu.clone()
        bad[3] = 100                                           # past the rows
        assert run(cu=bad, q4=q4)[0] == 6
        bad = torch.tensor([0, 9, 4, 12], dtype=torch.int32)   # out of order
        code = run(cu=bad, q4=q4)[0]
        assert code in (0, 6)                                  # each token is placed or reported, never out of range
        A.device_status()
    # a sequence beginning behind row 0: the rows before it are nobody's
    shifted = torch.tensor([2, 5, 9, 12], dtype=torch.int32)
    code, q_out, _, _ = run(cu=shifted)
    assert code == 0 and (q_out[:2] == 7.0).all() and not (q_out[2:] == 7.0).any()


def test_append_then_attend_as_a_server_does(A):
    """Prompt chunks, then single tokens, into the paged cache, each with the attention that reads it."""
    Hq, Hkv, B = 8, 2, 3
    g = torch.Generator().manual_seed(30)
    freq = R.inv_freq(128)
    rope = A.rope_table(freq)
    w = (torch.rand(128, generator=g) + 0.5).to(torch.bfloat16)
    chunks = [(5, 40, 17), (30, 1, 16), (1, 1, 1), (1, 1, 1)]
    total = [sum(c[b] for c in chunks) for b in range(B)]
    width = max((t + 15) // 16 for t in total)
    table = torch.randperm(B * width, generator=g).to(torch.int32).reshape(B, width)
    kp, vp = (torch.full((B * width, 16, Hkv, 128), float("nan"), dtype=torch.bfloat16).cuda() for _ in range(2))
    done = torch.zeros(B, dtype=torch.int32)
    for c in chunks:
        done = done + torch.tensor(c, dtype=torch.int32)
        cu = torch.tensor((0,) + c).cumsum(0).to(torch.int32)
        qkv = torch.randn(sum(c), (Hq + 2 * Hkv) * 128, generator=g).to(torch.bfloat16).cuda()
        q, k, v = _split(qkv, Hq, Hkv)
        args = (table.cuda(), done.cuda())
        q_rot = A.append_paged(q, k, v, kp, vp, *args, cu.cuda(), rope=rope, q_weight=w.cuda(), k_weight=w.cuda())
        if max(c) > 1:
            out, lse = A.fwd_paged(q_rot, kp, vp, *args, cu.cuda(), max_seqlen_q=max(c))
            ref_o, ref_l = oracle.attention_paged(q_rot.cpu(), kp.cpu(), vp.cpu(), table, done, cu, Hq=Hq, Hkv=Hkv,
                                                  causal=True, scale=128 ** -0.5)
        else:
            out, lse = A.decode_paged(q_rot, kp, vp, *args)
            ref_o, ref_l = oracle.decode_paged(q_rot.cpu(), kp.cpu(), vp.cpu(), table, done, scale=128 ** -0.5)
        torch.cuda.synchronize()
        check_out(out, ref_o, f"chunk {c}")
        check_lse(lse, ref_l, f"chunk {c}")
    assert A.device_status()[0] == 0


def test_captured_appends_replay_with_new_lengths(A):
    """A captured decode step reads its lengths, table and inputs at each replay; two graphs share nothing."""
    qkv, q, k, v, kp, vp, table, lens, cu = _case((1,) * 4, (14, 15, 16, 100), 4, 2, seed=40, max_blocks=9)
    dqkv, dt, dl = qkv.cuda(), table.cuda(), lens.cuda()
    dq, dk, dv = _split(dqkv, 4, 2)
    rope = A.rope_table(R.inv_freq(128))
    kpc, vpc, q_out = kp.cuda(), vp.cuda(), torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        A.append_paged(dq, dk, dv, kpc, vpc, dt, dl, rope=rope, q_out=q_out, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        A.append_paged(dq, dk, dv, kpc, vpc, dt, dl, rope=rope, q_out=q_out, stream=s)
    dl -= 3
    dqkv.copy_(torch.randn(qkv.shape).to(torch.bfloat16))
    kpc.copy_(kp), vpc.copy_(vp)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    ke, ve = kp.cuda(), vp.cuda()
    qe = A.append_paged(dq, dk, dv, ke, ve, dt, dl, rope=rope)
    torch.cuda.synchronize()
    assert torch.equal(kpc, ke) and torch.equal(vpc, ve) and torch.equal(q_out, qe) and A.device_status()[0] == 0


def test_idle_rows_of_a_batch_of_single_tokens(A):
    """A batch of fixed size: rows of length 0 are skipped by the append and attend to nothing."""
    qkv, q, k, v, kp, vp, table, lens, cu = _case((1,) * 5, (14, 0, 16, 0, 100), 4, 2, seed=41)
    lens[[1, 3]] = 0
    dq, dk, dv = _split(qkv.cuda(), 4, 2)
    live = [0, 2, 4]
    want_k, want_v = kp.cuda(), vp.cuda()
    want_q = A.append_paged(dq[live], dk[live], dv[live], want_k, want_v, table[live].cuda(), lens[live].cuda())
    ke, ve = kp.cuda(), vp.cuda()
    q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    A.append_paged(dq, dk, dv, ke, ve, table.cuda(), lens.cuda(), q_out=q_out)
    cache = torch.zeros(kp.shape[0], 2, R.BLOCK, dtype=torch.uint8, device="cuda")
    q4_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    A.append_paged_q4(dq, dk, dv, cache, table.cuda(), lens.cuda(), q_out=q4_out)
    out, lse = A.decode_paged_q4(q4_out, cache, table.cuda(), lens.cuda())
    assert A.device_status()[0] == 0
    assert torch.equal(ke, want_k) and torch.equal(ve, want_v)
    assert torch.equal(q_out[live], want_q) and torch.equal(q4_out, q_out) and (q_out[[1, 3]] == 7.0).all()
    assert (out[[1, 3]] == 0).all() and torch.isneginf(lse[[1, 3]]).all() and torch.isfinite(lse[live]).all()
    # with offsets, a sequence of no length that has a token is still an error
    A.append_paged(dq, dk, dv, ke, ve, table.cuda(), lens.cuda(), cu.cuda())
    assert A.device_status()[0] == 6


def test_queries_in_place(A):
    qkv, q, k, v, kp, vp, table, lens, cu = _case((3, 1, 18, 0, 9), (14, 0, 16, 5, 100), 6, 2, seed=42, pad=4)
    rope = A.rope_table(R.inv_freq(96))
    w = (torch.rand(128) + 0.5).to(torch.bfloat16).cuda()
    for inter in (False, True):
        for fn, pools in ((A.append_paged, (kp.cuda(), vp.cuda())),
                          (A.append_paged_q4, (torch.zeros(kp.shape[0], 2, R.BLOCK, dtype=torch.uint8).cuda(),))):
            rest = (k.contiguous().cuda(), v.contiguous().cuda(), *pools, table.cuda(), lens.cuda(), cu.cuda())
            want = fn(q.contiguous().cuda(), *rest, rope=rope, q_weight=w, interleaved=inter)
            mine = q.contiguous().cuda()
            assert fn(mine, *rest, rope=rope, q_weight=w, interleaved=inter, q_out=mine) is mine
            n = int(cu[-1])
            assert torch.equal(mine[:n], want[:n]) and torch.equal(mine[n:].cpu(), q[n:])
    assert A.device_status()[0] == 0


def test_offsets_past_32_bits(A):
    """Pages behind the 2^31st element of the bf16 pools and the 2^32nd byte of the 4-bit cache."""
    Hkv, P = 8, 270000
    if torch.cuda.get_device_properties(0).total_memory < 2**35:
        pytest.skip("needs 16 GB")
    new, lens = (20, 1), torch.tensor([36, 18], dtype=torch.int32)
    g = torch.Generator().manual_seed(43)
    k, v = (torch.randn(21, Hkv, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(2, 16, 128, generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor((0,) + new).cumsum(0).to(torch.int32).cuda()
    cu_k = torch.tensor([0, 36, 54], dtype=torch.int32).cuda()
    res = []
    for pages, first in ((6, 0), (P, P - 6)):
        table = (torch.tensor([[5, 0, 3], [1, 4, -1]], dtype=torch.int32) + first).clamp_min(-1).cuda()
        kp, vp = (torch.empty(pages, 16, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kp[first:] = 0
        vp[first:] = 0
        A.append_paged(None, k, v, kp, vp, table, lens.cuda(), cu)
        part = [kp[first:].clone(), vp[first:].clone()]
        del kp, vp
        cache = torch.empty(2 * pages if first else pages, Hkv, R.BLOCK, dtype=torch.uint8, device="cuda")
        skip = cache.shape[0] - pages
        cache[skip + first:] = 0
        table += skip
        A.append_paged_q4(None, k, v, cache, table, lens.cuda(), cu)
        out, lse = A.decode_paged_q4(q, cache, table, lens.cuda())
        kk, vv = A.gather_paged_q4(cache, table, lens.cuda(), cu_k)
        o2, l2 = A.fwd_paged_q4(q, cache, table, lens.cuda(), torch.tensor([0, 1, 2], dtype=torch.int32).cuda())
        assert A.device_status()[0] == 0
        res.append(part + [cache[skip + first:].clone(), out, lse, kk, vv, o2, l2])
        del cache
    assert all(torch.equal(a, b) for a, b in zip(*res))
