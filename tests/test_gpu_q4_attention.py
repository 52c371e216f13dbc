"""GPU tests of the attention over the 4-bit cache: single tokens
(attn_decode_paged_q4) against 64 bits over the values the codes stand for,
the read-back (attn_gather_paged_q4) bit for bit, prompt chunks
(attn_fwd_paged_q4) against the oracle over the read-back values; lengths
around the page and the split, garbage past the end, bad tables, and the run
of appends and attention together."""
import pytest
import torch

import cache_ref as R
import oracle
from parity_util import check_lse, check_out

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_06_gb300 as attn
    attn.load()
    return attn


def _cache(lens, Hkv, seed, width=None, spread=1.0, garbage=True):
    """(cache, block table, lens): randn keys and values quantised; slots past each end and spare pages hold random
    bytes (NaN and infinite scales among them)."""
    g = torch.Generator().manual_seed(seed)
    pages = [(x + 15) // 16 for x in lens]
    P = sum(pages) + 2
    width = width or max(1, max(pages))
    perm = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    cache = torch.randint(0, 256, (P, Hkv, R.BLOCK), generator=g, dtype=torch.uint8)
    if garbage:
        cache[:, :, 2048:][torch.rand(P, Hkv, 512, generator=g) < 0.3] = 0xff
    off = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[off:off + n]
        off += n
        L = lens[b]
        if L == 0:
            continue
        t = torch.arange(L)
        k, v = (torch.randn(L, Hkv, 128, generator=g) for _ in range(2))
        k[torch.rand(L, generator=g) < 0.02] *= spread
        for h in range(Hkv):
            R.write_tokens(cache, table[b].long()[t // 16], t % 16, torch.full_like(t, h), k[:, h].to(torch.bfloat16),
                           v[:, h].to(torch.bfloat16))
    return cache, table, torch.tensor(lens, dtype=torch.int32)


def _decode(A, lens, Hq, Hkv, seed, scale=SCALE, **kw):
    cache, table, dl = _cache(lens, Hkv, seed, **kw)
    q = torch.randn(len(lens), Hq, 128, generator=torch.Generator().manual_seed(seed + 1)).to(torch.bfloat16)
    out, lse = A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda(), scale=scale)
    torch.cuda.synchronize()
    assert A.device_status()[0] == 0
    R.check_decode_q4(out, lse, q, cache, table, lens, scale, f"Hq={Hq} Hkv={Hkv}")
    return q, cache, table, dl, out, lse


EDGE = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 255, 257]


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (8, 2), (32, 8), (8, 1), (10, 2), (12, 1), (16, 1), (48, 2)])
def test_decode_edges_match_64_bits(A, Hq, Hkv):
    _decode(A, EDGE, Hq, Hkv, seed=Hq * 10 + Hkv)


@pytest.mark.parametrize("lens,width", [([1000, 4097, 0, 2048, 5], None), ([70000], None), ([300, 20], 3000),
                                        ([4096] * 40, None)])
def test_decode_long_and_wide_tables(A, lens, width):
    """Key splits: ragged lengths, one long sequence, a table far wider than the sequences, many sequences."""
    _decode(A, lens, 4, 1, seed=len(lens) + lens[0], width=width)


@pytest.mark.parametrize("lens", [[1280], [300, 1152, 20, 1500], [30000, 9000, 5]])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 1), (32, 1), (20, 2)])
def test_decode_merges_of_few_and_many_parts(A, Hq, Hkv, lens):
    """Runs cut into two, into about as many parts as there are heads, and into far more."""
    _decode(A, lens, Hq, Hkv, seed=90 + len(lens))


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 8)])
@pytest.mark.parametrize("B,hi,long", [(1, 0, 0), (31, 0, 0), (32, 90, 0), (33, 90, 2500), (57, 260, 0), (60, 40, 700),
                                       (130, 30, 0), (200, 33, 9000), (500, 20, 0)])
def test_decode_ways_to_share_out_a_batch(A, B, hi, long, Hq, Hkv):
    """Batches of up to and of more than 32 sequences, of nothing, of short ragged ones with a long one among them, with
    fewer and with more KV heads than CTAs: whole runs, runs in parts and equal shares."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    if long:
        lens[B // 2] = long
    _decode(A, lens, Hq, Hkv, seed=B)


@pytest.mark.parametrize("width", [32, 33, 34])
@pytest.mark.parametrize("B,Hkv", [(1, 1), (3, 2), (57, 8), (58, 8)])
def test_decode_around_the_width_that_is_never_cut(A, B, Hkv, width):
    """Tables of 512 tokens, where no merge is launched, and just above; as many KV heads as there are CTAs, and more."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 16 * width + 1, (B,), generator=g).tolist()
    lens[B // 2] = 16 * width
    _decode(A, lens, 2 * Hkv, Hkv, seed=B + width, width=width)


def test_decode_peaked_scores_and_scales(A):
    _decode(A, [500, 33, 1200], 8, 2, seed=5, spread=30.0)
    for scale in (0.0, 1.0):
        _decode(A, [200, 47], 8, 2, seed=6, scale=scale)


def test_decode_extreme_values_and_queries(A):
    """Values near the top and the bottom of bf16, keys of very different sizes, queries of zeros and far apart."""
    g = torch.Generator().manual_seed(60)
    for v_scale, k_scale, q_scale in ((1e38, 1.0, 1.0), (1e-36, 1.0, 1.0), (1.0, 1e-30, 1e20), (1.0, 0.0, 1.0), (1.0, 1.0, 0.0)):
        L = 75
        cache = torch.zeros(5, 1, R.BLOCK, dtype=torch.uint8)
        table = torch.tensor([[3, 0, 4, 1, 2]], dtype=torch.int32)
        t = torch.arange(L)
        k = (torch.randn(L, 128, generator=g) * k_scale).to(torch.bfloat16)
        v = (torch.rand(L, 128, generator=g) * 2 - 1).mul(v_scale).to(torch.bfloat16)
        R.write_tokens(cache, table[0].long()[t // 16], t % 16, torch.zeros_like(t), k, v)
        q = (torch.randn(1, 3, 128, generator=g) * q_scale).to(torch.bfloat16)
        out, lse = A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), torch.tensor([L], dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        R.check_decode_q4(out, lse, q, cache, table, [L], SCALE, f"v {v_scale} k {k_scale} q {q_scale}")


def _mixed(lens, Hkv, G, kind, seed):
    """(q, cache, table): channel 0 of the queries is 8 (-8 in every fourth head), so that a key's channel 0 decides
    how likely its token is."""
    g = torch.Generator().manual_seed(seed)
    pages = [(x + 15) // 16 for x in lens]
    table = torch.zeros(len(lens), max(pages), dtype=torch.int32)
    perm = torch.randperm(sum(pages), generator=g).to(torch.int32)
    cache = torch.full((sum(pages), Hkv, R.BLOCK), 0xff, dtype=torch.uint8)
    off = 0
    for b, L in enumerate(lens):
        table[b, :pages[b]] = perm[off:off + pages[b]]
        off += pages[b]
        t = torch.arange(L)
        k, v = (torch.randn(L, Hkv, 128, generator=g) for _ in range(2))
        if kind.startswith("hidden"):                  # large values that most heads do not attend to
            rare = torch.rand(L, Hkv, generator=g) < 0.02
            rare[0] = False
            k[..., 0][rare] = -40.0
            v[rare] *= 2.0 ** int(kind[6:])
        elif kind == "sink":                           # small values behind a likely token with next to none
            v *= 2.0 ** -7
            v[0] *= 2.0 ** -6
            k[0, :, 0] = 14.0
        elif kind == "growing":
            v *= 2.0 ** (t / L * 60 - 30)[:, None, None]
        elif kind == "shrinking":
            v *= 2.0 ** (30 - t / L * 60)[:, None, None]
        else:                                          # zeros, or tiny values, in the first pages
            v[:L * 2 // 3] *= 0.0 if kind == "zeros" else 2.0 ** -100
        for h in range(Hkv):
            R.write_tokens(cache, table[b].long()[t // 16], t % 16, torch.full_like(t, h), k[:, h].to(torch.bfloat16),
                           v[:, h].to(torch.bfloat16))
    q = torch.randn(len(lens), Hkv * G, 128, generator=g)
    q[..., 0] = 8.0
    q[:, 3::4, 0] = -8.0
    return q.to(torch.bfloat16), cache, table


@pytest.mark.parametrize("kind", ["hidden12", "hidden20", "hidden36", "sink", "growing", "shrinking", "zeros", "tiny"])
@pytest.mark.parametrize("lens,Hkv,G", [([600, 33, 2, 64, 2000], 2, 4), ([1500] * 24, 8, 4), ([700, 47, 1900], 2, 12)])
def test_decode_values_of_very_different_scales(A, lens, Hkv, G, kind):
    """A token that a head does not attend to takes no precision from it, whatever its scale; scales that grow and
    shrink by 2^60 along a sequence; pages of zeros or of next to nothing before the others."""
    q, cache, table = _mixed(lens, Hkv, G, kind, seed=len(lens) + G)
    out, lse = A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert A.device_status()[0] == 0
    R.check_decode_q4_mixed(out, lse, q, cache, table, lens, SCALE, kind)


@pytest.mark.parametrize("Hq", [8, 16])
def test_decode_heads_of_very_different_queries(A, Hq):
    """Queries of 2^-60 to 2^118 beside the usual ones; heads of NaN or infinities leave the others' bits alone."""
    lens = [150, 40, 1]
    cache, table, dl = _cache(lens, 1, seed=70)
    q = torch.randn(3, Hq, 128, generator=torch.Generator().manual_seed(71))
    run = lambda q: A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda())  # noqa: E731
    for big in (30, 100, 118):
        x = q.clone()
        x[:, 1] *= 2.0 ** big
        x[:, 3] *= 2.0 ** -60
        out, lse = run(x.to(torch.bfloat16))
        R.check_decode_q4(out, lse, x.to(torch.bfloat16), cache, table, lens, SCALE, f"2^{big}")
    x = q.to(torch.bfloat16)
    x[:, 2] = x[:, 5] = 0
    clean = run(x)
    x[:, 2], x[:, 5] = float("nan"), float("inf")
    x[1, 5, 7:] = 0
    out, lse = run(x)
    assert A.device_status()[0] == 0
    rest = [h for h in range(Hq) if h not in (2, 5)]
    assert torch.equal(out[:, rest], clean[0][:, rest]) and torch.equal(lse[:, rest], clean[1][:, rest])
    assert torch.isnan(out[:, 2].float()).all()


def test_decode_is_deterministic_and_takes_given_outputs(A):
    q, cache, table, dl, out, lse = _decode(A, [900, 1, 3000], 8, 2, seed=7)
    ws = torch.full((A.decode_q4_workspace_bytes(3, 8, 2, 128, table.shape[1]),), 0xff, dtype=torch.uint8, device="cuda")
    o, l = torch.empty_like(out), torch.empty_like(lse)
    for _ in range(3):
        r = A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda(), out=o, lse=l, workspace=ws)
        torch.cuda.synchronize()
        assert r[0] is o and torch.equal(o, out) and torch.equal(l, lse)
    o2, none = A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda(), lse=False, workspace=ws)
    assert none is None and torch.equal(o2, out)
    with pytest.raises(A.AttnError):
        A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda(), workspace=ws[:256])


def test_decode_nan_key_and_value_reach_only_their_sequence(A):
    lens = [40, 40, 40]
    cache, table, dl = _cache(lens, 1, seed=8, garbage=False)
    q = torch.randn(3, 2, 128).to(torch.bfloat16)
    clean = A.decode_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda())[0].cpu()
    bad = cache.clone()
    bad[int(table[1, 2]), 0, 2304 + 8 * 7 + 2 * 3:][:2] = 0xff        # token 39's value scale of group 3
    got = A.decode_paged_q4(q.cuda(), bad.cuda(), table.cuda(), dl.cuda())[0].cpu()
    assert torch.isnan(got[1, :, 96:].float()).all() and torch.isfinite(got[1, :, :96].float()).all()
    assert torch.equal(got[[0, 2]], clean[[0, 2]])
    bad = cache.clone()
    bad[int(table[2, 0]), 0, 2048:2050] = 0xff                        # token 0's key scale of group 0
    got = A.decode_paged_q4(q.cuda(), bad.cuda(), table.cuda(), dl.cuda())[0].cpu()
    assert torch.isnan(got[2].float()).all() and torch.equal(got[:2], clean[:2])


def test_decode_bad_tables_and_lengths_are_reported(A):
    lens = [40, 100, 33]
    cache, table, dl = _cache(lens, 2, seed=9)
    q = torch.randn(3, 4, 128).to(torch.bfloat16)
    run = lambda t, l: A.decode_paged_q4(q.cuda(), cache.cuda(), t.cuda(), l.cuda())  # noqa: E731
    clean = run(table, dl)
    for wrong in (cache.shape[0], -1, 2**31 - 1):
        bad = table.clone()
        bad[1, 6] = wrong                                             # its last page: keys 96 .. 99 count as absent
        out, lse = run(bad, dl)
        assert A.device_status()[0] == 6
        R.check_decode_q4(out[1:2], lse[1:2], q[1:2], cache, table[1:2], [96], SCALE, "bad page")
        assert torch.equal(out[[0, 2]], clean[0][[0, 2]])
    for wrong in (-1, 16 * table.shape[1] + 1):
        bad = dl.clone()
        bad[0] = wrong
        out, lse = run(table, bad)
        assert A.device_status()[0] == 6
        # (the other sequences' sums are the same up to their order, which goes by the whole batch's lengths)
        R.check_decode_q4(out, lse, q, cache, table, [0, 100, 33], SCALE, "bad length")


@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_gather_bits(A, Hkv):
    lens = EDGE + [0, 700]
    cache, table, dl = _cache(lens, Hkv, seed=10 + Hkv)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    total = sum(lens) + 5                                             # rows behind the last sequence
    k, v = (torch.full((total, Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.gather_paged_q4(cache.cuda(), table.cuda(), dl.cuda(), cu.cuda(), k_out=k, v_out=v)
    torch.cuda.synchronize()
    assert A.device_status()[0] == 0
    for b, L in enumerate(lens):
        kp, vp = R.read_tokens(cache, table[b], L) if L else (None, None)
        for got, parts in ((k, kp), (v, vp)):
            if L:
                assert torch.equal(got[int(cu[b]):int(cu[b + 1])].cpu(), R.values_bf16(parts))
    assert (k[sum(lens):] == 7.0).all() and (v[sum(lens):] == 7.0).all()


def test_gather_bad_arguments_are_reported(A):
    lens = [40, 100, 33]
    cache, table, dl = _cache(lens, 2, seed=12)
    cu = torch.tensor([0, 40, 140, 173], dtype=torch.int32)

    def run(table=table, dl=dl, cu=cu):
        k, v = (torch.full((173, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        A.gather_paged_q4(cache.cuda(), table.cuda(), dl.cuda(), cu.cuda(), k_out=k, v_out=v)
        return A.device_status()[0], k.cpu()

    code, good = run()
    assert code == 0
    bad = table.clone()
    bad[1, 1] = cache.shape[0]
    code, k = run(table=bad)
    assert code == 6 and (k[56:72] == 0).all() and torch.equal(k[72:], good[72:]) and torch.equal(k[:56], good[:56])
    bad = dl.clone()
    bad[1] = 99                                                       # not the offsets' difference: skipped
    code, k = run(dl=bad)
    assert code == 6 and (k[40:140] == 7.0).all() and torch.equal(k[140:], good[140:])
    bad = cu.clone()
    bad[3] = 174
    assert run(cu=bad)[0] == 6


CHUNKS, CTX = (1, 5, 16, 17, 127, 129, 300, 2), (0, 30, 0, 200, 1, 260, 77, 15)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 1)])
def test_fwd_matches_oracle_over_the_values_read_back(A, Hq, Hkv, causal):
    lens = [a + c for a, c in zip(CHUNKS, CTX)]
    cache, table, dl = _cache(lens, Hkv, seed=13)
    cu = torch.tensor((0,) + CHUNKS).cumsum(0).to(torch.int32)
    cu_k = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    q = torch.randn(sum(CHUNKS), Hq, 128, generator=torch.Generator().manual_seed(14)).to(torch.bfloat16)
    parts = [R.read_tokens(cache, table[b], L) for b, L in enumerate(lens)]
    k, v = (torch.cat([R.values_bf16(p[i]) for p in parts]) for i in (0, 1))
    ref_o, ref_l = oracle.attention_varlen(q, k, v, cu, cu_k, Hq=Hq, Hkv=Hkv, causal=causal, scale=SCALE)
    # a workspace of NaN, a bound above the lengths' sum, and both read from the device
    need = A.fwd_paged_q4_workspace_bytes(len(lens), Hkv, 128, sum(lens) + 100)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = A.fwd_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda(), cu.cuda(), max_total_k=sum(lens) + 100,
                              causal=causal, workspace=ws)
    out2, lse2 = A.fwd_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda(), cu.cuda(), causal=causal)
    torch.cuda.synchronize()
    assert A.device_status()[0] == 0
    check_out(out, ref_o, "chunks over the 4-bit cache")
    check_lse(lse, ref_l, "chunks over the 4-bit cache")
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_fwd_reports_lengths_past_the_bound_and_the_table(A):
    lens = [40, 100, 33]
    cache, table, dl = _cache(lens, 1, seed=15)
    cu = torch.tensor([0, 4, 9, 12], dtype=torch.int32)
    q = torch.randn(12, 2, 128).to(torch.bfloat16).cuda()
    run = lambda l, bound: A.fwd_paged_q4(q, cache.cuda(), table.cuda(), l.cuda(), cu.cuda(), max_total_k=bound)  # noqa: E731
    good = run(dl, 173)[0]
    assert A.device_status()[0] == 0
    out, lse = run(dl, 172)                                           # the last sequence goes past the bound
    assert A.device_status()[0] == 6
    assert torch.equal(out[:9], good[:9]) and (out[9:] == 0).all() and torch.isneginf(lse[:, 9:]).all()
    out, lse = run(dl, 50)                                            # the second and the third
    assert A.device_status()[0] == 6 and torch.equal(out[:4], good[:4]) and (out[4:] == 0).all()
    bad = dl.clone()
    bad[0] = -5
    out, lse = run(bad, 173)
    assert A.device_status()[0] == 6 and (out[:4] == 0).all() and torch.equal(out[4:], good[4:])


def test_fwd_many_sequences(A):
    """More sequences than one round of the offsets' sum."""
    B = 1500
    g = torch.Generator().manual_seed(16)
    lens = [int(x) for x in torch.randint(0, 20, (B,), generator=g)]
    cache, table, dl = _cache(lens, 1, seed=17)
    new = [min(1, x) for x in lens]
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    q = torch.randn(sum(new), 1, 128, generator=g).to(torch.bfloat16)
    out, lse = A.fwd_paged_q4(q.cuda(), cache.cuda(), table.cuda(), dl.cuda(), cu.cuda())
    torch.cuda.synchronize()
    assert A.device_status()[0] == 0
    cu_k = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    parts = [R.read_tokens(cache, table[b], L) for b, L in enumerate(lens) if L]
    k, v = (torch.cat([R.values_bf16(p[i]) for p in parts]) for i in (0, 1))
    ref_o, ref_l = oracle.attention_varlen(q, k, v, cu, cu_k, Hq=1, Hkv=1, causal=True, scale=SCALE)
    check_out(out, ref_o, "many sequences")
    check_lse(lse, ref_l, "many sequences")


def test_serving_run_over_the_4_bit_cache(A):
    """Prompt chunks, then single tokens, appended and attended to; at the end the cache against one quantised from the
    bf16 cache that the same run builds."""
    Hq, Hkv, B = 8, 2, 3
    g = torch.Generator().manual_seed(31)
    rope = A.rope_table(R.inv_freq(128))
    chunks = [(5, 40, 17), (30, 1, 16), (1, 1, 1), (1, 1, 1)]
    total = [sum(c[b] for c in chunks) for b in range(B)]
    width = max((t + 15) // 16 for t in total)
    table = torch.randperm(B * width, generator=g).to(torch.int32).reshape(B, width)
    cache = torch.full((B * width, Hkv, R.BLOCK), 0xff, dtype=torch.uint8, device="cuda")
    kp, vp = (torch.zeros(B * width, 16, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    done = torch.zeros(B, dtype=torch.int32)
    for c in chunks:
        done = done + torch.tensor(c, dtype=torch.int32)
        cu = torch.tensor((0,) + c).cumsum(0).to(torch.int32)
        qkv = torch.randn(sum(c), (Hq + 2 * Hkv) * 128, generator=g).to(torch.bfloat16).cuda()
        q = qkv[:, :Hq * 128].unflatten(-1, (Hq, 128))
        k = qkv[:, Hq * 128:(Hq + Hkv) * 128].unflatten(-1, (Hkv, 128))
        v = qkv[:, (Hq + Hkv) * 128:].unflatten(-1, (Hkv, 128))
        args = (table.cuda(), done.cuda())
        q_rot = A.append_paged_q4(q, k, v, cache, *args, cu.cuda(), rope=rope)
        A.append_paged(None, k, v, kp, vp, *args, cu.cuda(), rope=rope)
        lens = done.tolist()
        if max(c) > 1:
            out, lse = A.fwd_paged_q4(q_rot, cache, *args, cu.cuda(), max_seqlen_q=max(c), max_total_k=sum(lens))
            parts = [R.read_tokens(cache.cpu(), table[b], L) for b, L in enumerate(lens)]
            kk, vv = (torch.cat([R.values_bf16(p[i]) for p in parts]) for i in (0, 1))
            cu_k = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
            ref_o, ref_l = oracle.attention_varlen(q_rot.cpu(), kk, vv, cu, cu_k, Hq=Hq, Hkv=Hkv, causal=True, scale=SCALE)
            check_out(out, ref_o, f"chunk {c}")
            check_lse(lse, ref_l, f"chunk {c}")
        else:
            out, lse = A.decode_paged_q4(q_rot, cache, *args)
            R.check_decode_q4(out, lse, q_rot.cpu(), cache.cpu(), table, lens, SCALE, f"step {c}")
    want = R.pack_pools(kp.cpu(), vp.cpu())
    for b in range(B):
        for x, y in zip(R.read_tokens(cache.cpu(), table[b], total[b]), R.read_tokens(want, table[b], total[b])):
            assert all(torch.equal(i, j) for i, j in zip(x, y))
    assert A.device_status()[0] == 0


def test_captured_steps_and_two_streams(A):
    """Two captured decode steps with workspaces of their own, replayed on two streams at once after the lengths
    changed, equal the eager results; a captured chunk as well."""
    cases = []
    for seed in (50, 51):
        lens = [100, 2000, 17]
        cache, table, dl = _cache(lens, 2, seed=seed, width=128)
        q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
        d = [t.cuda() for t in (q, cache, table, dl)]
        ws = torch.empty(A.decode_q4_workspace_bytes(3, 8, 2, 128, 128), dtype=torch.uint8, device="cuda")
        ws2 = torch.empty(A.fwd_paged_q4_workspace_bytes(3, 2, 128, 2200), dtype=torch.uint8, device="cuda")
        cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
        o, l, o2, l2 = (torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, device="cuda"),
                        torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 3, device="cuda"))
        s = torch.cuda.Stream()

        def step(d=d, ws=ws, ws2=ws2, cu=cu, o=o, l=l, o2=o2, l2=l2, s=s):
            A.decode_paged_q4(*d, out=o, lse=l, workspace=ws, stream=s)
            A.fwd_paged_q4(*d, cu, max_seqlen_q=1, max_total_k=2200, out=o2, lse=l2, workspace=ws2, stream=s)

        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        cases.append((graph, s, d, (o, l, o2, l2), step))
    for graph, s, d, outs, step in cases:
        d[3] -= 16
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s, *_ in cases:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for graph, s, d, outs, step in cases:
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))
    assert A.device_status()[0] == 0
