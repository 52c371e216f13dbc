"""GPU tests of the head norms with the position rotation (attn_qk_norm_rope)
against 64 bits: head counts, odd lengths, layouts, strided views, both pair
orders, parts of the head dimension, several position axes, far and negative
positions, norms of one tensor only, in place, subnormal and huge rows."""
import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_06_gb300 as attn
    attn.load()
    return attn


def _inputs(B, S, Hq, Hkv, seed, norm=True):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, S, (Hq + 2 * Hkv) * 128, generator=g).to(torch.bfloat16)
    w = [(torch.rand(128, generator=g) * 2 - 0.5).to(torch.bfloat16) if norm else None for _ in range(2)]
    return qkv, w


def _views(qkv, Hq, Hkv, layout):
    q = qkv[..., :Hq * 128].unflatten(-1, (Hq, 128))
    k = qkv[..., Hq * 128:(Hq + Hkv) * 128].unflatten(-1, (Hkv, 128))
    return (q, k) if layout == "bshd" else (q.transpose(1, 2), k.transpose(1, 2))


def _check(got, x, w, pos, freq, axes, inter, layout, what):
    """got and x in the layout; pos [n_axes, B, S]."""
    if layout == "bhsd":
        got, x = got.transpose(1, 2), x.transpose(1, 2)
    ref = R.norm_rope(x.flatten(0, 1), w, EPS, pos.flatten(1), freq, axes, inter)
    R.check_norm_rope(got.cpu().flatten(0, 1), ref, what)


@pytest.mark.parametrize("layout", ["bshd", "bhsd"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hkv,rdim", [(1, 1, 1, 1, 128), (2, 37, 6, 2, 64), (1, 17, 32, 8, 96), (3, 5, 7, 7, 8),
                                             (1, 130, 12, 12, 120), (1, 3, 64, 1, 0)])
def test_matches_64_bits(A, layout, inter, B, S, Hq, Hkv, rdim):
    qkv, (wq, wk) = _inputs(B, S, Hq, Hkv, seed=B * S + rdim)
    freq = R.inv_freq(rdim) if rdim else []
    rope = A.rope_table(freq) if rdim else None
    pos = torch.arange(S).expand(1, B, S)
    dq, dk = _views(qkv.cuda(), Hq, Hkv, layout)
    cq, ck = _views(qkv, Hq, Hkv, layout)
    oq, ok = A.qk_norm_rope(dq, dk, rope=rope, q_weight=wq.cuda(), k_weight=wk.cuda(), eps=EPS, interleaved=inter,
                            layout=layout)
    torch.cuda.synchronize()
    assert oq.is_contiguous() and ok.is_contiguous() and A.device_status()[0] == 0
    _check(oq, cq, wq, pos, freq, [0] * len(freq), inter, layout, "q")
    _check(ok, ck, wk, pos, freq, [0] * len(freq), inter, layout, "k")


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n_axes", [1, 2, 3, 4])
def test_axes_and_far_positions(A, n_axes, inter):
    B, S, Hq, Hkv = 2, 29, 4, 2
    qkv, _ = _inputs(B, S, Hq, Hkv, seed=n_axes)
    freq = R.inv_freq(128)
    axes = [i * n_axes // 64 for i in range(64)] if inter else [i % n_axes for i in range(64)]
    g = torch.Generator().manual_seed(5)
    # positions over the whole range of 32 bits; the reference angle in 64 bits is then good to 2^31 2^-52
    pos = torch.randint(-2**31, 2**31, (n_axes, B, S), generator=g)
    pos[:, 0, :10] = torch.randint(0, 1000000, (n_axes, 10), generator=g)
    pos = pos.to(torch.int32)
    dq, dk = _views(qkv.cuda(), Hq, Hkv, "bshd")
    oq, ok = A.qk_norm_rope(dq, dk, rope=A.rope_table(freq, axes), positions=pos.cuda(), interleaved=inter)
    torch.cuda.synchronize()
    assert A.device_status()[0] == 0
    for o, x in zip((oq, ok), _views(qkv, Hq, Hkv, "bshd")):
        _check(o, x, None, pos, freq, axes, inter, "bshd", f"{n_axes} axes")


def test_norm_of_one_tensor_no_rotation_and_q_alone(A):
    qkv, (wq, _) = _inputs(1, 19, 5, 5, seed=9)
    dq, dk = _views(qkv.cuda(), 5, 5, "bshd")
    cq, ck = _views(qkv, 5, 5, "bshd")
    pos = torch.arange(19).expand(1, 1, 19)
    oq, ok = A.qk_norm_rope(dq, dk, q_weight=wq.cuda(), eps=EPS)
    _check(oq, cq, wq, pos, [], [], False, "bshd", "q normed")
    assert torch.equal(ok.cpu(), ck)                           # neither norm nor rotation: the same bits
    oq2, none = A.qk_norm_rope(dq, q_weight=wq.cuda(), eps=EPS)
    assert none is None and torch.equal(oq, oq2)


def test_packed_in_place_and_given_outputs(A):
    qkv, (wq, wk) = _inputs(1, 50, 6, 3, seed=10)
    q, k = (t[0].contiguous().cuda() for t in _views(qkv, 6, 3, "bshd"))
    rope = A.rope_table(R.inv_freq(128))
    pos = torch.arange(100, 150, dtype=torch.int32).cuda()
    kw = dict(rope=rope, positions=pos, q_weight=wq.cuda(), k_weight=wk.cuda())
    oq, ok = A.qk_norm_rope(q, k, **kw)
    q2, k2 = q.clone(), k.clone()
    r = A.qk_norm_rope(q2, k2, q_out=q2, k_out=k2, **kw)
    torch.cuda.synchronize()
    assert r[0] is q2 and r[1] is k2 and torch.equal(q2, oq) and torch.equal(k2, ok)
    with pytest.raises(ValueError):
        A.qk_norm_rope(q, k, q_out=torch.empty(50, 6, 64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        A.qk_norm_rope(q, k, rope=rope, positions=pos[:49])


def test_rows_of_zeros_and_of_extreme_values(A):
    x = torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16)
    x[0, 1] = 1e-30                                            # squares underflow: the norm is by eps alone
    x[0, 2] = 1e18                                             # squares' sum near the top of fp32
    x[0, 3, 0, 7] = 1.0
    w = torch.ones(128, dtype=torch.bfloat16)
    rope = A.rope_table(R.inv_freq(128))
    o, _ = A.qk_norm_rope(x.cuda(), rope=rope, q_weight=w.cuda(), eps=EPS)
    _check(o, x, w, torch.arange(4).expand(1, 1, 4), R.inv_freq(128), [0] * 64, False, "bshd", "extremes")


def test_nan_stays_in_its_row(A):
    qkv, (wq, wk) = _inputs(1, 8, 4, 2, seed=11)
    dq, dk = _views(qkv.cuda(), 4, 2, "bshd")
    kw = dict(rope=A.rope_table(R.inv_freq(128)), q_weight=wq.cuda(), k_weight=wk.cuda())
    clean = A.qk_norm_rope(dq, dk, **kw)[0]
    dq[0, 3, 2, 50] = float("nan")
    got = A.qk_norm_rope(dq, dk, **kw)[0]
    assert torch.isnan(got[0, 3, 2].float()).all()
    keep = torch.ones(1, 8, 4, dtype=torch.bool)
    keep[0, 3, 2] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])


def test_plan_with_an_axis_past_the_positions_is_reported(A):
    x = torch.randn(1, 4, 2, 128).to(torch.bfloat16).cuda()
    rope = A.rope_table(R.inv_freq(16), [0, 0, 0, 2, 0, 0, 0, 0])
    pos = torch.arange(4, dtype=torch.int32)[None].cuda()
    A.qk_norm_rope(x, rope=rope, positions=pos)
    assert A.device_status()[0] == 6
    A.qk_norm_rope(x, rope=rope)                               # default positions serve every axis
    assert A.device_status()[0] == 0
