"""Refusals of the operators around the paged cache, before any launch (CPU):
the C ABI's argument checks and the binding's, and the rotation plan."""
import fractions
import math

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


NORM = dict(q=256, k=512, qo=1024, ko=2048, qw=16, kw=16, eps=1e-6, pos=4, axes=1, rope=16, R=128, inter=0, B=2, S=8,
            Hq=4, Hkv=2, d=128, layout=0, qb=4096, qs=512, qh=128, kb=2048, ks=256, kh=128)


def _norm(lib, **kw):
    a = dict(NORM, **kw)
    return lib.attn_qk_norm_rope(*[a[n] for n in NORM], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(q=264), 1), (dict(qo=None), 1), (dict(qo=1032), 1), (dict(ko=None), 1),
    (dict(k=None), 1),                              # k_out without k
    (dict(k=520), 1), (dict(qw=18), 1), (dict(kw=24), 1), (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1),
    (dict(pos=6), 1), (dict(axes=0), 1), (dict(axes=5), 1), (dict(rope=None), 1), (dict(rope=8), 1),
    (dict(R=0), 1), (dict(R=-8), 1), (dict(R=136), 1), (dict(R=12), 2), (dict(d=64), 2), (dict(B=0), 1),
    (dict(S=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(layout=2), 1), (dict(qs=516), 1), (dict(kh=4), 1),
    (dict(qo=256, qh=256), 1),                      # in place over a strided q
    (dict(ko=512, ks=512), 1), (dict(B=1 << 20, S=1 << 20), 1), (dict(Hq=1 << 20), 1),
])
def test_norm_rope_rejects_before_any_launch(lib, kw, code):
    assert _norm(lib, **kw) == code


APPEND = dict(q=256, k=512, v=1024, qo=2048, kp=4096, vp=8192, bt=4, sl=4, cu=4, qw=16, kw=16, eps=1e-6, pos=None,
              axes=1, rope=16, R=128, inter=0, B=2, total=5, Hq=4, Hkv=2, d=128, page=16, npages=10, maxb=4, qs=512,
              ks=256, vs=256)


def _append(lib, q4, **kw):
    a = dict(APPEND, **kw)
    names = [n for n in APPEND if not (q4 and n == "vp")]
    return (lib.attn_append_paged_q4 if q4 else lib.attn_append_paged)(*[a[n] for n in names], None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(v=1028), 1), (dict(kp=None), 1), (dict(kp=4100), 1),
    (dict(bt=None), 1), (dict(bt=6), 1), (dict(sl=None), 1), (dict(cu=6), 1),
    (dict(cu=None), 1),                             # one token per sequence needs total == B
    (dict(q=None), 1),                              # q_out without q
    (dict(qo=None), 1), (dict(q=260), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(B=0), 1), (dict(total=0), 1),
    (dict(npages=0), 1), (dict(maxb=0), 1), (dict(npages=1 << 28), 1), (dict(qs=511), 1), (dict(qs=256), 1),
    (dict(ks=248), 1), (dict(vs=260), 1), (dict(qo=256, qs=1024), 1), (dict(d=64), 2), (dict(page=32), 2),
    (dict(R=20), 2), (dict(axes=7), 1), (dict(rope=None), 1), (dict(eps=float("inf")), 1),
])
def test_append_rejects_before_any_launch(lib, q4, kw, code):
    assert _append(lib, q4, **kw) == code


def _gather(lib, **kw):
    a = dict(c=16, bt=4, sl=4, cu=4, ko=16, vo=16, B=2, Hkv=2, total=10, d=128, page=16, npages=4, maxb=4)
    a.update(kw)
    return lib.attn_gather_paged_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), 1), (dict(c=8), 1), (dict(ko=None), 1), (dict(vo=8), 1), (dict(cu=None), 1), (dict(cu=2), 1),
    (dict(bt=2), 1), (dict(sl=None), 1), (dict(B=0), 1), (dict(Hkv=0), 1), (dict(total=0), 1), (dict(npages=0), 1),
    (dict(maxb=0), 1), (dict(d=64), 2), (dict(page=8), 2), (dict(total=1 << 30, Hkv=1 << 10), 1),
])
def test_gather_rejects_before_any_launch(lib, kw, code):
    assert _gather(lib, **kw) == code


def _decode(lib, **kw):
    a = dict(q=16, c=16, bt=16, sl=16, out=16, lse=None, B=2, Hq=4, Hkv=2, d=128, page=16, npages=10, maxb=4,
             scale=0.1, ws=256, wsb=1 << 20)
    a.update(kw)
    return lib.attn_decode_paged_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(c=None), 1), (dict(c=24), 1), (dict(bt=18), 1), (dict(Hq=5), 1), (dict(npages=0), 1),
    (dict(maxb=0), 1), (dict(maxb=1 << 28), 1), (dict(scale=float("nan")), 1), (dict(scale=-0.5), 1),
    (dict(page=32), 2), (dict(d=256), 2), (dict(B=70000), 1), (dict(ws=None), 5), (dict(ws=272), 5), (dict(wsb=16), 5),
])
def test_decode_q4_rejects_before_any_launch(lib, kw, code):
    assert _decode(lib, **kw) == code


def _fwd(lib, **kw):
    a = dict(q=16, c=16, bt=4, sl=4, cu=4, out=16, lse=None, B=2, Hq=4, Hkv=2, tq=100, mq=60, d=128, page=16,
             npages=10, maxb=4, mk=128, causal=1, scale=0.1, mode=0, ws=256, wsb=1 << 22)
    a.update(kw)
    return lib.attn_fwd_paged_q4(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(c=8), 1), (dict(out=None), 1), (dict(lse=2), 1), (dict(cu=None), 1), (dict(bt=None), 1),
    (dict(sl=6), 1), (dict(B=0), 1), (dict(Hq=3), 1), (dict(tq=0), 1), (dict(mq=0), 1), (dict(mq=101), 1),
    (dict(mk=0), 1), (dict(mk=1 << 30, Hkv=4), 1), (dict(mode=3), 1), (dict(scale=float("inf")), 1), (dict(d=64), 2),
    (dict(page=32), 2), (dict(ws=None), 5), (dict(ws=128), 5), (dict(wsb=100), 5),
])
def test_fwd_paged_q4_rejects_before_any_launch(lib, kw, code):
    assert _fwd(lib, **kw) == code


def test_workspace_sizes_are_pure_functions(lib):
    a = A.decode_q4_workspace_bytes(32, 32, 8, 128, 512)
    assert a == A.decode_q4_workspace_bytes(32, 32, 8, 128, 512) > 0
    assert A.decode_q4_workspace_bytes(32, 30, 8, 128, 512) == 0
    assert A.decode_q4_workspace_bytes(32, 32, 8, 64, 512) == 0
    assert A.decode_q4_workspace_bytes(32, 32, 8, 128, 0) == 0
    b = A.fwd_paged_q4_workspace_bytes(4, 8, 128, 1000)
    assert b >= 2 * 1000 * 8 * 256 and b < 2 * 1000 * 8 * 256 + 4096
    assert A.fwd_paged_q4_workspace_bytes(4, 8, 128, 0) == 0


def test_rope_table_holds_exact_turns():
    freq = [1.0, 10000.0 ** -0.5, 1e-6, -0.25, 7.0, 0.0]
    t = A.rope_table(freq, [0, 1, 2, 3, 0, 1], device="cpu")
    assert t.dtype == torch.int64 and tuple(t.shape) == (6, 2)
    assert t[:, 1].tolist() == [0, 1, 2, 3, 0, 1]
    for f, turns in zip(freq, t[:, 0].tolist()):
        # the fraction of a turn at far positions, against 64-bit angles
        for pos in (1, 12345, 1000000, -77):
            frac = fractions.Fraction(pos * turns % 2**64, 2**64)
            want = math.fmod(pos * f, 2 * math.pi)
            # fmod is exact; the angle is rounded once in 64 bits and once more by the comparison's 2 pi
            assert abs(math.sin(2 * math.pi * float(frac)) - math.sin(want)) <= 2.0 ** -52 * (abs(pos * f) + 4)
    assert torch.equal(A.rope_table(torch.tensor(freq, dtype=torch.float64), device="cpu")[:, 0], t[:, 0])


@pytest.mark.parametrize("freq,axes", [([], None), ([1.0], [0, 1]), ([float("nan")], None), ([1.0], [4]),
                                       ([1.0], [-1])])
def test_rope_table_refuses(freq, axes):
    with pytest.raises(ValueError):
        A.rope_table(freq, axes, device="cpu")


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x = torch.zeros(1, 2, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        A.qk_norm_rope(x, x)
    with pytest.raises(TypeError):
        A.append_paged(None, x[0], x[0], x, x, x, x)
    with pytest.raises(TypeError):
        A.append_paged_q4(None, x[0], x[0], x, x, x)
    with pytest.raises(TypeError):
        A.decode_paged_q4(x[0], x, x, x)
    with pytest.raises(TypeError):
        A.gather_paged_q4(x, x, x, x)
    with pytest.raises(ValueError):
        A.qk_norm_rope(x, x, layout="bsdh")


def test_quick_way_turns_down_what_is_not_in_order(lib):
    """Wrong counts and kinds of arguments, and tensors that are not on a GPU: None, for the long way to say why."""
    quick = _binding._quick
    t = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    for name, n in (("qk_norm_rope", 11), ("append", 15), ("gather", 7), ("decode", 8), ("fwd", 13)):
        fn = getattr(quick, name)
        assert fn() is None and fn(*[None] * n) is None and fn(*["x"] * n) is None and fn(*[t] * n) is None
        assert fn(*[t] * (n - 1)) is None
