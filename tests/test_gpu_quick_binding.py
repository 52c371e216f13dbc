"""GPU tests of the binding's quick way (_quick.so) into the operators around the paged cache: the same results as
the long way for every form of a call, the long way's errors for calls that are out of order, given outputs kept as
they are, and nothing left behind by repeated calls."""
import gc
import sys

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
Hq, Hkv, B = 8, 2, 3


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_06_gb300 as attn
    attn.load()
    return attn


class _Never:
    """In _quick's place: every call goes the long way."""

    def __getattr__(self, name):
        return lambda *a: None


class _Only:
    """In _quick's place: a call that it turns down is an error."""

    def __init__(self, quick):
        self.quick = quick

    def __getattr__(self, name):
        def call(*a):
            r = getattr(self.quick, name)(*a)
            assert r is not None, name
            return r
        return call


def _state():
    g = torch.Generator().manual_seed(80)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    new = torch.tensor([5, 1, 20], dtype=torch.int32)
    s = dict(qkv=r(26, (Hq + 2 * Hkv) * 128), w=r(128), table=torch.randperm(12, generator=g).int().reshape(B, 4).cuda(),
             lens=torch.tensor([25, 1, 33], dtype=torch.int32).cuda(), cu=torch.cat([torch.zeros(1), new.cumsum(0)]).int().cuda(),
             cu_k=torch.tensor([0, 25, 26, 59], dtype=torch.int32).cuda(), x=r(2, 7, Hq, 128), y=r(2, 7, Hkv, 128),
             pos=torch.randint(-50, 5000, (2, 2, 7), generator=g, dtype=torch.int32).cuda(), one=r(B, Hq, 128),
             pos1=torch.randint(0, 99, (26,), generator=g, dtype=torch.int32).cuda(),
             pos2=torch.randint(0, 99, (2, 26), generator=g, dtype=torch.int32).cuda())
    c = [Hq * 128, Hkv * 128, Hkv * 128]
    s["q"], s["k"], s["v"] = (t.unflatten(-1, (-1, 128)) for t in s["qkv"].split(c, -1))
    s["kp"], s["vp"] = r(12, 16, Hkv, 128), r(12, 16, Hkv, 128)
    s["cache"] = torch.zeros(12, Hkv, R.BLOCK, dtype=torch.uint8, device="cuda")
    return s


def _calls(A):
    """name -> (call of a state, the tensors to compare)."""
    rope, rope3 = A.rope_table(R.inv_freq(128)), A.rope_table(R.inv_freq(64), [0, 1] * 16)
    t = lambda s: (s["table"], s["lens"])  # noqa: E731
    return {
        "norm": lambda s: A.qk_norm_rope(s["x"], s["y"], rope=rope, q_weight=s["w"], k_weight=s["w"]),
        "norm bhsd": lambda s: A.qk_norm_rope(s["x"].transpose(1, 2), s["y"].transpose(1, 2), rope=rope3,
                                              positions=s["pos"], layout="bhsd", interleaved=True),
        "norm packed q": lambda s: A.qk_norm_rope(s["q"], rope=rope, positions=s["pos1"], eps=1e-3, q_weight=s["w"]),
        "norm in place": lambda s: A.qk_norm_rope(s["x"], s["y"], rope=rope, q_out=s["x"], k_out=s["y"]),
        "append": lambda s: [A.append_paged(s["q"], s["k"], s["v"], s["kp"], s["vp"], *t(s), s["cu"], rope=rope,
                                            k_weight=s["w"]), s["kp"], s["vp"]],
        "append one": lambda s: [A.append_paged(None, s["k"][:3], s["v"][:3], s["kp"], s["vp"], *t(s)), s["kp"], s["vp"]],
        "append q4": lambda s: [A.append_paged_q4(s["q"], s["k"], s["v"], s["cache"], *t(s), s["cu"], rope=rope3,
                                                  positions=s["pos2"], interleaved=True), s["cache"]],
        "gather": lambda s: A.gather_paged_q4(s["cache"], *t(s), s["cu_k"], total_k=59),
        "decode": lambda s: A.decode_paged_q4(s["one"], s["cache"], *t(s)),
        "decode given": lambda s: A.decode_paged_q4(s["one"], s["cache"], *t(s), scale=0.5, lse=False, workspace=torch.empty(
            A.decode_q4_workspace_bytes(B, Hq, Hkv, 128, 4), dtype=torch.uint8, device="cuda")),
        "fwd": lambda s: A.fwd_paged_q4(s["q"].contiguous(), s["cache"], *t(s), s["cu"], max_seqlen_q=20, max_total_k=59),
        "fwd full": lambda s: A.fwd_paged_q4(s["q"].contiguous(), s["cache"], *t(s), s["cu"], max_seqlen_q=26,
                                             max_total_k=70, causal=False, scale=0.1, rounding="rtz"),
    }


def test_both_ways_give_the_same(A, monkeypatch):
    from exact_attention_forward_06_gb300 import _binding
    quick = _binding._quick
    for name, call in _calls(A).items():
        got = []
        for way in (_Only(quick), _Never()):
            monkeypatch.setattr(_binding, "_quick", way)
            s = _state()
            if name not in ("append", "append one", "append q4"):
                A.append_paged_q4(s["q"], s["k"], s["v"], s["cache"], s["table"], s["lens"], s["cu"])
            got.append(call(s))
        assert len(got[0]) == len(got[1]), name
        for a, b in zip(*got):
            assert (a is None) == (b is None), name
            if a is not None:
                assert a.shape == b.shape and a.dtype == b.dtype and a.is_contiguous() and torch.equal(a, b), name
    assert A.device_status()[0] == 0


def test_out_of_order_calls_raise_as_ever(A):
    s = _state()
    t = (s["table"], s["lens"])
    wrong = [
        (TypeError, lambda: A.decode_paged_q4(s["one"].float(), s["cache"], *t)),
        (TypeError, lambda: A.decode_paged_q4(s["one"].cpu(), s["cache"], *t)),
        (TypeError, lambda: A.decode_paged_q4(s["one"], s["cache"], s["table"].long(), s["lens"])),
        (TypeError, lambda: A.decode_paged_q4(None, s["cache"], *t)),
        (ValueError, lambda: A.decode_paged_q4(s["one"][:2], s["cache"], *t)),
        (ValueError, lambda: A.decode_paged_q4(s["one"], s["cache"][..., :2559].contiguous(), *t)),
        (ValueError, lambda: A.decode_paged_q4(s["one"], s["cache"], s["table"].T, s["lens"])),
        (ValueError, lambda: A.decode_paged_q4(s["one"], s["cache"], *t, out=s["one"][:2])),
        (A.AttnError, lambda: A.decode_paged_q4(s["one"], s["cache"], *t, scale=float("nan"))),
        (A.AttnError, lambda: A.decode_paged_q4(s["one"][:, :3].contiguous(), s["cache"], *t)),
        (A.AttnError, lambda: A.decode_paged_q4(s["one"], s["cache"], *t, workspace=s["cache"][0, 0, :256])),
        (ValueError, lambda: A.append_paged(s["q"], s["k"], s["v"], s["kp"], s["vp"][:5], *t, s["cu"])),
        (ValueError, lambda: A.append_paged(s["q"], s["k"], s["v"], s["kp"], s["vp"], *t)),
        (TypeError, lambda: A.append_paged(s["q"], s["k"], s["v"], s["kp"], None, *t, s["cu"])),
        (ValueError, lambda: A.append_paged(None, s["k"], s["v"], s["kp"], s["vp"], *t, s["cu"], q_out=s["one"])),
        (ValueError, lambda: A.append_paged_q4(s["q"], s["k"][:, :1], s["v"][:, :1], s["cache"], *t, s["cu"])),
        (ValueError, lambda: A.append_paged_q4(s["q"], s["k"], s["v"], s["cache"], *t, s["cu"], positions=s["pos1"][:5])),
        (ValueError, lambda: A.append_paged_q4(s["q"], s["k"], s["v"], s["cache"], *t, s["cu"], q_weight=s["w"][:64])),
        (A.AttnError, lambda: A.append_paged_q4(s["q"], s["k"], s["v"], s["cache"], *t, s["cu"], q_weight=s["w"], eps=-1.0)),
        (ValueError, lambda: A.qk_norm_rope(s["x"], s["y"], layout="sbhd")),
        (ValueError, lambda: A.qk_norm_rope(s["x"], s["y"][:1])),
        (A.AttnError, lambda: A.qk_norm_rope(s["qkv"][:, 4:].unfold(1, 128, 128)[:, :2])),    # not 16-byte aligned
        (ValueError, lambda: A.gather_paged_q4(s["cache"], *t, s["cu"][:2], total_k=5)),
        (A.AttnError, lambda: A.gather_paged_q4(s["cache"], *t, s["cu_k"], total_k=0)),
        (ValueError, lambda: A.fwd_paged_q4(s["one"], s["cache"], *t, s["cu"], max_seqlen_q=1, max_total_k=59, rounding="up")),
        (A.AttnError, lambda: A.fwd_paged_q4(s["one"], s["cache"], *t, s["cu"], max_seqlen_q=0, max_total_k=59)),
    ]
    for i, (error, call) in enumerate(wrong):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was taken")
    assert A.device_status()[0] == 0


def test_given_outputs_and_repeated_calls_leave_nothing(A):
    s = _state()
    out, lse = torch.empty_like(s["one"]), torch.empty(B, Hq, device="cuda")
    calls = list(_calls(A).values())
    for call in calls:
        call(s)
    refs = [sys.getrefcount(t) for t in (out, lse, s["one"], s["cache"], s["w"])]
    gc.collect()
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for _ in range(50):
        o, l = A.decode_paged_q4(s["one"], s["cache"], s["table"], s["lens"], out=out, lse=lse)
        assert o is out and l is lse
        for call in calls:
            call(s)
    del o, l
    gc.collect()
    assert [sys.getrefcount(t) for t in (out, lse, s["one"], s["cache"], s["w"])] == refs
    assert torch.cuda.memory_allocated() == held
