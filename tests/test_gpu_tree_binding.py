"""The binding's quick way (_quick.so) into the tree operators: the same results as the long way for every form of a call,
the long way's errors for calls that are out of order, and nothing left behind by repeated calls."""
import gc

import pytest
import torch

import exact_attention_forward_06_gb300 as A
from exact_attention_forward_06_gb300 import _binding
from test_gpu_quick_binding import _Never, _Only
from test_gpu_verify_tree import make
from tree_ref import Batch

pytestmark = pytest.mark.gpu


def _state():
    b = Batch(1, [5, 9, 2], [60, 20, 0], 8, 2)
    s = dict(q=b.q, k=b.k, v=b.v, table=b.table, lens=b.lens, cu=b.cu, parents=b.parents)
    s["layers"] = torch.stack([b.k, b.k])
    s["path"] = torch.tensor([p + [-1] * (9 - len(p)) for p in ([0, 2, 4], [0, 5], [0, 1])], dtype=torch.int32)
    s["counts"] = torch.tensor([3, 2, 2], dtype=torch.int32)
    for kind in ("greedy", "draft", "top"):
        for name, x in make(2, [5, 9, 2], 700, kind, torch.float32 if kind == "top" else torch.bfloat16).items():
            s[kind + name] = x
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}


def _tree(s, **kw):
    return A.fwd_tree_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["parents"], max_seqlen_q=9, **kw)


def _verify(s, kind, **kw):
    g = lambda n: s[kind + n]  # noqa: E731
    kw.setdefault("logits", g("logits"))
    return A.verify_tree(kw.pop("logits"), g("tokens"), g("parents"), g("cu"), draft_logits=g("draft"),
                         temperature=g("temperature"), uniforms=g("uniforms"), noise=g("noise"), max_seqlen=9, **kw)


def _compact(s, k, v, **kw):
    return [A.compact_paged(s[k], s[v], s["table"], s["lens"], s["cu"], s["path"], s["counts"], total=16, **kw), s[k]]


CALLS = {
    "tree": _tree,
    "tree given": lambda s: _tree(s, scale=0.2, lse=False, rounding="rtz", workspace=torch.empty(
        A.fwd_tree_paged_workspace_bytes(3, 8, 2, 128, 9), dtype=torch.uint8, device="cuda")),
    "verify greedy": lambda s: _verify(s, "greedy"),
    "verify top": lambda s: _verify(s, "top"),
    "verify draft": lambda s: _verify(s, "draft", workspace=torch.empty(
        A.verify_tree_workspace_bytes(3, 16, 700, 9, with_draft=True), dtype=torch.uint8, device="cuda")),
    "verify strided": lambda s: _verify(s, "draft", logits=torch.cat([s["draftlogits"]] * 2, 1)[:, :700]),
    "compact": lambda s: _compact(s, "k", "v"),
    "compact layers": lambda s: _compact(s, "layers", "layers"),
}


def test_both_ways_give_the_same(monkeypatch):
    A.load()
    quick = _binding._quick
    for name, call in CALLS.items():
        got = []
        for way in (_Only(quick), _Never()):
            monkeypatch.setattr(_binding, "_quick", way)
            got.append(call(_state()))
        for a, b in zip(*got):
            assert (a is None) == (b is None), name
            if a is not None:
                assert a.shape == b.shape and a.dtype == b.dtype and a.is_contiguous(), name
                assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)), name
    assert A.device_status()[0] == 0


def test_out_of_order_calls_raise():
    s = _state()
    t = (s["table"], s["lens"], s["cu"])
    d = lambda **kw: {**dict(draft_logits=s["draftdraft"], temperature=s["drafttemperature"],  # noqa: E731
                             uniforms=s["draftuniforms"], noise=s["draftnoise"], max_seqlen=9), **kw}
    v = (s["draftlogits"], s["drafttokens"], s["draftparents"], s["draftcu"])
    wrong = [
        (TypeError, lambda: A.fwd_tree_paged(s["q"].float(), s["k"], s["v"], *t, s["parents"], max_seqlen_q=9)),
        (TypeError, lambda: A.fwd_tree_paged(s["q"], s["k"], s["v"], *t, s["parents"].long(), max_seqlen_q=9)),
        (TypeError, lambda: A.fwd_tree_paged(s["q"], s["k"].cpu(), s["v"], *t, s["parents"], max_seqlen_q=9)),
        (ValueError, lambda: A.fwd_tree_paged(s["q"], s["k"], s["v"], *t, s["parents"][:5], max_seqlen_q=9)),
        (ValueError, lambda: A.fwd_tree_paged(s["q"], s["k"], s["v"][:2], *t, s["parents"], max_seqlen_q=9)),
        (ValueError, lambda: A.fwd_tree_paged(s["q"][:, ::2], s["k"], s["v"], *t, s["parents"], max_seqlen_q=9)),
        (ValueError, lambda: A.fwd_tree_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"][:2], s["parents"])),
        (ValueError, lambda: _tree(s, out=s["q"][:3])),
        (ValueError, lambda: _tree(s, rounding="up")),
        (A.AttnError, lambda: _tree(s, out=s["q"])),
        (A.AttnError, lambda: _tree(s, scale=-1.0)),
        (A.AttnError, lambda: _tree(s, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))),
        (A.AttnError, lambda: A.fwd_tree_paged(s["q"], s["k"], s["v"], *t, s["parents"], max_seqlen_q=257)),
        (TypeError, lambda: A.verify_tree(v[0].half(), *v[1:], **d())),
        (TypeError, lambda: A.verify_tree(v[0].float(), *v[1:], **d())),          # of another type than the draft's
        (TypeError, lambda: A.verify_tree(v[0], v[1].long(), *v[2:], **d())),
        (TypeError, lambda: A.verify_tree(*v, **d(noise=s["draftnoise"].double()))),
        (ValueError, lambda: A.verify_tree(v[0][0], *v[1:], **d())),
        (ValueError, lambda: A.verify_tree(v[0].t(), *v[1:], **d())),
        (ValueError, lambda: A.verify_tree(*v, **d(draft_logits=s["draftdraft"][:, :699]))),
        (ValueError, lambda: A.verify_tree(*v, **d(noise=s["draftnoise"][:2]))),
        (ValueError, lambda: A.verify_tree(*v, **d(uniforms=None))),
        (ValueError, lambda: A.verify_tree(*v, **d(temperature=None))),
        (ValueError, lambda: A.verify_tree(*v, **d(temperature=s["drafttemperature"][:2]))),
        (ValueError, lambda: A.verify_tree(v[0], v[1][:4], *v[2:], **d())),
        (ValueError, lambda: A.verify_tree(*v, **d(), path=s["path"][:2])),
        (A.AttnError, lambda: A.verify_tree(*v, **d(max_seqlen=257))),
        (A.AttnError, lambda: A.verify_tree(*v, **d(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))),
        (TypeError, lambda: A.compact_paged(s["k"], s["v"], *t, s["path"].long(), s["counts"])),
        (ValueError, lambda: A.compact_paged(s["k"][0], s["v"][0], *t, s["path"], s["counts"])),
        (ValueError, lambda: A.compact_paged(s["k"], s["layers"], *t, s["path"], s["counts"])),
        (ValueError, lambda: A.compact_paged(s["k"], s["v"], *t, s["path"][:2], s["counts"])),
        (ValueError, lambda: A.compact_paged(s["k"], s["v"], *t, s["path"], s["counts"], seqlens_out=s["lens"][:2])),
        (A.AttnError, lambda: A.compact_paged(s["k"], s["v"], *t, s["path"], s["counts"], seqlens_out=s["lens"])),
    ]
    for i, (error, call) in enumerate(wrong):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was taken")
    assert A.device_status()[0] == 0


def test_bounds_read_from_the_offsets():
    s = _state()
    a = A.fwd_tree_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["cu"], s["parents"])
    assert torch.equal(a[0], _tree(s)[0])
    g = A.verify_tree(s["greedylogits"], s["greedytokens"], s["greedyparents"], s["greedycu"])
    assert all(torch.equal(x, y) for x, y in zip(g, _verify(s, "greedy")))
    n = A.compact_paged(s["k"], s["v"], s["table"], s["lens"], s["cu"], s["path"], s["counts"], total=16)
    assert n.tolist() == [63, 22, 2]


def test_repeated_calls_leave_nothing():
    s = _state()
    for call in CALLS.values():
        call(s)
    gc.collect()
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for _ in range(30):
        for call in CALLS.values():
            call(s)
    gc.collect()
    assert torch.cuda.memory_allocated() == held
