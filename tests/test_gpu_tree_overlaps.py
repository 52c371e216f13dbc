"""Outputs over inputs, as tensors: both ways into the library refuse them, and nothing is written."""
import pytest
import torch

import exact_attention_forward_06_gb300 as A
from test_gpu_compact_paged import make as make_compact
from test_gpu_verify_tree import make as make_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", [False, True])
def test_verify(stream):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v
         for k, v in make_verify(130, [4, 4, 4], 600, "draft", tree="chain").items()}
    kw = dict(draft_logits=d["draft"], temperature=d["temperature"], uniforms=d["uniforms"], noise=d["noise"], max_seqlen=4)
    if stream:
        kw["stream"] = torch.cuda.current_stream()
    trees = (d["logits"], d["tokens"], d["parents"], d["cu"])
    before = [t.clone() for t in trees]
    both = torch.full((2, 3, 4), 7, dtype=torch.int32, device="cuda")
    for given in (dict(out_tokens=d["tokens"].view(3, 4)), dict(path=d["parents"].view(3, 4)), dict(counts=d["cu"][1:]),
                  dict(counts=d["cu"][:3]), dict(path=both[0], out_tokens=both[0]),
                  dict(path=both[0], counts=both.view(-1)[11:14])):
        with pytest.raises(A.AttnError):
            A.verify_tree(*trees, **kw, **given)
    assert all(torch.equal(a, b) for a, b in zip(before, trees)) and (both == 7).all()
    got = A.verify_tree(*trees, **kw, path=both[0], out_tokens=both[1])
    want = A.verify_tree(*trees, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("stream", [False, True])
def test_compact(stream):
    b, k, v, _, path, counts = make_compact(131, [6, 9], [30, 4], 2, 0)
    k, v, table, lens, cu, path, counts = (x.cuda() for x in (k, v, b.table, b.lens, b.cu, path, counts))
    kw = dict(stream=torch.cuda.current_stream()) if stream else {}
    before = [x.clone() for x in (table, lens, cu, path, counts)]
    for out in (table[0, :2], lens, cu[:2], cu[1:], path[0, :2], path[1, -2:], counts):
        with pytest.raises(A.AttnError):
            A.compact_paged(k, v, table, lens, cu, path, counts, seqlens_out=out, **kw)
    whole = torch.cat([k.flatten(), v.flatten()])
    with pytest.raises(A.AttnError):        # pools that share some of their pages
        A.compact_paged(whole[:k.numel()].view(k.shape), whole[4096:4096 + k.numel()].view(k.shape), table, lens, cu, path,
                        counts, **kw)
    assert all(torch.equal(x, y) for x, y in zip(before, (table, lens, cu, path, counts)))
