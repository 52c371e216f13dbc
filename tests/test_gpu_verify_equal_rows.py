"""Verification where the draft's rows are the target's: every drawn token is kept, whatever its number below 1.

p and q of a token then come out of the same numbers in the same order, so they are the same fp32 number x.  Of the largest
number below 1, u = 1 - 2^-24, u x = x - 2^-24 x rounds to a number below x: for x = 2^e it is exact, and for 2^e < x < 2^(e+1)
it lies between half a step and a whole step of 2^(e-23) below x (x well above the smallest normal number, as here)."""
import pytest
import torch

import exact_attention_forward_06_gb300 as A
from test_gpu_verify_tree import call, make, want

pytestmark = pytest.mark.gpu

LAST = 1.0 - 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes,V,temps", [
    ([9, 9, 9], 5000, [1.0]),
    ([16, 1, 7, 12], 1003, [0.7, 1.3]),
    ([40, 3, 25, 40], 131072, [1.0, 0.6]),      # rows summed up by the walk
])
def test_chains_are_kept_whole(sizes, V, temps, dtype):
    d = make(64, sizes, V, "draft", dtype, temps=temps, tree="chain")
    d["draft"] = d["logits"].clone()
    for b in range(len(sizes)):                 # tokens drawn from the very rows
        for i in range(1, sizes[b]):
            row = d["draft"][int(d["cu"][b]) + i - 1].float() / float(d["temperature"][b])
            gen = torch.Generator().manual_seed(1000 * b + i)
            d["tokens"][int(d["cu"][b]) + i] = int(torch.multinomial(torch.softmax(row, -1), 1, generator=gen))
    d["uniforms"][:] = LAST
    path, tokens, counts = (x.cpu() for x in call(d))
    assert A.device_status()[0] == 0
    assert counts.tolist() == sizes
    for b, n in enumerate(sizes):
        assert path[b, :n].tolist() == list(range(n)) and (path[b, n:] == -1).all()
        assert torch.equal(tokens[b, :n - 1], d["tokens"][int(d["cu"][b]) + 1:int(d["cu"][b + 1])])
        assert 0 <= tokens[b, n - 1] < V and (tokens[b, n:] == -1).all()
    if V < 10000:
        assert torch.equal(tokens, want(d)[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_of_siblings_the_first_is_kept(dtype):
    d = make(65, [30, 4, 12], 3001, "draft", dtype, tree="bush")
    d["draft"] = d["logits"].clone()
    d["uniforms"][:] = LAST
    path, tokens, counts = (x.cpu() for x in call(d))
    assert counts.tolist() == [2, 2, 2] and (path[:, :2] == torch.tensor([0, 1])).all()
    assert torch.equal(tokens, want(d)[1])
