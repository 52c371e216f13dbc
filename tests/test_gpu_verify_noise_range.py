"""The noise's range in verify_tree, as documented: numbers from 2^-126 to 2^126 count as they are, larger ones and those
that are not positive are never drawn."""
import math

import pytest
import torch

import exact_attention_forward_06_gb300 as A

pytestmark = pytest.mark.gpu

V = 12


def last(noise, kind):
    """The token that a root alone, of equal logits, is followed by."""
    logits = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *x: torch.tensor(x, device="cuda")  # noqa: E731
    _, out, _ = A.verify_tree(logits, i(0), i(-1), i(0, 1), draft_logits=logits if kind == "draft" else None,
                              temperature=f(1.0), uniforms=f(0.5), noise=noise.cuda()[None].contiguous(), max_seqlen=1)
    return int(out[0, 0])


@pytest.mark.parametrize("kind", ["top", "draft"])
def test_range(kind):
    far = torch.full((V,), 2.0 ** 126)
    assert last(far, kind) == 0
    far[7] = 2.0 ** 125
    assert last(far, kind) == 7
    for never in (2.0 ** 127, math.inf, math.nan, 0.0, -1.0, -math.inf):
        x = torch.full((V,), never)
        assert last(x, kind) == -1
        x[9] = 2.0 ** 126
        assert last(x, kind) == 9
    near = torch.full((V,), 2.0 ** -125)
    near[4] = 2.0 ** -126
    assert last(near, kind) == 4
