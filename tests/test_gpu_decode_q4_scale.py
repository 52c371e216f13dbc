"""The attention over the 4-bit cache at its largest scales and queries: finite and right."""
import math

import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_06_gb300 as attn
    attn.load()
    return attn


@pytest.mark.parametrize("q_bits,scale_bits", [(0, 93), (26, 93), (27, 92), (60, 59), (118, 1), (119, 0)])
def test_the_likeliest_key_takes_all(A, q_bits, scale_bits):
    """Scores far apart: the key that lies along the query has weight 1 (its own score less itself, so P is exact), all
    others 0, at any such size.  The value then takes its last rounding and fp32's few steps.  The score is a product of
    one channel's terms with the factor, a few steps of 2^-24 each; the other head's scores are at most 1.01 in size
    times 2^-100 scale, so its lse lies that near the logarithm of the number of keys."""
    L = 40
    k = torch.zeros(1, 48, 1, 128)
    k[0, :, 0, 0] = -1.0
    k[0, 17, 0, 0] = 1.0                       # (a group of zeros and one 1: held exactly at its ends)
    v = torch.randn(1, 48, 1, 128, generator=torch.Generator().manual_seed(1))
    pools = [t.view(3, 16, 1, 128).to(torch.bfloat16) for t in (k, v)]
    cache = R.pack_pools(*pools)
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    q = torch.zeros(1, 2, 128)
    q[..., 0] = 2.0 ** q_bits
    q[0, 1, 0] = -2.0 ** -100
    out, lse = A.decode_paged_q4(q.to(torch.bfloat16).cuda(), cache.cuda(), table.cuda(),
                                 torch.tensor([L], dtype=torch.int32).cuda(), scale=2.0 ** scale_bits)
    assert A.device_status()[0] == 0
    kp, vp = R.read_tokens(cache, table[0], L)
    want = R.values(vp)[17, 0]
    score = float(R.values(kp)[17, 0, 0]) * 2.0 ** (q_bits + scale_bits)
    steps = 2.0 ** -20 * (8 * vp[1] + vp[2].abs())[17, 0]
    assert ((out[0, 0].double().cpu() - want).abs() <= R.HALF * want.abs() + steps).all()
    assert abs(float(lse[0, 0]) - score) <= 2.0 ** -20 * abs(score)
    assert torch.isfinite(out[0, 1].float()).all()
    assert abs(float(lse[0, 1]) - math.log(L)) <= 1.01 * 2.0 ** (scale_bits - 100) + 2.0 ** -18
