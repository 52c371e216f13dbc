"""Failure detection in the paged decode, without a GPU fault.

attn_debug_inject(2) makes the load-issuing warps of the next decode issue nothing, so the other warps run out of their
(short) wait budget or leave on the flag that one of them raised.  The call ends, ATTN_ERR_TIMEOUT is recorded, and the
next call gives the same bits as before."""
import pytest
import torch

from exact_attention_forward_06_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_06_gb300 as attn
    attn.load()
    return attn


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (4, 2), (8, 2)])     # one, two and four heads a CTA
def test_expired_wait_is_reported_and_the_next_call_is_right(A, Hq, Hkv, append):
    w = inputs.DecodeWorkload("timeout", B=3, Hq=Hq, Hkv=Hkv, max_blocks=80, len_lo=40, len_hi=1200, seed=23)
    q, kp, vp, table, lens = (t.cuda() for t in inputs.make_decode(w))
    new = torch.randn(2, w.B, Hkv, 128, generator=torch.Generator().manual_seed(24)).to(torch.bfloat16).cuda()

    def run():
        if append:
            return A.decode_paged_append(q, new[0], new[1], kp, vp, table, lens - 1)
        return A.decode_paged(q, kp, vp, table, lens)

    good = run()
    assert A.device_status()[0] == 0
    A.set_wait_budget_ns(20_000_000)          # 20 ms
    try:
        A.debug_inject(2)
        run()
        code, site = A.device_status()       # synchronises
        assert code == 4 and site in (8, 9), (code, site)
        assert A.device_status()[0] == 0      # reading clears it, and the request has been taken
    finally:
        A.debug_inject(0)
        A.set_wait_budget_ns(0)
    again = run()
    assert A.device_status()[0] == 0
    assert all(torch.equal(x, y) for x, y in zip(good, again))
