"""Failure detection in the attention over the 4-bit cache, without a GPU fault.

attn_debug_inject(2) makes two of the four warps of the next attn_decode_paged_q4's CTAs issue no copy: one of them
runs out of its (short) wait budget and raises the CTA's abort flag, the other leaves on the flag, the remaining two
have finished by themselves.  The call ends, ATTN_ERR_TIMEOUT is recorded, and the next call gives the same bits as
before."""
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


# One run a CTA without a merge; cut runs with their merge; equal shares of several runs each; two tiles of heads.
@pytest.mark.parametrize("lens,Hq,Hkv", [([400, 40], 4, 1), ([5000, 33, 70], 4, 1), ([900] * 70, 8, 8), ([3000, 9], 12, 1)])
def test_expired_wait_is_reported_and_the_next_call_is_right(A, lens, Hq, Hkv):
    g = torch.Generator().manual_seed(sum(lens))
    pages = [(x + 15) // 16 for x in lens]
    P = sum(pages)
    pools = [torch.randn(P, 16, Hkv, 128, generator=g).to(torch.bfloat16) for _ in range(2)]
    cache = R.pack_pools(*pools).cuda()
    table = torch.zeros(len(lens), max(pages), dtype=torch.int32)
    off = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(off, off + n)
        off += n
    args = (torch.randn(len(lens), Hq, 128, generator=g).to(torch.bfloat16).cuda(), cache, table.cuda(),
            torch.tensor(lens, dtype=torch.int32).cuda())
    good = A.decode_paged_q4(*args)
    assert A.device_status()[0] == 0
    A.set_wait_budget_ns(20_000_000)          # 20 ms
    try:
        A.debug_inject(2)
        A.fwd(*[torch.zeros(1, 16, 2, 128, dtype=torch.bfloat16, device="cuda")] * 3)
        assert A.device_status()[0] == 0      # a prefill does not take the decode's request
        A.decode_paged_q4(*args)
        code, site = A.device_status()       # synchronises
        assert code == 4 and site in (7, 26), (code, site)
        assert A.device_status()[0] == 0      # reading clears it, and the request has been taken
    finally:
        A.debug_inject(0)
        A.set_wait_budget_ns(0)
    again = A.decode_paged_q4(*args)
    assert A.device_status()[0] == 0
    assert all(torch.equal(x, y) for x, y in zip(good, again))
