"""Failure detection in the prefill's three forms, without a GPU fault.

attn_debug_inject(1) makes the load-issuing warp of the next prefill issue nothing and hand out no work, so every
other warp runs out of its (short) wait budget or leaves on the flag that one of them raised, and the softmax groups
leave by the barrier that their warps share.  The call ends, ATTN_ERR_TIMEOUT is recorded, and the next call gives the
same bits as before."""
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


def _dense(A):
    w = inputs.PrefillWorkload("timeout", 3, 8, 2, 700, 900, causal=True, seed=62)
    q, k, v = (t.cuda() for t in inputs.make_prefill(w))
    return lambda: A.fwd(q, k, v, causal=True, scale=w.scale)


def _packed(A):
    g = torch.Generator().manual_seed(63)
    cu = torch.tensor([0, 300, 301, 900], dtype=torch.int32).cuda()
    q, k, v = (torch.randn(900, h, 128, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    return lambda: A.fwd_varlen(q, k, v, cu, cu, max_seqlen_q=599, max_seqlen_k=599, causal=True)


def _paged(A):
    g = torch.Generator().manual_seed(64)
    kp, vp = (torch.randn(60, 16, 2, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    table = torch.randperm(60, generator=g).to(torch.int32).reshape(2, 30).cuda()
    lens = torch.tensor([470, 200], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 260, 290], dtype=torch.int32).cuda()
    q = torch.randn(290, 4, 128, generator=g).to(torch.bfloat16).cuda()
    return lambda: A.fwd_paged(q, kp, vp, table, lens, cu, max_seqlen_q=260)


@pytest.mark.parametrize("form", [_dense, _packed, _paged])
def test_expired_wait_is_reported_and_the_next_call_is_right(A, form):
    run = form(A)
    good = run()
    assert A.device_status()[0] == 0
    A.set_wait_budget_ns(20_000_000)          # 20 ms
    try:
        A.debug_inject(1)
        run()
        code, site = A.device_status()       # synchronises
        assert code == 4 and site in (19, 20), (code, site)   # a work item or a store command that never came
        assert A.device_status()[0] == 0      # reading clears it
    finally:
        A.debug_inject(0)
        A.set_wait_budget_ns(0)
    again = run()
    assert A.device_status()[0] == 0
    assert all(torch.equal(x, y) for x, y in zip(good, again))
