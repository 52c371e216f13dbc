"""GPU test of calls back to back, without a synchronisation: every call reads what the call before it has just written
(rotated queries, pages, lengths), into the same memory each time, and must give the bits of the same calls one by one."""
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


@pytest.mark.parametrize("n", [1, 37])
def test_steps_see_what_the_step_before_wrote(A, n):
    """Norm and rotation, append, decode, read-back and chunk attention over the same pages and rows, 30 times; n new
    tokens of each of B sequences a step, always into the same last slots."""
    B, Hq, Hkv, steps = 6, 8, 2, 30
    g = torch.Generator().manual_seed(n)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    rope = A.rope_table(R.inv_freq(128))
    lens = torch.tensor([n, 40, 333, 64, 500, 1000], dtype=torch.int32).cuda()
    width = 64
    table = torch.randperm(B * width, generator=g).to(torch.int32).reshape(B, width).cuda()
    cu = (torch.arange(B + 1) * n).to(torch.int32).cuda()
    lens = torch.maximum(lens, torch.full_like(lens, n))
    cu_k = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), lens.cumsum(0).to(torch.int32)])
    total_k = int(cu_k[-1])
    new = [(r(B * n, Hq, 128), r(B * n, Hkv, 128), r(B * n, Hkv, 128)) for _ in range(steps)]
    kp, vp = r(B * width, 16, Hkv, 128), r(B * width, 16, Hkv, 128)
    start = R.pack_pools(kp.cpu(), vp.cpu()).cuda()
    w = r(128)

    def run(sync):
        cache, k16, v16 = start.clone(), kp.clone(), vp.clone()
        q = torch.empty(B * n, Hq, 128, dtype=torch.bfloat16, device="cuda")
        k_new = torch.empty(B * n, Hkv, 128, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(A.decode_q4_workspace_bytes(B, Hq, Hkv, 128, width), dtype=torch.uint8, device="cuda")
        kept = []
        torch.cuda.synchronize()
        for q_in, k_in, v_in in new:
            calls = [lambda: A.qk_norm_rope(q_in, k_in, q_weight=w, k_weight=w, q_out=q, k_out=k_new),
                     lambda: A.append_paged_q4(q, k_new, v_in, cache, table, lens, cu, rope=rope, q_out=q),
                     lambda: A.gather_paged_q4(cache, table, lens, cu_k, total_k=total_k),
                     lambda: A.append_paged(None, k_new, v_in, k16, v16, table, lens, cu, rope=rope),
                     lambda: A.fwd_paged_q4(q, cache, table, lens, cu, max_seqlen_q=n, max_total_k=total_k)]
            if n == 1:
                calls.insert(2, lambda: A.decode_paged_q4(q, cache, table, lens, workspace=ws))
            for call in calls:
                made = call()                     # (q itself, or None, from an append)
                kept += [t for t in made if t is not q and t is not k_new] if isinstance(made, tuple) else []
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return kept + [q, cache, k16, v16]

    one_by_one, back_to_back = run(True), run(False)
    assert A.device_status()[0] == 0
    assert len(one_by_one) == len(back_to_back) > steps
    for i, (a, b) in enumerate(zip(one_by_one, back_to_back)):
        assert torch.equal(a, b), i
