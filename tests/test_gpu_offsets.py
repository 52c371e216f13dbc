"""GPU tests of offsets out of order, which the appends and the read-back must report wherever they stand, and of unusual
ones that are in order, which they must not."""
import pytest
import torch

import cache_ref as R

pytestmark = pytest.mark.gpu
Hkv = 2


@pytest.fixture(scope="module")
def A():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_forward_06_gb300 as attn
    attn.load()
    return attn


MANY = [i // 3 for i in range(3001)]          # 3000 sequences of no or one token


def _swapped(at):
    cu = list(MANY)
    cu[at], cu[at + 3] = cu[at + 3], cu[at]
    return cu


APPEND = [([0, 12, 4], 12, 6), ([3, 1, 12], 12, 6), ([0, 4, 4, 2, 12], 12, 6), ([-1, 5, 12], 12, 6), ([0, 5, 13], 12, 6),
          ([12, 12, 0], 12, 6), (_swapped(6), 1000, 6), (_swapped(1501), 1000, 6), (_swapped(2994), 1000, 6),
          ([0, 5, 12], 12, 0), ([2, 2, 2, 9, 9], 12, 0), ([0, 0], 12, 0), ([12, 12], 12, 0), (MANY, 1000, 0)]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_reports_offsets_out_of_order(A, case, q4):
    cu, total, want = APPEND[case]
    B = len(cu) - 1
    g = torch.Generator().manual_seed(case)
    k, v = (torch.randn(total, Hkv, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    table = torch.arange(B * 2, dtype=torch.int32).reshape(B, 2).cuda()
    lens = torch.full((B,), 20, dtype=torch.int32).cuda()
    off = torch.tensor(cu, dtype=torch.int32).cuda()
    if q4:
        A.append_paged_q4(None, k, v, torch.zeros(B * 2, Hkv, R.BLOCK, dtype=torch.uint8, device="cuda"), table, lens, off)
        assert A.device_status()[0] == want
        return
    kp, vp = (torch.zeros(B * 2, 16, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.append_paged(None, k, v, kp, vp, table, lens, off)
    assert A.device_status()[0] == want
    if want == 0:                             # every token where it belongs, nothing elsewhere
        flat = kp.view(B, 32, Hkv, 128)
        for b in range(0, B, max(1, B // 50)):
            n = cu[b + 1] - cu[b]
            assert torch.equal(flat[b, 20 - n:20], k[cu[b]:cu[b + 1]])
            assert (flat[b, :20 - n] == 0).all() and (flat[b, 20:] == 0).all()


def _many_lens():
    return [b - a for a, b in zip(MANY, MANY[1:])]


GATHER = [([0, 64, 16, 32], [64, 0, 16], 32, 6), ([0, 16, 0, 16], [16, 5, 16], 16, 6), ([16, 0, 32], [16, 32], 32, 6),
          ([0, 16, 16], [16, 5], 16, 6), ([0, 10, 20], [10, -10], 20, 6), (_swapped(1501), _many_lens(), 1000, 6),
          (_swapped(2994), _many_lens(), 1000, 6), (MANY, [*_many_lens()[:-2], 5, 1], 1000, 6),
          ([0, 16, 32], [16, 16], 32, 0), ([3, 3, 19, 19, 20], [0, 16, 0, 1], 32, 0), (MANY, _many_lens(), 1000, 0)]


@pytest.mark.parametrize("case", range(len(GATHER)))
def test_gather_reports_offsets_out_of_order(A, case):
    cu, lens, total, want = GATHER[case]
    B = len(lens)
    g = torch.Generator().manual_seed(100 + case)
    pools = [torch.randn(B * 4, 16, Hkv, 128, generator=g).to(torch.bfloat16) for _ in range(2)]
    table = torch.arange(B * 4, dtype=torch.int32).reshape(B, 4)
    used = table.flatten()[:8].long()         # (packing all 12000 pages takes long: those of two sequences, the others zero)
    cache = torch.zeros(B * 4, Hkv, R.BLOCK, dtype=torch.uint8)
    cache[used] = R.pack_pools(pools[0][used], pools[1][used])
    k, v = (torch.full((total, Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.gather_paged_q4(cache.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                      torch.tensor(cu, dtype=torch.int32).cuda(), k_out=k, v_out=v)
    assert A.device_status()[0] == want
    if want == 0:
        for b in range(0, B, max(1, B // 50)):
            if lens[b]:
                parts = R.read_tokens(cache, table[b], lens[b])
                assert torch.equal(k[cu[b]:cu[b + 1]].cpu(), R.values_bf16(parts[0]))
                assert torch.equal(v[cu[b]:cu[b + 1]].cpu(), R.values_bf16(parts[1]))
        assert (k[:cu[0]] == 7.0).all() and (k[cu[-1]:] == 7.0).all()
