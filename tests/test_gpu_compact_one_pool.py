"""compact_paged where keys and values are one pool: every row moves once (equal bit by bit)."""
import pytest
import torch

import exact_attention_forward_06_gb300 as A
from test_gpu_compact_paged import make, moved, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers", [0, 3])
def test_each_row_moves_once(layers):
    """All nodes but the second are kept: each row moves by one place, over the row that moved before it."""
    b, k, _, _, _, _ = make(7, [250, 40, 120], [3, 10, 77], 8, layers)
    paths = [[0] + list(range(2, n)) for n in b.sizes]
    path = torch.full((3, 250), -1, dtype=torch.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    args = [x.cuda() for x in (b.table, b.lens, b.cu, path, counts)]
    want = moved(b, k, paths)
    for _ in range(20):
        pool = k.cuda()
        lens = A.compact_paged(pool, pool, *args)
        assert same(pool.cpu(), want)
    assert lens.tolist() == [252, 49, 196] and A.device_status()[0] == 0
