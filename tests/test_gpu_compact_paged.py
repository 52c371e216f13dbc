"""The paged cache cut down to the accepted path (compact_paged): rows are copied, so everything is equal bit by bit."""
import random

import pytest
import torch

import exact_attention_forward_06_gb300 as A
from tree_ref import Batch, ancestors

pytestmark = pytest.mark.gpu


def make(seed, sizes, contexts, Hkv, layers, kind="tree"):
    rng = random.Random(seed)
    b = Batch(seed, sizes, contexts, Hkv, Hkv, kind)
    gen = torch.Generator().manual_seed(seed)
    shape = ((layers,) if layers else ()) + tuple(b.k.shape)
    k, v = (torch.randint(-2 ** 15, 2 ** 15, shape, generator=gen, dtype=torch.int16).view(torch.bfloat16) for _ in range(2))
    paths = [ancestors(t, rng.randrange(len(t))) if t else [] for t in b.trees]
    N = max(1, max(sizes))
    path = torch.full((len(sizes), N), -1, dtype=torch.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    return b, k, v, paths, path, counts


def moved(b, pool, paths):
    """What a pool [..., P, 16, Hkv, 128] holds afterwards."""
    out = pool.clone()
    for s, p in enumerate(paths):
        base = b.lens_list[s] - b.sizes[s]
        for j, node in enumerate(p):
            (to, ts), (of, fs) = ((int(b.table[s, t // 16]), t % 16) for t in (base + j, base + node))
            out[..., to, ts, :, :] = pool[..., of, fs, :, :]
    return out


def call(b, k, v, path, counts, **kw):
    k, v = k.cuda(), v.cuda()
    lens = A.compact_paged(k, v, b.table.cuda(), b.lens.cuda(), b.cu.cuda(), path.cuda(), counts.cuda(), **kw)
    return k.cpu(), v.cpu(), lens.cpu()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("sizes, contexts, Hkv, layers", [
    ([1], [0], 1, 0),
    ([5], [11], 8, 0),
    ([64], [100], 8, 3),
    ([17, 1, 40, 0, 3], [0, 300, 77, 15, 14], 3, 7),
    ([256, 200], [9, 31], 2, 2),
    ([9] * 33, list(range(33)), 1, 5),
    ([30], [2], 5, 1),
])
def test_paths(sizes, contexts, Hkv, layers):
    b, k, v, paths, path, counts = make(1, sizes, contexts, Hkv, layers)
    gk, gv, lens = call(b, k, v, path, counts)
    assert same(gk, moved(b, k, paths)) and same(gv, moved(b, v, paths))
    assert lens.tolist() == [c + len(p) for c, p in zip(contexts, paths)]
    assert A.device_status()[0] == 0


def test_long_paths_whose_rows_overlap():
    """Every node but the root's neighbour is kept: each row moves by one place, over the row before it."""
    b, k, v, _, _, _ = make(2, [250, 40], [3, 10], 2, 2)
    paths = [[0] + list(range(2, 250)), list(range(1, 40))]
    path = torch.full((2, 250), -1, dtype=torch.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    gk, gv, lens = call(b, k, v, path, torch.tensor([249, 39], dtype=torch.int32))
    assert same(gk, moved(b, k, paths)) and same(gv, moved(b, v, paths))
    assert lens.tolist() == [252, 49]


def test_a_path_in_place_and_a_dropped_tree():
    b, k, v, paths, path, counts = make(3, [20, 20], [5, 50], 4, 2, "chain")
    path[0] = torch.arange(20)
    path[1] = -1
    gk, gv, lens = call(b, k, v, path, torch.tensor([20, 0], dtype=torch.int32))
    assert same(gk, k) and same(gv, v) and lens.tolist() == [25, 50]


def test_bad_entries_are_reported_and_left_alone():
    b, k, v, paths, path, counts = make(4, [20, 30, 10], [40, 50, 60], 2, 2, "bush")
    path[:, 0] = 0
    path[:, 1] = torch.tensor([7, 9, 4])
    path[:, 2:] = -1
    counts = torch.tensor([2, 2, 2], dtype=torch.int32)
    paths = [[0, 7], [0, 9], [0, 4]]
    others = [paths[0], [], paths[2]]

    def expect(got, site, lens1):
        gk, gv, lens = got
        assert A.device_status() == (6, site)
        assert same(gk, moved(b, k, others)) and same(gv, moved(b, v, others))
        assert lens.tolist() == [42, lens1, 62]

    for bad in ([0, 0], [3, 2], [-1, 4], [0, 30], [0, 2 ** 31 - 1]):
        p = path.clone()
        p[1, :2] = torch.tensor(bad)
        expect(call(b, k, v, p, counts), 32, 80)
    for n in (-1, 31):
        c = counts.clone()
        c[1] = n
        expect(call(b, k, v, path, c), 32, 80)
    keep = b.lens.clone()
    for n in (29, -1, b.table.shape[1] * 16 + 1):
        b.lens = keep.clone()
        b.lens[1] = n
        expect(call(b, k, v, path, counts), 31, n)
    b.lens = keep
    # a tree wider than path
    expect(call(b, k, v, path[:, :25].contiguous(), counts, total=60), 32, 80)
    # a page outside the pool: the row that it holds does not move
    t = 50 + 9
    page = int(b.table[1, t // 16])
    for bad in (-1, b.k.shape[0]):
        b.table[1, t // 16] = bad
        expect(call(b, k, v, path, counts), 33, 52)
    b.table[1, t // 16] = page


def test_captured_given_output_and_stream():
    b, k, v, paths, path, counts = make(5, [64, 33], [100, 7], 8, 2)
    dk, dv = k.cuda(), v.cuda()
    args = [x.cuda() for x in (b.table, b.lens, b.cu, path, counts)]
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert A.compact_paged(dk, dv, *args, seqlens_out=lens, stream=s) is lens
    s.synchronize()
    assert same(dk.cpu(), moved(b, k, paths)) and lens.tolist() == [100 + len(paths[0]), 7 + len(paths[1])]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.compact_paged(dk, dv, *args, seqlens_out=lens)
    dk.copy_(k), dv.copy_(v), lens.zero_()
    g.replay()
    assert same(dk.cpu(), moved(b, k, paths)) and same(dv.cpu(), moved(b, v, paths))
    assert lens.tolist() == [100 + len(paths[0]), 7 + len(paths[1])]


def test_pools_past_32_bit_offsets():
    """The same batch with its pages at the end of a pool of more than 2^32 elements."""
    b, k, v, paths, path, counts = make(6, [30, 64], [40, 9], 8, 0)
    few = k.shape[0]
    pages = (1 << 18) + few
    dev = []
    for pool in (k, v):
        big = torch.empty((2, pages, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
        big[:, -few:] = pool.cuda()
        dev.append(big)
    table = torch.where(b.table >= 0, b.table + (pages - few), b.table)
    A.compact_paged(*dev, table.cuda(), b.lens.cuda(), b.cu.cuda(), path.cuda(), counts.cuda())
    for got, pool in zip(dev, (k, v)):
        for layer in range(2):
            assert same(got[layer, -few:].cpu(), moved(b, pool, paths))
    assert A.device_status()[0] == 0
    del dev, big, got
    torch.cuda.empty_cache()
