"""Speculative decoding as it is run: a tree's keys and values into the pages, its attention, the verification, the cache
cut down, step by step, for a small attention model.  Every emitted token has to be the largest logit of the model in 64
bits over all that was emitted before it, to within what bf16 attention leaves open."""
import math
import random

import pytest
import torch

import exact_attention_forward_06_gb300 as A

pytestmark = pytest.mark.gpu

V, HQ, HKV, D = 50, 4, 2, 128


class Model:
    def __init__(self, seed):
        gen = torch.Generator().manual_seed(seed)
        self.q, self.k, self.v = (torch.randn(V, h, D, generator=gen).to(torch.bfloat16).cuda() for h in (HQ, HKV, HKV))
        self.head = (torch.randn(HQ * D, V, generator=gen) / math.sqrt(HQ * D)).cuda()
        self.rope = A.rope_table([10000.0 ** (-i / 64) for i in range(64)])

    def logits(self, attention):
        return attention.float().flatten(1) @ self.head

    def exact(self, tokens):
        """The logits after a sequence of tokens, in 64 bits (rotated keys rounded to bf16, as the cache holds them)."""
        x = torch.tensor(tokens, device="cuda")
        pos = torch.arange(len(tokens), dtype=torch.int32, device="cuda")
        q, k = A.qk_norm_rope(self.q[x], self.k[x], rope=self.rope, positions=pos)
        k, v = k.double().repeat_interleave(2, 1), self.v[x].double().repeat_interleave(2, 1)
        p = torch.softmax(torch.einsum("hd,lhd->hl", q[-1].double(), k) / math.sqrt(D), -1)
        o = torch.einsum("hl,lhd->hd", p, v)
        mass = torch.einsum("hl,lhd->hd", p, v.abs())
        bound = ((2.0 ** -8 + 2e-4) * mass + 2.0 ** -8 * o.abs()).flatten() @ self.head.double().abs()
        return o.flatten() @ self.head.double(), bound


def test_steps():
    model, rng = Model(1), random.Random(1)
    B, steps, blocks = 3, 12, 12
    history = [[rng.randrange(V) for _ in range(n)] for n in (1, 30, 77)]   # the last one is not in the cache yet
    table = torch.randperm(B * blocks, generator=torch.Generator().manual_seed(1)).view(B, blocks).to(torch.int32).cuda()
    k_pages, v_pages = (torch.full((B * blocks, 16, HKV, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = torch.tensor([len(h) - 1 for h in history], dtype=torch.int32, device="cuda")
    # the prompts
    x = torch.tensor(sum((h[:-1] for h in history), []), device="cuda")
    cu = torch.tensor([0] + [len(h) - 1 for h in history]).cumsum(0).to(torch.int32).cuda()
    A.append_paged(None, model.k[x], model.v[x], k_pages, v_pages, table, lens, cu, rope=model.rope)
    accepted = 0
    for step in range(steps):
        # a tree a sequence: the likeliest next tokens of the model itself (sometimes wrong), some noise among them
        trees, tokens, depths = [], [], []
        for b in range(B):
            parent, tok, depth, prefix = [-1], [history[b][-1]], [0], [history[b]]
            for i in range(1, rng.choice([1, 4, 9])):
                up = rng.randrange(max(0, i - 3), i)
                guess = int(model.exact(prefix[up])[0].argmax()) if rng.random() < 0.7 else rng.randrange(V)
                parent.append(up), tok.append(guess), depth.append(depth[up] + 1), prefix.append(prefix[up] + [guess])
            trees.append(parent), tokens.append(tok), depths.append(depth)
        cu = torch.tensor([0] + [len(t) for t in trees]).cumsum(0).to(torch.int32).cuda()
        i32 = lambda rows: torch.tensor(sum(rows, []), dtype=torch.int32, device="cuda")
        pos = i32([[len(h) - 1 + d for d in ds] for h, ds in zip(history, depths)])
        full = lens + (cu[1:] - cu[:-1])
        x = i32(tokens).long()
        q = A.append_paged(model.q[x], model.k[x], model.v[x], k_pages, v_pages, table, full, cu, rope=model.rope,
                           positions=pos)
        out, _ = A.fwd_tree_paged(q, k_pages, v_pages, table, full, cu, i32(trees), max_seqlen_q=9)
        path, new, counts = A.verify_tree(model.logits(out), i32(tokens), i32(trees), cu, max_seqlen=9)
        lens = A.compact_paged(k_pages, v_pages, table, full, cu, path, counts)
        assert A.device_status()[0] == 0
        for b in range(B):
            n = int(counts[b])
            accepted += n - 1
            for t in new[b, :n].tolist():
                ref, bound = model.exact(history[b])
                assert ref[t] + bound[t] >= (ref - bound).max(), (step, b)
                history[b].append(t)
            assert int(lens[b]) == len(history[b]) - 1
    assert accepted >= 5
    # the cache that is left is the one that the tokens make by themselves
    x = torch.tensor([h[-1] for h in history], device="cuda")
    q = A.append_paged(model.q[x], model.k[x], model.v[x], k_pages, v_pages, table, lens + 1, rope=model.rope)
    out, _ = A.decode_paged(q, k_pages, v_pages, table, lens + 1)
    got = model.logits(out).double()
    for b in range(B):
        ref, bound = model.exact(history[b])
        assert ((got[b] - ref).abs() <= bound + 1e-3).all()
