"""Measured cases of speculative decoding over the paged KV cache: attention of a
tree of drafted tokens over a cache (fwd_tree_paged), verification of the drafted
tokens against the target's probabilities from given random numbers (verify_tree),
and the cache cut down to the accepted path (compact_paged).

A step of a sequence: its tree's tokens (the last token that was emitted as the
root, node 0, then drafted tokens, each behind its parent) are the last tokens of
its cache.  Their attention gives the model's logits at every node; verification
walks down from the root and emits the drafted tokens that it accepts and one more;
the accepted nodes' keys and values move to the front of the tree's places.

With ``own`` false, ``run`` computes each operator in plain torch operations in
32 bits (probabilities, which are compared with random numbers, in 64); with
``own`` true it calls the package.  ``exact`` gives the same results in 64 bits,
written apart from the plain form.
"""
import math
import random

import torch

own = False
device = "cuda"

D = 128                 # head dimension
PAGE = 16               # tokens per page


# ---------------------------------------------------------------------------
# The cases

def listed():
    return [
        # One sequence with a few drafted tokens in a row behind a short context: latency.
        dict(name="tree_1x5_chain", op="tree", B=1, Hq=32, Hkv=8, n_lo=5, n_hi=5, chain=True, ctx_lo=200, ctx_hi=200,
             mix=11),
        # Small odd trees, five query heads to a KV head, contexts from nothing on.
        dict(name="tree_5seq_g5_ragged", op="tree", B=5, Hq=20, Hkv=4, n_lo=1, n_hi=37, chain=False, ctx_lo=0,
             ctx_hi=700, mix=12),
        # The paged decode workload's lengths, each sequence with four drafted tokens in a row.
        dict(name="tree_32seq_chain", op="tree", B=32, Hq=32, Hkv=8, n_lo=5, n_hi=5, chain=True, ctx_lo=1019,
             ctx_hi=8187, mix=13),
        # Long contexts of few sequences with one KV head for all 32 query heads, trees of odd sizes.
        dict(name="tree_mqa_3x100k", op="tree", B=3, Hq=32, Hkv=1, n_lo=17, n_hi=61, chain=False, ctx_lo=60001,
             ctx_hi=131000, mix=14),
        # A full serving batch with trees of 64 tokens.
        dict(name="tree_32seq_64", op="tree", B=32, Hq=32, Hkv=8, n_lo=64, n_hi=64, chain=False, ctx_lo=960,
             ctx_hi=8128, mix=15),
        # One sequence's five tokens against the largest logit of each row, nothing drawn: latency.
        dict(name="verify_1x5_greedy", op="verify", B=1, V=32768, n_lo=5, n_hi=5, chain=True, kind="greedy",
             dtype="bf16", mix=16),
        # An odd vocabulary in 32 bits, trees whose siblings are drawn from the draft's distribution one after the other.
        dict(name="verify_5seq_tree_fp32", op="verify", B=5, V=50001, n_lo=1, n_hi=29, chain=False, kind="draft",
             dtype="fp32", mix=17),
        # A serving batch: four tokens in a row, drawn from a draft model's distributions.
        dict(name="verify_64seq_chain", op="verify", B=64, V=131072, n_lo=5, n_hi=5, chain=True, kind="draft",
             dtype="bf16", mix=18),
        # Trees of the draft's likeliest tokens.
        dict(name="verify_16seq_tree64", op="verify", B=16, V=131072, n_lo=40, n_hi=64, chain=False, kind="top",
             dtype="bf16", mix=19),
        # One layer of one sequence after a step: latency.
        dict(name="compact_1x64", op="compact", B=1, layers=1, Hkv=8, n_lo=64, n_hi=64, chain=False, ctx_lo=100,
             ctx_hi=100, mix=20),
        # All layers of a serving batch in one pool.
        dict(name="compact_32seq_32layers", op="compact", B=32, layers=32, Hkv=8, n_lo=33, n_hi=64, chain=False,
             ctx_lo=0, ctx_hi=200, mix=21),
        # Odd sizes: three KV heads, seven layers.
        dict(name="compact_13seq_7layers", op="compact", B=13, layers=7, Hkv=3, n_lo=1, n_hi=100, chain=False,
             ctx_lo=0, ctx_hi=333, mix=22),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "verify", "compact"])
    mix = rng.randrange(1 << 20)
    chain = op != "compact" and rng.random() < 0.4    # of tokens in a row nothing moves
    top = _log_int(rng, 1, 12 if chain else 128)
    n = dict(n_lo=max(1, top // rng.choice([1, 1, 2, 5])), n_hi=top, chain=chain, mix=mix)
    if op == "tree":
        # no more than the largest listed case: keys of all heads, and query rows against them
        Hkv = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16, 32] if Hkv == 1 else [1, 2, 3, 4, 5, 6, 8])
        B = _log_int(rng, 1, 32)
        most = min(1100000 // (B * Hkv), 270000000 // (B * Hkv * G * top))
        ctx = _log_int(rng, 1, max(1, min(131000, most - top)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, ctx_lo=ctx // rng.choice([1, 3, 10]), ctx_hi=ctx, **n)
    if op == "verify":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        V = _log_int(rng, 1000, 140000)
        if rng.random() < 0.5:
            V = (V + 63) // 64 * 64
        B = _log_int(rng, 1, max(1, min(64, 64 * 5 * 131072 // (V * top) // (2 if dtype == "fp32" else 1))))
        return dict(op=op, B=B, V=V, kind=rng.choice(["greedy", "draft", "draft", "top"]), dtype=dtype, **n)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    B = _log_int(rng, 1, 32)
    return dict(op=op, B=B, layers=_log_int(rng, 1, max(1, 32 * 32 * 8 // (B * Hkv * 2))), Hkv=Hkv, ctx_lo=0,
                ctx_hi=_log_int(rng, 1, 300), **n)


def _trees(case):
    """Of each sequence, from the case alone: its tree (each node's parent, -1 for the root), its cache's length with
    the tree, and a path down the tree from the root."""
    rng = random.Random(case["mix"])
    out = []
    for _ in range(case["B"]):
        n = rng.randint(case["n_lo"], case["n_hi"])
        # Children lie behind their parent, the early nodes have the most: the depth grows with log n.
        parent = [-1] + [i - 1 if case["chain"] else rng.randrange(i // 3, i) for i in range(1, n)]
        ctx = rng.randint(case["ctx_lo"], case["ctx_hi"]) if "ctx_lo" in case else 0
        node, path = rng.randrange(n), []
        while node >= 0:
            path.append(node)
            node = parent[node]
        out.append((parent, ctx + n, path[::-1]))
    return out


def work(case):
    trees = _trees(case)
    T = sum(len(p) for p, _, _ in trees)
    if case["op"] == "tree":
        Hq, Hkv = case["Hq"], case["Hkv"]
        pairs = 0
        for parent, L, _ in trees:
            depth = []
            for a in parent:
                depth.append(1 if a < 0 else depth[a] + 1)
            pairs += len(parent) * (L - len(parent)) + sum(depth)
        return dict(bytes=sum(L for _, L, _ in trees) * Hkv * 2 * D * 2 + T * (Hq * (2 * D * 2 + 4) + 4),
                    flops=4 * D * Hq * pairs)
    if case["op"] == "verify":
        # The rows that are read depend on what is accepted: at least the root's of every sequence, with the draft's
        # where tokens were drawn from it and the numbers that draw the last token.
        size = 2 if case["dtype"] == "bf16" else 4
        rows = dict(greedy=size, top=size + 4, draft=2 * size + 4)[case["kind"]]
        return dict(bytes=case["B"] * case["V"] * rows + T * 12, flops=case["B"] * case["V"] * 8)
    moved = sum(sum(1 for j, node in enumerate(path) if node != j) for _, _, path in trees)
    return dict(bytes=moved * case["layers"] * case["Hkv"] * 2 * D * 2 * 2 + T * 4, flops=0)


# ---------------------------------------------------------------------------
# What a program has in hand before the call

def _ranks(parent):
    """Of each node, how many of its siblings come before it."""
    seen, out = {}, []
    for a in parent:
        out.append(seen.get(a, 0))
        seen[a] = out[-1] + 1
    return out


def prepare(case, seed):
    gen = torch.Generator(device=device).manual_seed(seed)
    trees = _trees(case)
    B, op = case["B"], case["op"]
    new = [len(p) for p, _, _ in trees]
    lens = [L for _, L, _ in trees]
    T, N = sum(new), max(new)
    s = dict(op=op, B=B, new=new, lens_list=lens, max_new=N)
    s["cu"] = torch.tensor([0] + new, device=device).cumsum(0).to(torch.int32)
    s["parents"] = torch.tensor(sum((p for p, _, _ in trees), []), dtype=torch.int32, device=device)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    if op == "verify":
        V = case["V"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        rank = torch.tensor(sum((_ranks(p) for p, _, _ in trees), []), device=device)
        first = torch.repeat_interleave(s["cu"][:-1].long(), torch.tensor(new, device=device))
        above = first + s["parents"].long().clamp(min=0)           # the parent's row
        K = int(rank.max()) + 1
        if case["kind"] == "draft":
            base = randn(T, V) * 3
            s["logits"] = base.to(dtype)
            # the draft model's logits differ by some noise; its last few entries are padding
            base += randn(T, V) * 0.7
            base[:, V - V // 100:] = -math.inf
            s["draft"] = base.to(dtype)
            cdf = torch.softmax(s["draft"].float(), -1).cumsum(-1)
            at = torch.rand(T, K, generator=gen, device=device) * cdf[:, -1:]
            drawn = torch.searchsorted(cdf, at).clamp(max=V - V // 100 - 1)
            del cdf
        else:
            base = randn(T, V) * 6                                 # the likeliest token has about half of a row
            s["logits"] = base.to(dtype)
            s["draft"] = None
            drawn = (base + randn(T, V)).topk(K, -1).indices       # the draft's likeliest tokens
        del base
        s["tokens"] = drawn[above, rank].to(torch.int32)
        s["temperature"] = s["uniforms"] = s["noise"] = None
        if case["kind"] != "greedy":
            s["temperature"] = torch.ones(B, device=device)
            if case["kind"] == "top":                              # requests of one batch sample as they like
                s["temperature"] = torch.tensor([(1.0, 0.7, 0.0, 1.3)[b % 4] for b in range(B)], device=device)
            s["uniforms"] = torch.rand(T, generator=gen, device=device)
            s["noise"] = torch.empty(B, V, device=device).exponential_(generator=gen)
        return s

    # A block table over a shuffled pool and lengths, as a serving engine keeps them.
    n = [(x + PAGE - 1) // PAGE for x in lens]
    total = sum(n)
    perm = torch.randperm(total, generator=gen, device=device).to(torch.int32)
    slot = torch.arange(max(n), device=device)[None, :]
    begin = torch.tensor([0] + n, device=device).cumsum(0)
    at = (begin[:-1, None] + slot).clamp(max=total - 1)
    s["table"] = torch.where(slot < torch.tensor(n, device=device)[:, None], perm[at], torch.full_like(perm[at], -1))
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=device)
    Hkv = case["Hkv"]
    if op == "compact":
        s["k_pages"], s["v_pages"] = (randn(case["layers"], total, PAGE, Hkv, D).bfloat16() for _ in range(2))
        s["path"] = torch.tensor([p + [-1] * (N - len(p)) for _, _, p in trees], dtype=torch.int32, device=device)
        s["counts"] = torch.tensor([len(p) for _, _, p in trees], dtype=torch.int32, device=device)
        return s
    s["Hkv"], s["Hq"] = Hkv, case["Hq"]
    s["k_pages"], s["v_pages"] = (randn(total, PAGE, Hkv, D).bfloat16() for _ in range(2))
    s["q"] = randn(T, case["Hq"], D).bfloat16()
    if own:
        import exact_attention_forward_06_gb300 as A
        need = A.fwd_tree_paged_workspace_bytes(B, case["Hq"], Hkv, D, N)
        s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=device)
    return s


# ---------------------------------------------------------------------------
# The plain forms

def _plain_tree(s):
    Hq, Hkv = s["Hq"], s["Hkv"]
    G = Hq // Hkv
    outs, lses, begin = [], [], 0
    for b in range(s["B"]):
        n, L = s["new"][b], s["lens_list"][b]
        pages = s["table"][b, :(L + PAGE - 1) // PAGE].long()
        k, v = (x[pages].flatten(0, 1)[:L].transpose(0, 1).float() for x in (s["k_pages"], s["v_pages"]))
        q = s["q"][begin:begin + n].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3).flatten(1, 2)  # [Hkv, G n, 128]
        # a node sees itself and what its parent sees
        parent = s["parents"][begin:begin + n].long()
        step = torch.zeros(n + 1, n + 1, device=q.device)
        step[torch.arange(n, device=q.device), torch.where(parent < 0, n, parent)] = 1
        step[n, n] = 1
        reach = torch.eye(n + 1, device=q.device) + step
        for _ in range(max(1, n.bit_length())):
            reach = (reach @ reach).clamp(max=1)
        seen = torch.cat([torch.ones(n, L - n, dtype=torch.bool, device=q.device), reach[:n, :n] > 0], 1)
        x = torch.matmul(q, k.transpose(-1, -2)).unflatten(1, (G, n)) * (1.0 / math.sqrt(D))
        x = x.masked_fill(~seen, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - m)
        del x
        l = p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(1, 2), v).unflatten(1, (G, n)) / l
        outs.append(o.flatten(0, 1).transpose(0, 1))
        lses.append((m + torch.log(l)).squeeze(-1).flatten(0, 1))
        begin += n
    return [torch.cat(outs).bfloat16().contiguous(), torch.cat(lses, 1).contiguous()]


def _plain_verify(s):
    B, N = s["B"], s["max_new"]
    logits = s["logits"]
    dev = logits.device
    cu, new = s["cu"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    V = logits.shape[1]
    first = cu[:-1]
    temp = torch.zeros(B, device=dev) if s["temperature"] is None else s["temperature"]
    draws = temp > 0
    inv = torch.where(draws, 1.0 / temp.clamp(min=1e-30), torch.ones_like(temp)).double()[:, None]

    def probabilities(x, row):
        x = x[row].double()
        p = torch.exp((x - x.amax(-1, keepdim=True)) * inv)
        return p / p.sum(-1, keepdim=True)

    cur = torch.zeros(B, dtype=torch.long, device=dev)
    count = torch.ones_like(cur)
    path = torch.full((B, N), -1, dtype=torch.int32, device=dev)
    tokens = torch.full((B, N), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    seq = torch.arange(B, device=dev)
    best = logits[first].argmax(-1)
    left = probabilities(logits, first) if s["noise"] is not None else None
    for i in range(1, N):
        row = (first + i).clamp(max=logits.shape[0] - 1)
        child = (i < new) & (s["parents"][row].long() == cur)
        x = s["tokens"][row].long()
        take = x == best
        if left is not None:
            ahead = s["uniforms"][row].double()
            if s["draft"] is not None:
                q = probabilities(s["draft"], first + cur)
                rest = (left - q).clamp(min=0)
                ahead = ahead * q.gather(1, x[:, None])[:, 0]
            else:
                rest = left.scatter(1, x[:, None], 0.0)
            take = torch.where(draws, ahead < left.gather(1, x[:, None])[:, 0], take)
            total = rest.sum(-1, keepdim=True)
            rest = torch.where(total > 0, rest / total, left)
            left = torch.where((child & ~take)[:, None], rest, left)
        take = take & child
        cur = torch.where(take, i, cur)
        at = count.clamp(max=N - 1)
        path[seq, at] = torch.where(take, i, path[seq, at].long()).int()
        tokens[seq, at - 1] = torch.where(take, x, tokens[seq, at - 1].long()).int()
        count = count + take.long()
        best = torch.where(take, logits[row].argmax(-1), best)
        if left is not None:
            left = torch.where(take[:, None], probabilities(logits, row), left)
    if left is not None:
        best = torch.where(draws, (left / s["noise"].double()).argmax(-1), best)
    tokens[seq, count - 1] = best.int()
    return [path, tokens, count.int()]


def _plain_compact(s):
    path, counts, N = s["path"].long(), s["counts"].long(), s["max_new"]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    j = torch.arange(N, device=path.device)[None]
    kept = j < counts[:, None]
    base = (s["lens"].long() - new)[:, None]
    src = base + torch.where(kept, path, torch.zeros_like(path))
    dst = base + torch.where(kept, j, torch.zeros_like(path))     # past the path: the root onto itself
    src_page, dst_page = (s["table"].long().gather(1, t // PAGE) for t in (src, dst))
    for pool in (s["k_pages"], s["v_pages"]):
        pool[:, dst_page, dst % PAGE] = pool[:, src_page, src % PAGE]
    return [s["k_pages"], s["v_pages"], (s["lens"].long() - new + counts).int()]


def run(s):
    op = s["op"]
    if not own:
        return dict(tree=_plain_tree, verify=_plain_verify, compact=_plain_compact)[op](s)
    import exact_attention_forward_06_gb300 as A
    if op == "tree":
        return A.fwd_tree_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["parents"],
                                max_seqlen_q=s["max_new"], workspace=s["workspace"])
    if op == "verify":
        return A.verify_tree(s["logits"], s["tokens"], s["parents"], s["cu"], draft_logits=s["draft"],
                             temperature=s["temperature"], uniforms=s["uniforms"], noise=s["noise"],
                             max_seqlen=s["max_new"])
    lens = A.compact_paged(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], s["path"], s["counts"])
    return [s["k_pages"], s["v_pages"], lens]


# ---------------------------------------------------------------------------
# The operators' definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    trees = _trees(case)
    op, begin = case["op"], 0
    if op == "tree":
        Hq, Hkv = case["Hq"], case["Hkv"]
        outs, lses = [], []
        for b, (parent, L, _) in enumerate(trees):
            n = len(parent)
            t = torch.arange(L, device=device)
            page = s["table"][b].long()[t // PAGE]
            k, v = (x[page, t % PAGE].double() for x in (s["k_pages"], s["v_pages"]))      # [L, Hkv, 128]
            hidden = torch.zeros(n, L, dtype=torch.bool)
            for i in range(n):
                hidden[i, L - n:] = True
                a = i
                while a >= 0:
                    hidden[i, L - n + a] = False
                    a = parent[a]
            hidden = hidden.to(device)
            o = torch.empty(n, Hq, D, dtype=torch.float64, device=device)
            l = torch.empty(Hq, n, dtype=torch.float64, device=device)
            for h in range(Hq):
                g = h * Hkv // Hq
                x = s["q"][begin:begin + n, h].double() @ k[:, g].T / math.sqrt(D)
                x[hidden] = -math.inf
                l[h] = torch.logsumexp(x, -1)
                o[:, h] = torch.softmax(x, -1) @ v[:, g]
            outs.append(o)
            lses.append(l)
            begin += n
        return [torch.cat(outs), torch.cat(lses, 1)]
    N = s["max_new"]
    if op == "compact":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        k0, v0, lens = s["k_pages"], s["v_pages"], []
        table = s["table"].tolist()
        for b, (parent, L, path) in enumerate(trees):
            base = L - len(parent)
            for j, node in enumerate(path):
                to, of = (table[b][(base + x) // PAGE] for x in (j, node))
                k[:, to, (base + j) % PAGE] = k0[:, of, (base + node) % PAGE].double()
                v[:, to, (base + j) % PAGE] = v0[:, of, (base + node) % PAGE].double()
            lens.append(base + len(path))
        return [k, v, torch.tensor(lens, device=device)]
    paths, emitted, counts = [], [], []
    tokens = s["tokens"].tolist()
    for b, (parent, _, _) in enumerate(trees):
        temp = 0.0 if s["temperature"] is None else float(s["temperature"][b])
        node, path, out = 0, [0], []
        while True:
            row = begin + node
            children = [i for i in range(node + 1, len(parent)) if parent[i] == node]
            if temp <= 0:
                last = int(s["logits"][row].argmax())
                hit = [i for i in children if tokens[begin + i] == last]
            else:
                left = torch.softmax(s["logits"][row].double() / temp, -1)
                draft = None if s["draft"] is None else torch.softmax(s["draft"][row].double() / temp, -1)
                hit = []
                for i in children:
                    x, u = tokens[begin + i], float(s["uniforms"][begin + i])
                    if u * (1.0 if draft is None else float(draft[x])) < float(left[x]):
                        hit = [i]
                        break
                    rest = left.clone()
                    if draft is None:
                        rest[x] = 0
                    else:
                        rest = torch.relu(rest - draft)
                    if float(rest.sum()) > 0:
                        left = rest / rest.sum()
                last = None if hit else int((left / s["noise"][b].double()).argmax())
            if not hit:
                out.append(last)
                break
            node = hit[0]
            path.append(node)
            out.append(tokens[begin + node])
        paths.append(path + [-1] * (N - len(path)))
        emitted.append(out + [-1] * (N - len(out)))
        counts.append(len(path))
        begin += len(parent)
    return [torch.tensor(x, device=device) for x in (paths, emitted, counts)]
