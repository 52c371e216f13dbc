"""Plain 64-bit forms of the tree operators, one sequence, node and head at a time."""
import math
import random

import torch

PAGE = 16


def make_tree(rng, n, kind="tree"):
    """Parents of a tree of n nodes: a chain, a bush (all children of the root), several roots, or anything."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "bush":
        return [0 if i else -1 for i in range(n)]
    if kind == "roots":
        return [-1 if i % 3 == 0 else rng.randrange(i) for i in range(n)]
    return [rng.randrange(i // 3, i) if i else -1 for i in range(n)]


def ancestors(parent, i):
    """Node i and the nodes above it, from the top down."""
    out = []
    while i >= 0:
        out.append(i)
        i = parent[i]
    return out[::-1]


class Batch:
    """Trees behind cached contexts in a shuffled pool, as the operators take them (CPU tensors)."""

    def __init__(self, seed, sizes, contexts, Hq, Hkv, kind="tree", pad=2, consecutive=False, d=128):
        rng = random.Random(seed)
        gen = torch.Generator().manual_seed(seed)
        self.sizes, self.Hq, self.Hkv = sizes, Hq, Hkv
        self.lens_list = [n + c for n, c in zip(sizes, contexts)]
        kinds = kind if isinstance(kind, list) else [kind] * len(sizes)
        self.trees = [make_tree(rng, n, k) for n, k in zip(sizes, kinds)]
        T = sum(sizes)
        self.parents = torch.tensor(sum(self.trees, []), dtype=torch.int32)
        self.cu = torch.tensor([0] + sizes).cumsum(0).to(torch.int32)
        self.lens = torch.tensor(self.lens_list, dtype=torch.int32)
        need = [(x + PAGE - 1) // PAGE for x in self.lens_list]
        total = sum(need) + 3
        perm = list(range(total))
        if not consecutive:
            rng.shuffle(perm)
        self.table = torch.full((len(sizes), max(need) + pad), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        self.q = torch.randn(T, Hq, d, generator=gen).to(torch.bfloat16)
        self.k, self.v = (torch.randn(total, PAGE, Hkv, d, generator=gen).to(torch.bfloat16) for _ in range(2))
        # slots past each sequence's end and the pages of no sequence hold anything
        held = torch.zeros(total, PAGE, dtype=torch.bool)
        for b, L in enumerate(self.lens_list):
            t = torch.arange(L)
            held[self.table[b].long()[t // PAGE], t % PAGE] = True
        self.k[~held] = math.nan
        self.v[~held] = math.nan

    def rows(self, b):
        return slice(int(self.cu[b]), int(self.cu[b + 1]))

    def keys(self, b):
        """Keys and values of sequence b, [L, Hkv, d] in 64 bits (pages outside the pool: zeros)."""
        t = torch.arange(self.lens_list[b])
        page = self.table[b].long()[t // PAGE]
        ok = (page >= 0) & (page < self.k.shape[0])
        out = []
        for pool in (self.k, self.v):
            x = pool[page.clamp(0, pool.shape[0] - 1), t % PAGE].double()
            x[~ok] = 0
            out.append(x)
        return out

    def attention(self, scale=None):
        """out [T, Hq, d], lse [Hq, T] and the bound's part sum p |v| [T, Hq, d], in 64 bits."""
        T, Hq, d = self.q.shape
        scale = 1 / math.sqrt(d) if scale is None else scale
        G = Hq // self.Hkv
        out, mass = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
        lse = torch.full((Hq, T), -math.inf, dtype=torch.float64)
        for b, parent in enumerate(self.trees):
            n, L = len(parent), self.lens_list[b]
            if n == 0:
                continue
            k, v = self.keys(b)
            for i in range(n):
                t = int(self.cu[b]) + i
                seen = list(range(L - n)) + [L - n + a for a in ancestors(parent, i)]
                ks, vs = k[seen], v[seen]
                x = torch.einsum("hgd,lhd->hgl", self.q[t].double().unflatten(0, (self.Hkv, G)), ks) * scale
                p = torch.softmax(x, -1)
                out[t] = torch.einsum("hgl,lhd->hgd", p, vs).flatten(0, 1)
                mass[t] = torch.einsum("hgl,lhd->hgd", p, vs.abs()).flatten(0, 1)
                lse[:, t] = torch.logsumexp(x, -1).flatten()
        return out, lse, mass


def verify(logits, tokens, parents, cu, draft, temperature, uniforms, noise, width):
    """path, tokens [B, width] and counts [B]: the walk down each tree, in 64 bits and one step at a time."""
    B = len(cu) - 1
    path_out, tok_out = (torch.full((B, width), -1, dtype=torch.int32) for _ in range(2))
    counts = torch.zeros(B, dtype=torch.int32)
    V = logits.shape[1]

    def masses(row, temp):
        x = [float(v) for v in row]
        x = [-math.inf if math.isnan(v) else min(v, 3.4028234663852886e38) for v in x]
        top = max(x)
        w = [0.0 if v == -math.inf else math.exp((v - top) / temp) if temp != math.inf else 1.0 for v in x]
        total = math.fsum(w)
        return [v / total for v in w] if total > 0 else w

    for b in range(B):
        begin, n = int(cu[b]), int(cu[b + 1] - cu[b])
        if n == 0:
            continue
        temp = 0.0 if temperature is None else float(temperature[b])
        node, path, out = 0, [0], []
        while True:
            children = [i for i in range(node + 1, n) if int(parents[begin + i]) == node]
            hit = None
            if not temp > 0:
                row = [-math.inf if math.isnan(float(v)) else float(v) for v in logits[begin + node]]
                top = max(row)
                last = row.index(top) if top > -math.inf else -1
                for i in children:
                    if last >= 0 and int(tokens[begin + i]) == last:
                        hit = i
                        break
            else:
                p = masses(logits[begin + node], temp)
                q = None if draft is None else masses(draft[begin + node], temp)
                for i in children:
                    x, u = int(tokens[begin + i]), float(uniforms[begin + i])
                    px = p[x] if 0 <= x < V else 0.0
                    if u * (1.0 if q is None else q[x] if 0 <= x < V else 0.0) < px:
                        hit = i
                        break
                    if q is None:
                        rest = [0.0 if j == x else v for j, v in enumerate(p)]
                    else:
                        rest = [max(v - w, 0.0) for v, w in zip(p, q)]
                    total = math.fsum(rest)
                    if total > 0:
                        p = [v / total for v in rest]
                last, best = -1, 0.0
                if hit is None:
                    e = noise[b].tolist()
                    for j, v in enumerate(p):
                        if v > 0 and e[j] > 0 and v / e[j] > best:
                            last, best = j, v / e[j]
            if hit is None:
                out.append(last)
                break
            node = hit
            path.append(node)
            out.append(int(tokens[begin + node]))
        path_out[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        tok_out[b, :len(out)] = torch.tensor(out, dtype=torch.int32)
        counts[b] = len(path)
    return path_out, tok_out, counts
