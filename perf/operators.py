"""Measured cases of the operators around the paged KV cache: head norms with the
position rotation (qk_norm_rope), the same on the way into the paged cache
(append_paged) and into a cache held in 4 bits (append_paged_q4, read back with
gather_paged_q4), and attention over that cache for single tokens
(decode_paged_q4) and for prompt chunks (fwd_paged_q4).

With ``own`` false, ``run`` computes each operator in plain torch operations in
32 bits (angles in 64); with ``own`` true it calls the package.  ``exact`` gives
the same results in 64 bits, written apart from the plain form.
"""
import math
import random

import torch

own = False
device = "cuda"

D = 128                 # head dimension
PAGE = 16               # tokens per page
GROUP = 32              # channels that share one scale and one center in the 4-bit cache
NG = D // GROUP
BLOCK = 2560            # bytes of one page of one KV head in the 4-bit cache
EPS = 1e-6


# ---------------------------------------------------------------------------
# The cases

def listed():
    return [
        # A video transformer's self-attention inputs: 21 x 30 x 52 latent positions, 12 heads, three
        # position axes (time, height, width), both norms.
        dict(name="norm_rope_video_32760", op="norm_rope", B=1, S=32760, Hq=12, Hkv=12, axes=3, R=128, inter=False,
             norm=True, bhsd=False, far=64),
        # A short odd batch taken out of one fused projection as strided BHSD views, interleaved pairs over part
        # of the head dimension, far positions, no norm.
        dict(name="norm_rope_bhsd_3x257", op="norm_rope", B=3, S=257, Hq=32, Hkv=8, axes=1, R=96, inter=True,
             norm=False, bhsd=True, far=1000000),
        # One decode step's new tokens of 32 sequences on their way into the cache: latency.
        dict(name="append_step_32seq", op="append", B=32, Hq=32, Hkv=8, chunk_lo=1, chunk_hi=1, ctx_lo=1023,
             ctx_hi=8191, R=128, inter=False, norm=True, mix=11),
        # Prompt chunks of 16 sequences on contexts of up to 6144 cached tokens.
        dict(name="append_chunks_16seq", op="append", B=16, Hq=32, Hkv=8, chunk_lo=256, chunk_hi=2048, ctx_lo=0,
             ctx_hi=6144, R=128, inter=False, norm=True, mix=12),
        # A few short ragged chunks into the 4-bit cache, read back for the attention of the chunk.
        dict(name="append_q4_5seq_ragged", op="append_q4", B=5, Hq=6, Hkv=2, chunk_lo=1, chunk_hi=37, ctx_lo=0,
             ctx_hi=200, R=64, inter=True, norm=False, mix=13),
        # Prompt chunks of 16 sequences into the 4-bit cache, the whole caches read back.
        dict(name="append_q4_chunks_16seq", op="append_q4", B=16, Hq=32, Hkv=8, chunk_lo=256, chunk_hi=2048,
             ctx_lo=0, ctx_hi=6144, R=128, inter=False, norm=True, mix=14),
        # One short sequence: the smallest decode call, latency.
        dict(name="decode_q4_1x100", op="decode_q4", B=1, Hq=32, Hkv=8, len_lo=100, len_hi=100, mix=15),
        # The paged decode workload's shape: 32 sequences of 1024 to 8192 tokens.
        dict(name="decode_q4_32seq", op="decode_q4", B=32, Hq=32, Hkv=8, len_lo=1024, len_hi=8192, mix=16),
        # Long contexts of few sequences with one KV head for all 32 query heads: few CTAs without a key split.
        dict(name="decode_q4_mqa_3x100k", op="decode_q4", B=3, Hq=32, Hkv=1, len_lo=60001, len_hi=131072, mix=17),
        # A full serving batch with eight query heads to a KV head, lengths from nothing to 16384.
        dict(name="decode_q4_64seq_g8", op="decode_q4", B=64, Hq=64, Hkv=8, len_lo=0, len_hi=16384, mix=18),
        # Short ragged chunks of three sequences against small 4-bit caches: latency.
        dict(name="prefill_q4_3seq_ragged", op="prefill_q4", B=3, Hq=8, Hkv=2, chunk_lo=1, chunk_hi=40, ctx_lo=0,
             ctx_hi=300, causal=True, mix=19),
        # Chunked prefill: 8 sequences, chunks of up to 1024 on contexts of up to 7168 in the 4-bit cache.
        dict(name="prefill_q4_8seq", op="prefill_q4", B=8, Hq=32, Hkv=8, chunk_lo=128, chunk_hi=1024, ctx_lo=0,
             ctx_hi=7168, causal=True, mix=20),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "append_q4", "decode_q4", "decode_q4", "prefill_q4"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 6, 8])
    mix = rng.randrange(1 << 20)
    R = rng.choice([32, 64, 96, 128])
    inter = rng.random() < 0.4
    norm = rng.random() < 0.6
    if op == "norm_rope":
        tokens = _log_int(rng, 1, 32760 * 24 // (Hq + Hkv))
        B = rng.choice([1, 1, 2, 3])
        return dict(op=op, B=B, S=max(1, tokens // B), Hq=Hq, Hkv=Hkv, axes=rng.choice([1, 1, 2, 3]), R=R, inter=inter,
                    norm=norm, bhsd=rng.random() < 0.4, far=_log_int(rng, 64, 1000000))
    # no more than the largest listed case of the operator: new head rows, keys of all heads, visible pairs of all heads
    if op in ("append", "append_q4"):
        B = _log_int(rng, 1, 16)
        chunk = _log_int(rng, 1, min(2048, 880000 // (B * (Hq + 2 * Hkv))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, chunk_lo=max(1, chunk // 4), chunk_hi=chunk, ctx_lo=0,
                    ctx_hi=_log_int(rng, 1, 6000), R=R, inter=inter, norm=norm, mix=mix)
    if op == "decode_q4":
        B = _log_int(rng, 1, 64)
        top = _log_int(rng, 1, min(131072, 64 * 8192 * 8 // (B * Hkv)))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, len_lo=top // rng.choice([1, 3, 10]), len_hi=top, mix=mix)
    B = _log_int(rng, 1, 8)
    chunk = _log_int(rng, 1, 1000)
    ctx = _log_int(rng, 1, max(1, min(7000, 550000000 // (B * chunk * Hq) - chunk)))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, chunk_lo=max(1, chunk // 4), chunk_hi=chunk, ctx_lo=0, ctx_hi=ctx,
                causal=rng.random() < 0.8, mix=mix)


def _lengths(case):
    """(new tokens, tokens in the cache with the new ones) of each sequence, from the case alone."""
    rng = random.Random(case["mix"])
    if case["op"] == "decode_q4":
        lens = [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["B"])]
        return [1] * case["B"], lens
    new = [rng.randint(case["chunk_lo"], case["chunk_hi"]) for _ in range(case["B"])]
    return new, [n + rng.randint(case["ctx_lo"], case["ctx_hi"]) for n in new]


def work(case):
    op, Hq, Hkv = case["op"], case["Hq"], case["Hkv"]
    row = D * 2
    if op == "norm_rope":
        T = case["B"] * case["S"]
        return dict(bytes=T * (2 * (Hq + Hkv) * row + 4 * case["axes"]), flops=T * (Hq + Hkv) * D * 6)
    new, lens = _lengths(case)
    T, L = sum(new), sum(lens)
    if op == "append":
        return dict(bytes=T * 2 * (Hq + 2 * Hkv) * row, flops=T * (Hq + Hkv) * D * 6)
    q4_token = Hkv * BLOCK // PAGE
    if op == "append_q4":
        return dict(bytes=T * ((2 * Hq + 2 * Hkv) * row + q4_token) + L * (q4_token + 2 * Hkv * row),
                    flops=T * (Hq + 2 * Hkv) * D * 6 + L * Hkv * D * 4)
    if op == "decode_q4":
        return dict(bytes=L * q4_token + case["B"] * Hq * (2 * row + 4), flops=4 * L * Hq * D)
    pairs = sum(n * (k - n) + n * (n + 1) / 2 if case["causal"] else n * k for n, k in zip(new, lens))
    return dict(bytes=L * q4_token + T * Hq * (2 * row + 4), flops=4 * pairs * Hq * D)


# ---------------------------------------------------------------------------
# What a program has in hand before the call

def _inv_freq(R, axes):
    """Radians per position of each pair, and its axis: as many pairs to each axis as go, the rest to axis 0."""
    n = R // 2
    if axes == 1:
        return [10000.0 ** (-2.0 * i / R) for i in range(n)], [0] * n
    per = n // axes
    counts = [n - per * (axes - 1)] + [per] * (axes - 1)
    freq, axis = [], []
    for a, c in enumerate(counts):
        freq += [10000.0 ** (-i / c) for i in range(c)]
        axis += [a] * c
    return freq, axis


def _rotation(s, R, axes, inter, norm, gen):
    freq, axis = _inv_freq(R, axes)
    s["inter"] = inter
    s["freq"] = torch.tensor(freq, dtype=torch.float64, device=device)
    s["axis"] = torch.tensor(axis, dtype=torch.int64, device=device)
    s["qw"] = s["kw"] = None
    if norm:
        s["qw"], s["kw"] = ((torch.rand(D, generator=gen, device=device) + 0.5).bfloat16() for _ in range(2))
    if own:
        import exact_attention_forward_06_gb300 as A
        s["rope"] = A.rope_table(freq, axis, device=device)


def _pages(s, lens, gen):
    """A block table over a shuffled pool, lengths and offsets, as a serving engine keeps them."""
    n = [(x + PAGE - 1) // PAGE for x in lens]
    total = max(1, sum(n))
    perm = torch.randperm(total, generator=gen, device=device).to(torch.int32)
    width = max(1, max(n))
    slot = torch.arange(width, device=device)[None, :]
    first = torch.tensor([0] + n, device=device).cumsum(0)
    count = torch.tensor(n, device=device)[:, None]
    at = (first[:-1, None] + slot).clamp(max=total - 1)
    s["table"] = torch.where(slot < count, perm[at], torch.full_like(perm[at], -1)).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=device)
    s["num_pages"] = total
    s["max_len"] = max(lens)
    s["total_k"] = sum(lens)
    s["cu_k"] = torch.tensor([0] + lens, device=device).cumsum(0).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=device).manual_seed(seed)
    op, B, Hq, Hkv = case["op"], case["B"], case["Hq"], case["Hkv"]
    s = dict(op=op, B=B, Hq=Hq, Hkv=Hkv)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    if op == "norm_rope":
        S = case["S"]
        qkv = randn(B, S, (Hq + 2 * Hkv) * D).bfloat16()   # one fused projection's output
        q = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        k = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        s["layout"] = "bhsd" if case["bhsd"] else "bshd"
        s["q"], s["k"] = (q.transpose(1, 2), k.transpose(1, 2)) if case["bhsd"] else (q, k)
        pos = torch.randint(0, case["far"], (case["axes"], B, S), generator=gen, device=device)
        s["pos"] = pos.to(torch.int32)
        _rotation(s, case["R"], case["axes"], case["inter"], case["norm"], gen)
        return s

    new, lens = _lengths(case)
    _pages(s, lens, gen)
    T = sum(new)
    s["cu"] = torch.tensor([0] + new, device=device).cumsum(0).to(torch.int32)
    s["max_new"] = max(new)
    P = s["num_pages"]
    if op in ("append", "append_q4"):
        qkv = randn(T, (Hq + 2 * Hkv) * D).bfloat16()
        s["q"] = qkv[:, :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
        _rotation(s, case["R"], 1, case["inter"], case["norm"], gen)
        if op == "append":
            s["k_pages"], s["v_pages"] = (randn(P, PAGE, Hkv, D).bfloat16() for _ in range(2))
            return s
    else:
        s["q"] = randn(T, Hq, D).bfloat16()
        s["causal"] = case.get("causal", True)
    s["cache"] = _pack(randn(P, PAGE, Hkv, D).bfloat16(), randn(P, PAGE, Hkv, D).bfloat16())
    if own:
        import exact_attention_forward_06_gb300 as A
        if op == "decode_q4":
            need = A.decode_q4_workspace_bytes(B, Hq, Hkv, D, s["table"].shape[1])
            s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=device)
        if op == "prefill_q4":
            need = A.fwd_paged_q4_workspace_bytes(B, Hkv, D, s["total_k"])
            s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device=device)
    return s


# ---------------------------------------------------------------------------
# The 4-bit cache's bytes in plain torch

def _byte_map():
    """Place in a block of each of a token's 160 bytes (64 of key codes, 64 of value codes, then 8 each of key
    scales, key centers, value scales and value centers), for the page's 16 tokens: [16, 160]."""
    t = torch.arange(PAGE, device=device)[:, None]
    i = torch.arange(64, device=device)[None, :]
    word, byte = i // 4, i % 4
    k = t * 64 + (word % 4) * 16 + (word // 4) * 4 + byte
    g, r, b = i // 16, (i % 16) // 2, i % 2
    v = 1024 + r * 128 + (t % 8) // 2 * 32 + (t // 8 ^ (r & 1)) * 16 + t % 2 * 8 + g * 2 + b
    j = torch.arange(8, device=device)[None, :]
    return torch.cat([k, v, 2048 + t * 8 + j, 2176 + t * 8 + j, 2304 + t * 8 + j,
                      2432 + j // 2 * 32 + t * 2 + j % 2], 1)


def _quantise(x):
    """bf16 [..., 128] -> codes uint8 [..., 128], scales and centers bf16 [..., 4]."""
    g = x.float().unflatten(-1, (NG, GROUP))
    hi, lo = g.amax(-1), g.amin(-1)
    z = (0.5 * hi + 0.5 * lo).bfloat16()
    zf = z.float()
    s = (torch.maximum(hi - zf, zf - lo) * torch.tensor(2.0 / 15.0, dtype=torch.float32, device=x.device)).bfloat16()
    sf = s.float()[..., None]
    n = ((g - zf[..., None]) / sf + 7.5).round().clamp(0, 15)
    n = torch.where(sf > 0, n, torch.zeros_like(n))
    return n.flatten(-2).to(torch.uint8), s, z


def _token_bytes(k, v):
    """bf16 k, v [..., 128] -> the 160 bytes of each token and head."""
    parts, tail = [], []
    for x in (k, v):
        n, s, z = _quantise(x)
        parts.append(n[..., 0::2] | (n[..., 1::2] << 4))
        tail += [s.contiguous().view(torch.uint8), z.contiguous().view(torch.uint8)]
    return torch.cat(parts + tail, -1)


def _pack(k, v):
    """bf16 [P, 16, Hkv, 128] pools -> the 4-bit cache [P, Hkv, 2560] uint8."""
    b = _token_bytes(k, v).transpose(1, 2).flatten(2)   # [P, Hkv, 16 * 160]
    out = torch.empty_like(b)
    out[..., _byte_map().flatten()] = b
    return out


def _unpack(blocks):
    """uint8 [..., 2560] -> k, v fp32 [..., 16, 128]."""
    b = blocks[..., _byte_map().flatten()].unflatten(-1, (PAGE, 160))
    out = []
    for i in (0, 1):
        c = b[..., 64 * i:64 * i + 64]
        n = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
        p = b[..., 128 + 16 * i:144 + 16 * i].contiguous().view(torch.bfloat16).float()
        s, z = p[..., :NG, None], p[..., NG:, None]
        out.append((z + s * (n.unflatten(-1, (NG, GROUP)) - 7.5)).flatten(-2))
    return out


# ---------------------------------------------------------------------------
# The plain forms

def _norm_rotate(x, w, pos, s):
    """x [tokens, H, 128] bf16, pos int [axes, tokens] -> fp32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    angle = pos[s["axis"]].double().T * s["freq"]        # [tokens, R / 2]
    cos, sin = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    R = 2 * s["freq"].numel()
    if s["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _slots(s, T):
    """Of each new token: its position in its sequence, its page and its row there."""
    t = torch.arange(T, device=device)
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    pos = s["lens"].long()[seq] - new[seq] + t - s["cu"].long()[seq]
    return pos, s["table"].long()[seq, pos // PAGE], pos % PAGE


def _cached(s):
    """The cache's keys and values by sequence, fp32 [B, Hkv, L, 128] (rows past a sequence's end arbitrary)."""
    blocks = s["cache"][s["table"].long().clamp(min=0)]  # [B, width, Hkv, 2560]
    k, v = _unpack(blocks)
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)


def _attend(q, k, v, seen):
    """q [B, Hkv, rows, 128], k and v [B, Hkv, L, 128], seen [B, 1, rows, L] -> out, lse; a row that sees nothing
    gives 0 and -inf."""
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    del x
    l = p.sum(-1, keepdim=True)
    # a key that a row does not see has p = 0, but its value row may be past a sequence's end: the block holds
    # codes and finite scales there
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    return o, (m + torch.log(l)).squeeze(-1)


def _plain(s):
    op, Hq, Hkv, B = s["op"], s["Hq"], s["Hkv"], s["B"]
    if op == "norm_rope":
        out = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = x.transpose(1, 2) if s["layout"] == "bhsd" else x
            y = _norm_rotate(y.flatten(0, 1), w, s["pos"].flatten(1), s).bfloat16().unflatten(0, (x.shape[0], -1))
            out.append((y.transpose(1, 2) if s["layout"] == "bhsd" else y).contiguous())
        return out
    if op in ("append", "append_q4"):
        pos, page, row = _slots(s, s["q"].shape[0])
        q = _norm_rotate(s["q"], s["qw"], pos[None], s).bfloat16()
        k = _norm_rotate(s["k"], s["kw"], pos[None], s).bfloat16()
        if op == "append":
            s["k_pages"][page, row] = k
            s["v_pages"][page, row] = s["v"]
            return [q, s["k_pages"], s["v_pages"]]
        h = torch.arange(Hkv, device=device)[None, :, None]
        s["cache"][page[:, None, None], h, _byte_map()[row][:, None]] = _token_bytes(k, s["v"])
        keys, values = _cached(s)
        L = keys.shape[2]
        held = torch.arange(L, device=device)[None] < s["lens"][:, None]
        return [q, keys.transpose(1, 2)[held].bfloat16(), values.transpose(1, 2)[held].bfloat16()]
    k, v = _cached(s)
    if op == "prefill_q4":   # a chunk attends to the cache as it is read back: rounded to bf16 once
        k, v = k.bfloat16().float(), v.bfloat16().float()
    L = k.shape[2]
    key = torch.arange(L, device=device)
    G = Hq // Hkv
    if op == "decode_q4":
        seen = (key[None] < s["lens"][:, None])[:, None, None]
        o, lse = _attend(s["q"].float().unflatten(1, (Hkv, G)), k, v, seen)
        return [o.flatten(1, 2).bfloat16(), lse.flatten(1, 2)]
    # chunks, padded to the longest: row i of sequence b sees keys up to lens[b] - new[b] + i
    N = s["max_new"]
    i = torch.arange(N, device=device)[None]
    new = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    there = i < new
    token = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    last = s["lens"].long()[:, None] - new + i if s["causal"] else (s["lens"].long()[:, None] - 1).expand(B, N)
    last = torch.minimum(last, s["lens"].long()[:, None] - 1)
    q = s["q"].float()[token].unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4)    # [B, Hkv, G, N, 128]
    seen = (key[None, None] <= last[..., None])[:, None, None].expand(B, 1, G, N, L).flatten(2, 3)
    o, lse = _attend(q.flatten(2, 3), k, v, seen)
    o = o.unflatten(2, (G, N)).permute(0, 3, 1, 2, 4).flatten(2, 3)[there]
    lse = lse.unflatten(2, (G, N)).permute(0, 3, 1, 2).flatten(2, 3)[there]
    return [o.bfloat16(), lse.T.contiguous()]


def run(s):
    if not own:
        return _plain(s)
    import exact_attention_forward_06_gb300 as A
    op = s["op"]
    if op == "norm_rope":
        return A.qk_norm_rope(s["q"], s["k"], rope=s["rope"], positions=s["pos"], q_weight=s["qw"], k_weight=s["kw"],
                              eps=EPS, interleaved=s["inter"], layout=s["layout"])
    if op == "append":
        q = A.append_paged(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"],
                           rope=s["rope"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=s["inter"])
        return [q, s["k_pages"], s["v_pages"]]
    if op == "append_q4":
        q = A.append_paged_q4(s["q"], s["k"], s["v"], s["cache"], s["table"], s["lens"], s["cu"], rope=s["rope"],
                              q_weight=s["qw"], k_weight=s["kw"], eps=EPS, interleaved=s["inter"])
        k, v = A.gather_paged_q4(s["cache"], s["table"], s["lens"], s["cu_k"], total_k=s["total_k"])
        return [q, k, v]
    if op == "decode_q4":
        return A.decode_paged_q4(s["q"], s["cache"], s["table"], s["lens"], workspace=s["workspace"])
    return A.fwd_paged_q4(s["q"], s["cache"], s["table"], s["lens"], s["cu"], max_seqlen_q=s["max_new"],
                          max_total_k=s["total_k"], causal=s["causal"], workspace=s["workspace"])


# ---------------------------------------------------------------------------
# The operators' definitions in 64 bits

def _exact_head(x, w, pos, freq, axis, inter):
    """x [..., 128], pos [axes, ...] (broadcast over heads by the caller) in 64 bits, pair by pair."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + EPS) * w.double()
    z = y.clone()
    n = len(freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + n)
        t = pos[axis[i]].double() * freq[i]
        z[..., a] = y[..., a] * torch.cos(t) - y[..., b] * torch.sin(t)
        z[..., b] = y[..., b] * torch.cos(t) + y[..., a] * torch.sin(t)
    return z


def _exact_held(x):
    """What the 4-bit cache holds for the bf16 vectors x [..., 128], in 64 bits."""
    parts = []
    for g in x.double().split(GROUP, -1):
        top, low = g.max(-1, keepdim=True).values, g.min(-1, keepdim=True).values
        mid = ((top + low) / 2).to(torch.bfloat16).double()
        step = (torch.maximum(top - mid, mid - low) / 7.5).to(torch.bfloat16).double()
        code = torch.clamp(torch.round((g - mid) / torch.where(step > 0, step, torch.ones_like(step)) + 7.5), 0, 15)
        parts.append(torch.where(step > 0, mid + (code - 7.5) * step, mid.expand_as(g)))
    return torch.cat(parts, -1)


def _exact_rows(cache, table, L):
    """Keys and values of one sequence of L tokens, 64 bits [L, Hkv, 128], by the channel's place in the block."""
    t = torch.arange(L, device=device)[:, None]
    c = torch.arange(D, device=device)[None]
    blocks = cache[table[:(L + PAGE - 1) // PAGE].long()]           # [pages, Hkv, 2560]
    page, r = t // PAGE, t % PAGE
    k_at = r * 64 + (c // 8 % 4) * 16 + c // 32 * 4 + c % 8 // 2
    q = c % 32 // 4
    v_at = 1024 + q * 128 + r % 8 // 2 * 32 + ((r // 8) ^ (q % 2)) * 16 + r % 2 * 8 + c // 32 * 2 + c % 4 // 2
    g = c // GROUP
    out = []
    for at, s_at, z_at in ((k_at, 2048 + r * 8 + g * 2, 2176 + r * 8 + g * 2),
                           (v_at, 2304 + r * 8 + g * 2, 2432 + g * 32 + r * 2)):
        code = (blocks[page, :, at].int() >> (c % 2 * 4)[..., None]) & 15
        two = [(blocks[page, :, p].int() | (blocks[page, :, p + 1].int() << 8)) for p in (s_at, z_at)]
        step, mid = ((w << 16).view(torch.float32).double() for w in two)
        out.append((mid + step * (code.double() - 7.5)).transpose(1, 2))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hq, Hkv = s["op"], s["B"], s["Hq"], s["Hkv"]
    if op in ("norm_rope", "append", "append_q4"):
        freq, axis = _inv_freq(case["R"], case.get("axes", 1))
    if op == "norm_rope":
        pos = s["pos"][:, :, None] if case["bhsd"] else s["pos"][..., None]
        return [_exact_head(s[n], s[n + "w"], pos, freq, axis, case["inter"]) for n in "qk"]
    new, lens = _lengths(case)
    begin = [0]
    for n in new:
        begin.append(begin[-1] + n)
    if op in ("append", "append_q4"):
        pos = torch.cat([torch.arange(k - n, k, device=device) for n, k in zip(new, lens)])[None, :, None]
        q, k = (_exact_head(s[n], s[n + "w"], pos, freq, axis, case["inter"]) for n in "qk")
        if op == "append":
            kp, vp = s["k_pages"].double(), s["v_pages"].double()
            for b in range(B):
                p = torch.arange(lens[b] - new[b], lens[b], device=device)
                page = s["table"][b].long()[p // PAGE]
                kp[page, p % PAGE] = k[begin[b]:begin[b + 1]]
                vp[page, p % PAGE] = s["v"][begin[b]:begin[b + 1]].double()
            return [q, kp, vp]
        keys, values = [], []
        for b in range(B):
            old = lens[b] - new[b]
            ck, cv = _exact_rows(s["cache"], s["table"][b], lens[b])
            keys += [ck[:old], _exact_held(k[begin[b]:begin[b + 1]].to(torch.bfloat16))]
            values += [cv[:old], _exact_held(s["v"][begin[b]:begin[b + 1]])]
        return [q, torch.cat(keys), torch.cat(values)]
    outs, lses = [], []
    for b in range(B):
        L, n = lens[b], new[b]
        q = s["q"][begin[b]:begin[b + 1]].double()                   # [n, Hq, 128]
        if L == 0:
            outs.append(torch.zeros_like(q))
            lses.append(torch.full((n, Hq), -math.inf, dtype=torch.float64, device=device))
            continue
        k, v = _exact_rows(s["cache"], s["table"][b], L)
        if op == "prefill_q4":
            k, v = (x.float().to(torch.bfloat16).double() for x in (k, v))
        o, l = torch.empty_like(q), torch.empty(n, Hq, dtype=torch.float64, device=device)
        hidden = None
        if op == "prefill_q4" and s["causal"]:
            hidden = torch.arange(L, device=device)[None] > torch.arange(L - n, L, device=device)[:, None]
        for h in range(Hq):
            x = q[:, h] @ k[:, h * Hkv // Hq].T / math.sqrt(D)
            if hidden is not None:
                x[hidden] = -math.inf
            l[:, h] = torch.logsumexp(x, -1)
            o[:, h] = torch.softmax(x, -1) @ v[:, h * Hkv // Hq]
        outs.append(o)
        lses.append(l)
    out, lse = torch.cat(outs), torch.cat(lses)
    return [out, lse if op == "decode_q4" else lse.T.contiguous()]
