"""Plain 64-bit references of the operators around the paged cache (CPU, torch):
norm and rotation, the 4-bit cache's quantisation and byte layout, and softmax
attention; with the error bounds that the tests hold the kernels to.

Bounds.  A rounding to bf16 is off by at most HALF = 2^-8 of the value.  The
fp32 work before it is bounded per element from the operands' magnitudes."""
import math

import torch

HALF = 2.0 ** -8
D, PAGE, GROUP, NG, BLOCK = 128, 16, 32, 4, 2560


def inv_freq(R, base=10000.0):
    return [base ** (-2.0 * i / R) for i in range(R // 2)]


def norm_rope(x, w, eps, pos, freq, axes, interleaved):
    """x [tokens, H, 128] bf16, pos int [n_axes, tokens] -> (double result, per-element magnitude of the terms)."""
    y = x.double()
    if w is not None:
        y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    out, mag = y.clone(), y.abs()
    n = len(freq)
    if n:
        f = torch.tensor(freq, dtype=torch.float64)
        a = torch.tensor(axes, dtype=torch.int64)
        t = (pos.double()[a].T * f)[:, None]                     # [tokens, 1, n]
        ia = torch.arange(n) * 2 if interleaved else torch.arange(n)
        ib = ia + 1 if interleaved else ia + n
        p, q = y[..., ia], y[..., ib]
        out[..., ia] = p * torch.cos(t) - q * torch.sin(t)
        out[..., ib] = p * torch.sin(t) + q * torch.cos(t)
        mag[..., ia] = mag[..., ib] = p.abs() + q.abs()
    return out, mag


def check_norm_rope(got, ref, what=""):
    """Final rounding: HALF of the value.  Before it, in fp32 (steps of 2^-24): the norm's 128-term sum (8 chained
    and 4 tree additions, halved by the root), root, division and two products: at most 12; the angle (the conversion
    to fp32, times pi, and sincospi's 2 steps): at most 5; products and sum: 3.  Together at most 20 <= 32 of the
    pair's |a| + |b|; a result may also lie in the subnormal range (2^-133 steps)."""
    out, mag = ref
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    err = (got - out).abs()
    bound = HALF * out.abs() + (1 + HALF) * 2.0 ** -19 * mag + 2.0 ** -133
    assert (err <= bound).all(), f"{what}: worst excess {(err - bound).max():.3g}, {(err > bound).sum()} elements"


# ---------------------------------------------------------------- the 4-bit cache

def quantise(x):
    """bf16 [..., 128] -> codes int64 [..., 128], scales and centers bf16 [..., 4] (each step in fp32)."""
    g = x.float().unflatten(-1, (NG, GROUP))
    finite = torch.isfinite(g).all(-1)
    hi, lo = g.max(-1).values, g.min(-1).values
    z = (hi * 0.5 + lo * 0.5).to(torch.bfloat16)
    s = (torch.maximum(hi - z.float(), z.float() - lo) * torch.tensor(2.0 / 15.0, dtype=torch.float32)).to(torch.bfloat16)
    sf = s.float()[..., None]
    n = torch.round((g - z.float()[..., None]) / sf + 7.5).clamp(0, 15)
    n = torch.where((sf > 0) & finite[..., None], n, torch.zeros_like(n))
    nan = torch.tensor(float("nan"), dtype=torch.bfloat16)
    return n.flatten(-2).long(), torch.where(finite, s, nan), torch.where(finite, z, nan)


def _places():
    """(K word, V half-word) byte offsets by [token][channel], and the four parameter offsets by [token][group]."""
    t = torch.arange(PAGE)[:, None]
    c = torch.arange(D)[None]
    w = c // 8
    k = 64 * t + 16 * (w % 4) + 4 * (w // 4) + c % 8 // 2
    g, r = c // 32, c % 32 // 4
    v = 1024 + 128 * r + 32 * (t % 8 // 2) + 16 * ((t // 8) ^ (r % 2)) + 8 * (t % 2) + 2 * g + c % 4 // 2
    q = torch.arange(NG)[None]
    return k, v, 2048 + 8 * t + 2 * q, 2176 + 8 * t + 2 * q, 2304 + 8 * t + 2 * q, 2432 + 32 * q + 2 * t


def _bits(t):
    return t.contiguous().view(torch.int16).long() & 0xffff


def write_tokens(cache, page, row, head, k, v):
    """Quantise k, v [n, 128] into the cache (CPU uint8) at (page, row, head) [n] each."""
    K, V, ks, kz, vs, vz = _places()
    for x, code_at, s_at, z_at in ((k, K, ks, kz), (v, V, vs, vz)):
        n, s, z = quantise(x)
        pair = (n[:, 0::2] | n[:, 1::2] << 4).to(torch.uint8)
        cache[page[:, None], head[:, None], code_at[row][:, 0::2]] = pair
        for val, at in ((s, s_at), (z, z_at)):
            b = _bits(val)
            cache[page[:, None], head[:, None], at[row]] = (b & 255).to(torch.uint8)
            cache[page[:, None], head[:, None], at[row] + 1] = (b >> 8).to(torch.uint8)


def pack_pools(k_pages, v_pages):
    """bf16 pools [P, 16, H, 128] -> cache uint8 [P, H, 2560]."""
    P, _, H, _ = k_pages.shape
    cache = torch.zeros(P, H, BLOCK, dtype=torch.uint8)
    page, row, head = (x.flatten() for x in torch.meshgrid(torch.arange(P), torch.arange(PAGE), torch.arange(H),
                                                           indexing="ij"))
    write_tokens(cache, page, row, head, k_pages.flatten(0, 2), v_pages.flatten(0, 2))
    return cache


def read_tokens(cache, pages, L):
    """One sequence's L tokens: for K and for V (codes double [L, H, 128], scales, centers double [L, H, 128])."""
    places = _places()
    t = torch.arange(L)
    blocks, row = cache[pages.long()[t // PAGE]], t % PAGE              # [L, H, 2560]
    H = cache.shape[1]
    out = []
    for code_at, s_at, z_at in ((places[0], places[2], places[3]), (places[1], places[4], places[5])):
        at = code_at[row][:, None].expand(L, H, D)
        n = (blocks.gather(2, at).int() >> (torch.arange(D) % 2 * 4)) & 15
        sz = []
        for p in (s_at, z_at):
            a = p[row][:, None].expand(L, H, NG)
            bits = blocks.gather(2, a).int() | blocks.gather(2, a + 1).int() << 8
            sz.append((bits << 16).view(torch.float32).double().repeat_interleave(GROUP, -1))
        out.append((n.double(), sz[0], sz[1]))
    return out


def values(parts):
    n, s, z = parts
    return z + s * (n - 7.5)


def values_bf16(parts):
    """As read back: the sum rounded to fp32 and then to bf16."""
    return values(parts).float().to(torch.bfloat16)


def attend(q, k, v, scale, hidden=None):
    """q [n, Hq, 128] double, k, v [L, Hkv, 128] double -> (out, lse [n, Hq], weights [Hq, n, L])."""
    G = q.shape[1] // k.shape[1]
    kk, vv = (x.repeat_interleave(G, 1) for x in (k, v))
    s = torch.einsum("nhd,lhd->hnl", q, kk) * scale
    if hidden is not None:
        s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:2], -math.inf, dtype=torch.float64)
    w = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("hnl,lhd->nhd", w, vv), lse.T, w


def reference_unit(scales):
    """2^(e + 3) for the largest e that a warp's first page pair with a scale can give as its usual exponent: the
    tokens' mean one, or the pair's largest where that is at most 3 more.  scales [L, 4] of one KV head."""
    top = scales.double().amax(-1)
    top = torch.cat([top, torch.zeros(-len(top) % (2 * PAGE))]).view(-1, 2 * PAGE)
    ex = torch.where(top > 0, torch.floor(torch.log2(top.clamp_min(2.0 ** -127))), torch.zeros_like(top))
    n = (top > 0).sum(-1)
    usual = torch.minimum(torch.where(top > 0, ex, ex - 1000).amax(-1), torch.floor(ex.sum(-1) / n.clamp_min(1)) + 3)
    return 2.0 ** (float(usual[n > 0].max()) + 3) if (n > 0).any() else 0.0


def check_decode_q4_mixed(got, lse, q, cache, table, lens, scale, what=""):
    """check_decode_q4 for values of very different scales.  The same terms, but a key's weight is off by its own
    score's error and the weighted mean of the others', and f16's last steps are counted in the units that the kernel
    promises: P is taken over a reference below the head's largest score so that a usual scale 2^e makes at least 2^5
    of the largest P, 8 bits less where larger scales follow (2^-25 of that is w_max 2^(e + 3) 2^-25), or, where a
    product P s lies 2^15 above, so that the largest is 2^5 or more."""
    got, lse = got.double().cpu(), lse.double().cpu()
    Hq, Hkv = q.shape[1], cache.shape[1]
    G = Hq // Hkv
    for b, L in enumerate(lens):
        qb = q[b:b + 1].double()
        kp, vp = read_tokens(cache, table[b], L)
        out, ref_lse, w = attend(qb, values(kp), values(vp), scale)
        terms = (32 * kp[1] + kp[2].abs()).repeat_interleave(G, 1)
        e = 16 * 2.0 ** -24 * scale * torch.einsum("nhd,lhd->hnl", qb.abs(), terms)              # [Hq, 1, L]
        ws = w * (e + (w * e).sum(-1, keepdim=True) + 2.0 ** -20)
        codes = (vp[1] * (vp[0] - 7.5)).abs().repeat_interleave(G, 1)
        centers = vp[2].abs().repeat_interleave(G, 1)
        s8 = vp[1].repeat_interleave(G, 1)
        mix = lambda a, t: torch.einsum("hnl,lhd->nhd", a, t)  # noqa: E731
        unit = torch.tensor([reference_unit(vp[1][:, h, ::GROUP]) for h in range(Hkv)]).repeat_interleave(G)
        largest = torch.einsum("hnl,lh->hnl", w, s8.amax(-1)).amax(-1)[:, 0]                     # [Hq]
        small = (L * 7.5 * 2.0 ** -25) * torch.maximum(unit * w.amax(-1)[:, 0], largest * 2.0 ** -5)
        bound = HALF * out.abs() + (1 + HALF) * (mix(w, codes) * 2.0 ** -11 + mix(ws, codes) + mix(w, centers) * HALF +
                                                 mix(ws, centers) + small[:, None] + 2.0 ** -17 * mix(w, s8)) + 2.0 ** -133
        err = (got[b] - out[0]).abs()
        assert torch.isfinite(got[b]).all() and (err <= bound[0]).all(), \
            f"{what}: sequence {b} (L={L}): worst ratio {(err / bound[0]).max():.3g}, {(err > bound[0]).sum()} elements"
        lerr = (lse[b] - ref_lse[0]).abs()
        assert (lerr <= e.amax(-1)[:, 0] + 2.0 ** -20 * (1 + ref_lse[0].abs())).all(), f"{what}: lse off by {lerr.max():.3g}"


def check_decode_q4(got, lse, q, cache, table, lens, scale, what=""):
    """attn_decode_paged_q4 against 64 bits.

    Key codes enter the products as they are (n <= 15), 7.5 is taken off after them; value codes enter as n - 7.5.
    Scores are fp32 sums of 128 products q s n and 7.5 q s: errors of a few steps (16 at most) of the terms' sum,
    e = 16 * 2^-24 * scale * sum |q| (32 s + |z|); a weight is then off by that share and by ex2's and the merge's few
    steps (2^-20 in all).  The centers meet probabilities in bf16: HALF of w |z|.  The codes meet probability times scale
    in f16: 2^-11 of w |s (n - 7.5)|, and for the smallest ones half of f16's last step, 2^-25, times |n - 7.5| <= 7.5,
    for each key, over the row sum, which is at least 1 / (the largest weight), in units of 1 or, where scales are far
    from it, of at most 2^-5 of the largest scale.  fp32 accumulation adds 16 * 2^-24 of 8 w s.  The output is rounded
    once.  lse moves by at most the largest score error and ln's 2^-20."""
    got, lse = got.double().cpu(), lse.double().cpu()
    Hq = q.shape[1]
    for b, L in enumerate(lens):
        qb = q[b:b + 1].double()
        if L == 0:
            assert (got[b] == 0).all() and torch.isneginf(lse[b]).all(), f"{what}: empty sequence {b}"
            continue
        kp, vp = read_tokens(cache, table[b], L)
        out, ref_lse, w = attend(qb, values(kp), values(vp), scale)
        G = Hq // cache.shape[1]
        terms = (32 * kp[1] + kp[2].abs()).repeat_interleave(G, 1)
        e = 16 * 2.0 ** -24 * scale * torch.einsum("nhd,lhd->hnl", qb.abs(), terms).amax(-1)     # [Hq, 1]
        share = 2 * e + 2.0 ** -20
        codes = (vp[1] * (vp[0] - 7.5)).abs().repeat_interleave(G, 1)
        centers = vp[2].abs().repeat_interleave(G, 1)
        wc, wz, ws = (torch.einsum("hnl,lhd->nhd", w, t) for t in (codes, centers, (8 * vp[1]).repeat_interleave(G, 1)))
        top = vp[1].max()
        unit = max(1.0 if 2.0 ** -10 <= top < 2.0 ** 7 else 0.0, float(top) * 2.0 ** -5)
        small = (L * 7.5 * 2.0 ** -25 * unit) * w.amax(-1)                                       # [Hq, 1]
        bound = HALF * out.abs() + (1 + HALF) * (wc * (2.0 ** -11 + share[:, 0, None]) + wz * (HALF + share[:, 0, None]) +
                                                 small + 2.0 ** -20 * ws) + 2.0 ** -133
        err = (got[b] - out[0]).abs()
        assert torch.isfinite(got[b]).all() and (err <= bound[0]).all(), \
            f"{what}: sequence {b} (L={L}): worst excess {(err - bound[0]).max():.3g}"
        lerr = (lse[b] - ref_lse[0]).abs()
        assert (lerr <= e[:, 0] + 2.0 ** -20 * (1 + ref_lse[0].abs())).all(), f"{what}: lse off by {lerr.max():.3g}"
