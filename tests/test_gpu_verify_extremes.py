"""Verification of rows whose largest logit, over the temperature, is far from 0: very low and very high temperatures, rows
that are masked with the type's lowest value, logits far from 0.  Compared with the walk in 64 bits, as in
test_gpu_verify_tree.py: what is relative to the largest logit does not hang on how large that is.

A case's decisions lie further apart than fp32's rounding moves them.  A probability is off by less than 2^-15 of itself: its
exponent, (x - m) / T of at most 126 powers of two, by 126 * 3 * 2^-24 (difference, factor, their product), so itself by ln 2
times that (2^-15.9), its exponential and the sum by 2^-21 more.  p - q and its sum add no more than their own roundings where p and q are not nearly equal, and
the siblings here are few.  near() looks each case's decisions over, on the CPU, for gaps of 2^-12 or less of the larger side."""
import math

import pytest
import torch

from test_gpu_verify_tree import check, make, want

pytestmark = pytest.mark.gpu

FP, BF = torch.float32, torch.bfloat16


def near(d):
    """Whether a decision u q(x) < p(x), or between the two best tokens of a race, is a close one on some sequence's way."""
    path, _, counts = want(d)
    V = d["logits"].shape[1]
    for b in range(len(d["cu"]) - 1):
        begin, n, temp = int(d["cu"][b]), int(d["cu"][b + 1] - d["cu"][b]), float(d["temperature"][b])
        if not temp > 0:
            continue
        for node in path[b, :int(counts[b])].tolist():
            rows = []
            for t in (d["logits"], d["draft"]):
                if t is None:
                    continue
                x = t[begin + node].double().nan_to_num(nan=-math.inf, neginf=-math.inf, posinf=torch.finfo(FP).max)
                w = torch.where(x > -math.inf, ((x - x.max()) / temp).exp() if temp < math.inf else torch.ones_like(x), 0.0)
                rows.append(w / w.sum())
            p, q = rows[0], rows[1] if len(rows) > 1 else None
            kept = None
            for i in range(node + 1, n):
                if int(d["parents"][begin + i]) != node:
                    continue
                x, u = int(d["tokens"][begin + i]), float(d["uniforms"][begin + i])
                left, right = u * (1.0 if q is None else float(q[x])), float(p[x])
                if 0 < max(left, right) and abs(left - right) <= 2.0 ** -12 * max(left, right):
                    return True
                if left < right:
                    kept = i
                    break
                rest = (p - q).clamp(min=0) if q is not None else torch.where(torch.arange(V) == x, 0.0, p)
                if 0 < float(rest.sum()) < 2.0 ** -8:
                    return True
                p = rest / rest.sum() if float(rest.sum()) > 0 else p
            if kept is None:
                best = (p / d["noise"][b].double()).sort(descending=True)[0]
                if len(best) > 1 and best[0] - best[1] <= 2.0 ** -12 * best[0]:
                    return True
    return False


def run(d):
    assert not near(d)
    check(d)


@pytest.mark.parametrize("kind,dtype", [("top", BF), ("draft", BF), ("draft", FP)])
@pytest.mark.parametrize("temp", [1e-4, 1e-6, 1e-7, 1e-8, 1e-9, 1e-12, 1e-30, 1e-38, 1e9, 1e38, math.inf])
@pytest.mark.parametrize("sharp", [1.0, 30.0])
def test_temperatures(kind, dtype, temp, sharp):
    if dtype is BF and kind == "draft" and temp < 1:
        sharp *= 0.5      # (another set of trees)
    d = make(700 + int(sharp), [9, 1, 14], 333, kind, dtype, temps=[temp], sharp=sharp)
    run(d)


@pytest.mark.parametrize("kind,dtype", [("top", BF), ("draft", BF), ("top", FP), ("draft", FP)])
@pytest.mark.parametrize("temp", [0.01, 1.0, 5.0, 1e38, math.inf])
def test_rows_masked_with_the_lowest_value(kind, dtype, temp):
    """Some rows all of the type's lowest value (every token alike), others with a few tokens left."""
    d = make(720, [6, 4, 11, 3], 257, kind, dtype, temps=[temp], sharp=2.0)
    gen = torch.Generator().manual_seed(1)
    for name in ("logits", "draft"):
        if d[name] is None:
            continue
        low = torch.finfo(dtype).min
        d[name][torch.rand(d[name].shape, generator=gen) < 0.5] = low
        d[name][[0, 6, 12, 21]] = low
    run(d)


@pytest.mark.parametrize("kind", ["top", "draft"])
@pytest.mark.parametrize("temp", [1.0, 1e30, math.inf])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_infinities_and_the_lowest_value_together(kind, temp, dtype):
    d = make(730, [7, 5, 12], 129, kind, dtype, temps=[temp], sharp=2.0)
    gen = torch.Generator().manual_seed(2)
    for name in ("logits", "draft"):
        if d[name] is None:
            continue
        low = torch.finfo(dtype).min
        for value in (low, -math.inf, math.inf, math.nan):
            d[name][torch.rand(d[name].shape, generator=gen) < 0.1] = value
    run(d)


@pytest.mark.parametrize("kind", ["top", "draft"])
@pytest.mark.parametrize("offset", [1e3, 1e5, -1e5, 3e6, 6e6, -6e6, 5e7, -5e7, 1e9, -3e30])
def test_logits_far_from_zero(kind, offset):
    """fp32 rows that lie around any number, in steps of what is left of 32 bits there; drawn siblings are rejected."""
    d = make(740, [12, 9, 5], 200, kind, FP, tree="bush", temps=[1.0, 0.8], sharp=2.0)
    step = max(2.0 ** -10, abs(offset) * 2.0 ** -23)
    for name in ("logits", "draft"):
        if d[name] is not None:
            d[name] = ((d[name] / 0.5).round() * max(0.5, step) + offset).float()
    d["uniforms"][:] = 0.6 + d["uniforms"] * 0.4
    d["temperature"] *= max(1.0, step / 0.5)
    run(d)


@pytest.mark.parametrize("kind", ["top", "draft"])
def test_one_slice_far_below_another(kind):
    """Long rows, in several CTAs' slices, of which some hold only masked tokens and others the largest."""
    for seed, temp in ((750, 1.0), (761 if kind == "draft" else 751, 1e-7), (772 if kind == "draft" else 752, 100.0)):
        d = make(seed, [5, 7], 20011, kind, FP, temps=[temp], sharp=2.0, tree="bush" if seed == 750 else "tree")
        for name in ("logits", "draft"):
            if d[name] is not None:
                d[name][:, :9000] = torch.finfo(FP).min
                d[name][1::2, 9000:15000] -= 1e9
        run(d)
