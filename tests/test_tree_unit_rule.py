"""The rule by which fp_tree_attn keeps its 16-bit weights in range, modelled in numpy and checked against exact
softmax on adversarial rows.

A row's weights w = 2^(s - m) v (s scores in log2 units, v V's scales) are held in 16 bits, in a unit 2^m of the row's
own; its sum of 2^(s - m) in fp32.  Tiles of 128 tokens are taken in chunks of 32.  Where the largest score of
a chunk with the largest of its scales, or with 2^-kFar, passes 2^(kLift + kSlack), the products are looked at, and the unit
moves if the row's own largest passes: to where that is at most 2^kLift.  What the tile has in 16 bits
already is rescaled in fp32 and rounded again.  Parts of a row are added up relative to the power of two below their sums.

Tolerance, as in test_tree_numerics.py: 2^-11 (bf16 2^-8) of each weight, and for fp16 2^-26 of the row's
largest for each visible token; fp32 sums of 1024 terms, 2^-23 each.
"""
import os
import re

import numpy as np
import pytest
import torch

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_block_sparse_last_b200", "csrc",
                   "tree_kernels.cuh")
F = np.float32
CHUNK, TILE = 32, 128


def constants():
    """(kLift, kSlack) of bf16 and fp16, and kFar, as the kernels have them."""
    text = open(SRC).read()
    pair = {k: [float(x) for x in re.search(rf"{k} = KIND == kKvBf16 \? (-?[\d.]+)f : (-?[\d.]+)f;", text).groups()]
            for k in ("kLift", "kSlack")}
    far = float(re.search(r"kFar = ([\d.]+)f;", text).group(1))
    return {"bf16": (pair["kLift"][0], pair["kSlack"][0]), "f16": (pair["kLift"][1], pair["kSlack"][1])}, far


RANGE, FAR = constants()


def rounded(x, kind):
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=F))
    return t.to(torch.bfloat16 if kind == "bf16" else torch.float16).float().numpy()


def pow2(d):
    return F(0) if d < -126 else np.exp2(F(d))


def ex2(x):
    with np.errstate(over="ignore"):
        y = np.exp2(x.astype(F))
    return np.where(y < 2.0 ** -126, F(0), y)


def top_of(m, l):
    return -np.inf if l == 0 else m + np.floor(np.log2(np.float64(l)))


def part(s, v, code, kind, mistake=None):
    """One processor's tokens: (unit, sum, O, largest weight held)."""
    lift, slack = RANGE[kind]
    m, l, o, held = -np.inf, F(0), np.zeros(code.shape[1], F), 0.0
    biggest = -np.inf
    for t0 in range(0, len(s), TILE):
        alpha, acc, done = F(1), F(0), []
        for c0 in range(t0, min(t0 + TILE, len(s)), CHUNK):
            x, y = s[c0:c0 + CHUNK].astype(F), v[c0:c0 + CHUNK].astype(F)
            with np.errstate(divide="ignore"):
                lv = np.log2(y)
            top, key = x.max(), (x + lv).max()
            if mistake == "largest scale":      # what is hidden or has no weight counts too
                biggest = max(biggest, lv.max())
                key = top + biggest
            if top + max(lv.max(), -FAR) - (lift + slack) > m:
                to = np.ceil(max(key, top - FAR)) - lift
                if to > m + slack:
                    by = pow2(m - to)
                    if mistake == "factor in fp16":
                        done = [rounded(p * rounded(by, kind), kind) for p in done]
                    else:
                        done = [rounded(p * by, kind) for p in done]
                    alpha, acc, m = alpha * by, acc * by, to
            p = ex2(x - F(0 if m == -np.inf else m))
            acc = F(acc + p.sum(dtype=F))
            w = rounded(np.where(x == -np.inf, F(0), p * y), kind)
            held = max(held, float(w.max()))
            done.append(w)
        l = F(l * alpha + acc)
        w = np.concatenate(done)
        o = (o * alpha + (w[:, None] * code[t0:t0 + len(w)]).sum(0, dtype=F)).astype(F)
    return m, l, o, held


def model(s, v, code, kind, cuts=(), mistake=None):
    parts = [part(s[a:b], v[a:b], code[a:b], kind, mistake) for a, b in zip((0, *cuts), (*cuts, len(s)))]
    M = max(top_of(m, l) for m, l, _, _ in parts)
    L = F(sum(l * pow2(m - M) for m, l, _, _ in parts))
    O = sum(o * pow2(m - M) for m, _, o, _ in parts)
    return O / L, M + np.log2(L), max(h for *_, h in parts)


def exact(s, v, code, kind):
    """(result, bound, log2 of the sum)."""
    seen = np.isfinite(s)
    e = np.where(seen, np.exp2(s.astype(np.float64) - s[seen].max()), 0.0)
    P = e / e.sum()
    w = P * v.astype(np.float64)
    up = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    # scores are near 2^7 at most: 2^-17 in the exponent's argument
    bound = (up + 2.0 ** -16 + len(s) * 2.0 ** -23) * (w @ np.abs(code))
    if kind == "f16":
        bound = bound + 2.0 ** -26 * seen.sum() * w.max() * np.abs(code).max()
    return w @ code, bound, s[seen].max() + np.log2(e.sum())


def rows():
    """name: (scores, V's scales); -inf scores are hidden tokens."""
    r = np.random.default_rng(3)
    L = 1024
    base = 3 * r.standard_normal(L)
    i = np.arange(L)
    one = np.ones(L)
    plateau = np.where(i % 128 < 32, 0.0, np.where(i % 128 < 96, 13.875, 0.0))
    low = np.where(plateau > 0, 10.875, 0.0)    # where it does not move a unit that was set at 0
    return {
        "normal": (base, np.exp2(r.uniform(-1, 1, L))),
        "rising": (base + np.linspace(0, 120, L), one),
        "falling": (base + np.linspace(120, 0, L), one),
        "plateau, jump 24": (np.where(i % 128 == 100, 24.25, plateau), np.where(plateau > 0, 1.0, 0.0)),
        "plateau, jump 26": (np.where(i % 128 == 100, 26.0, plateau), np.where(plateau > 0, 1.0, 0.0)),
        "plateau, jump 38": (np.where(i % 128 == 100, 38.0, plateau), np.where(plateau > 0, 1.0, 0.0)),
        "low plateau, jump 24": (np.where(i < 128, np.where(i == 100, 24.25, low), -60.0), one),
        "low plateau, jump 30": (np.where(i < 128, np.where(i == 100, 30.0, low), -60.0), one),
        "hidden 2^22": (np.where(i % 50 == 7, -np.inf, base), np.where(i % 50 == 7, 2.0 ** 22, 1.0)),
        "hidden 2^100": (np.where(i % 50 == 7, -np.inf, base), np.where(i % 50 == 7, 2.0 ** 100, 1.0)),
        "weightless 2^30": (np.where(i % 9 == 4, -100.0, base), np.where(i % 9 == 4, 2.0 ** 30, 1.0)),
        "sinks without values": (np.where(i % 8 == 0, 21.3, base / 3), np.where(i % 8 == 0, 0.0, 1.0)),
        "no values": (base, 0 * one),
        "values of 2^-100, then 1": (base, np.where(i < 512, 2.0 ** -100, 1.0)),
        "values of 1, then 2^-100": (base, np.where(i < 512, 1.0, 2.0 ** -100)),
        "values of 2^100, then 2^-20": (base, np.where(i < 512, 2.0 ** 100, 2.0 ** -20)),
        "one visible": (np.where(i == 777, 3.0, -np.inf), one),
        "first tile hidden": (np.where(i < 200, -np.inf, base), one),
        "flat": (0 * one, one),
    }


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("cuts", [(), (512,), (128, 384, 640)])
@pytest.mark.parametrize("name", list(rows()))
def test_rule_against_exact_softmax(kind, cuts, name):
    s, v = rows()[name]
    if kind == "bf16":                       # no scales there
        v = np.ones(len(s))
    code = np.random.default_rng(4).integers(-127, 128, (len(s), 8)).astype(F)
    got, lse, held = model(s.astype(F), v.astype(F), code, kind, cuts)
    want, bound, top = exact(s.astype(F), v.astype(F), code, kind)
    assert np.isfinite(got).all()
    lift, slack = RANGE[kind]
    assert held <= 2.0 ** (lift + slack) * (1 + 2.0 ** -7)      # rounded to the type
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / np.maximum(bound, 1e-300))
    assert abs(lse - top) <= 2.0 ** -13


@pytest.mark.parametrize("mistake,name", [("factor in fp16", "low plateau, jump 24"), ("largest scale", "hidden 2^22"),
                                          ("largest scale", "weightless 2^30")])
def test_a_planted_mistake_fails(mistake, name):
    s, v = rows()[name]
    code = np.random.default_rng(4).integers(0, 128, (len(s), 8)).astype(F)
    got, _, _ = model(s.astype(F), v.astype(F), code, "f16", (), mistake)
    want, bound, _ = exact(s.astype(F), v.astype(F), code, "f16")
    assert not (np.abs(got - want) <= bound).all()


def test_a_hidden_token_changes_nothing_bit_for_bit():
    s, _ = rows()["hidden 2^22"]
    code = np.random.default_rng(4).integers(-127, 128, (len(s), 8)).astype(F)
    res = [model(s.astype(F), np.where(np.isfinite(s), 1.0, big).astype(F), code, "f16") for big in (1.0, 2.0 ** 22, 2.0 ** 110)]
    for r in res[1:]:
        assert np.array_equal(r[0], res[0][0]) and r[1] == res[0][1]
