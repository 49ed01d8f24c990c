"""Few rows on an 8-bit cache whose values span the whole range of their powers of two,
2^-60 to 2^119, against 64 bits: the sum of weights keeps what the values' weights keep.

Bound of each value, fixed before the first run, with A = sum_j p_j |v_j|:
* y's one rounding to bf16: 2^-8 |y|;
* weights rounded to fp16: 2^-11 A; those below fp16's normal range, by half of 2^-24 each where
  the largest p_j 2^e_j stands at 2^14 or above: 2^-39 of it, times a code of at most 448, for each key;
* scores, exponents and logarithms: a sum of at most 128 fp32 products (scale sum |q k| below 128), exponents'
  arguments and logarithms below 2^8, each off by 2^-24 of that and 2^-22 by the approximations: 2^-10 A in all allowed.
The 2-norm: y's rounding is 2^-8 / sqrt(3) of it at most, the weights' 2^-11 / sqrt(3): 2.3e-3 in squares.
"""
from __future__ import annotations

import math

import pytest
import torch

from test_gpu_attention import BF16, CASES, F64, Batch, quant_exp

pytestmark = pytest.mark.gpu

# requests, keys of each: whole heads, a few parts of a head, many
SHAPES = {"whole": (200, 100), "few parts": (1, 150), "more parts": (1, 500), "many parts": (1, 60_000)}


def check(b, q, y, exps, scale, rows=None):
    ref, mag = b.reference(q, scale)
    g = b.Hq // b.Hk
    tail = torch.zeros(b.cap, b.Hq, 1, dtype=F64, device="cuda")
    for r, (n, c, row) in enumerate(zip(b.lengths, b.context, b.cu)):
        if n:
            s = torch.einsum("mhgd,hkd->mhgk", q[row: row + n].to(F64).view(n, b.Hk, g, b.D), b.k[r]) * scale
            s.masked_fill_(torch.arange(n + c, device="cuda") > c + torch.arange(n, device="cuda")[:, None, None, None], -math.inf)
            most = (torch.log_softmax(s, -1) / math.log(2) + exps[r].to(F64)[None, :, None]).amax(-1)
            tail[row: row + n, :, 0] = (torch.exp2(most - 39) * 448 * (n + c)).view(n, b.Hq)
    rows = slice(0, b.cu[-1]) if rows is None else rows
    y, ref, mag, tail = (t[rows] for t in (y.to(F64), ref, mag, tail))
    assert bool(torch.isfinite(y).all())
    over = ((y - ref).abs() - (2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -10) * mag + tail)) / mag.clamp_min(1e-300)
    assert float(over.max()) <= 0, f"{float(over.max()):.3e} of A past the bound"
    assert b.cache.status() == 0
    return float((y - ref).norm() / ref.norm())


def batch(shape, n, Hq, Hk, D):
    R, keys = SHAPES[shape]
    return Batch([n] * R, [keys - n] * R, Hq, Hk, D, "e4m3", 64)


def fill(b, scores, values):
    """Puts keys whose scores are the given ones (in log2 units, exact in 8 bits; a list of [keys]) and the values, a
    list of [Hk, keys, D]; returns the queries, the values' exponents and the scale."""
    exps = []
    for r, (s, v) in enumerate(zip(scores, values)):
        b.k[r] = b.put(r, "k", s[None, :, None].expand(b.Hk, -1, b.D))
        b.v[r] = b.put(r, "v", v)
        exps.append(quant_exp(v.to(BF16).float()))
    return torch.ones(b.cap, b.Hq, b.D, dtype=BF16, device="cuda"), exps, math.log(2) / b.D


FORMS = [(1, 8, 1, 128), (3, 20, 2, 64)]  # rows, heads, key heads, channels: 16 rows of a group, and 32


@pytest.mark.parametrize("n,Hq,Hk,D", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("top", [0, 104, 119])
@pytest.mark.parametrize("below", [8, 16])
def test_light_keys_beside_a_heavy_one(n, Hq, Hk, D, shape, top, below):
    """All values at 2^top; one key's weight is 2^below times each other's.  The heavy one's values are 1/8 of the
    others', so that a sum that loses the others' weights is seen."""
    b = batch(shape, n, Hq, Hk, D)
    keys = b.lengths[0] + b.context[0]
    scores, values = [], []
    for r in range(len(b.lengths)):
        s = torch.zeros(keys, device="cuda")
        s[(7 * r) % (keys - n)] = below
        v = (0.5 + torch.rand(Hk, keys, D, generator=b.g, device="cuda") / 4) * 2.0 ** (top + 8)
        v[:, (7 * r) % (keys - n)] /= 8
        v[:, :, 0] = 1.75 * 2.0 ** (top + 8)  # the exponent is top throughout
        scores.append(s), values.append(v)
    q, exps, scale = fill(b, scores, values)
    assert all(bool((e == top).all()) for e in exps)
    check(b, q, b.attend(q, scale=scale), exps, scale)


@pytest.mark.parametrize("n,Hq,Hk,D", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("top", [30, 119])
@pytest.mark.parametrize("order", ["first half", "every other", "all but one"])
def test_zero_values_beside_large_ones(n, Hq, Hk, D, shape, top, order):
    """Heads of zero have the power 2^-60; their weights count in the sum all the same."""
    b = batch(shape, n, Hq, Hk, D)
    keys = b.lengths[0] + b.context[0]
    j = torch.arange(keys, device="cuda")
    zero = {"first half": j < keys // 2, "every other": j % 2 == 0, "all but one": j != 40}[order]
    scores, values = [], []
    for _ in b.lengths:
        v = torch.randn(Hk, keys, D, generator=b.g, device="cuda").clamp(-3, 3) * 2.0 ** (top + 6)
        v[:, zero] = 0
        scores.append(torch.zeros(keys, device="cuda")), values.append(v)
    q, exps, scale = fill(b, scores, values)
    check(b, q, b.attend(q, scale=scale), exps, scale)


@pytest.mark.parametrize("n,Hq,Hk,D", FORMS + [(4, 8, 1, 128), (1, 6, 2, 64)])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("order", [1, -1])
def test_scores_that_fall_as_values_rise(n, Hq, Hk, D, shape, order):
    """Score and exponent change by 16 in opposite directions along the keys, so that all contribute alike to y
    while the weights go from 1 to 2^-112."""
    b = batch(shape, n, Hq, Hk, D)
    keys = b.lengths[0] + b.context[0]
    step = torch.arange(keys, device="cuda") * 8 // keys  # 0 .. 7
    step = step if order == 1 else step.flip(0)
    scores, values = [], []
    for _ in b.lengths:
        v = torch.randn(Hk, keys, D, generator=b.g, device="cuda").clamp(-3, 3) * torch.exp2(16.0 * step - 10)[None, :, None]
        scores.append(-16.0 * step.float()), values.append(v)
    q, exps, scale = fill(b, scores, values)
    check(b, q, b.attend(q, scale=scale), exps, scale)


@pytest.mark.parametrize("n,Hq,Hk,D", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_of_minus_infinity(n, Hq, Hk, D, shape):
    """The first 64 keys, a warp's or a part's all, weigh nothing; the others weigh alike."""
    b = batch(shape, n, Hq, Hk, D)
    keys = b.lengths[0] + b.context[0]
    exps = []
    for r in range(len(b.lengths)):
        k = torch.zeros(Hk, keys, D, device="cuda")
        k[:, :64] = -3e38
        v = torch.randn(Hk, keys, D, generator=b.g, device="cuda")
        b.k[r], b.v[r] = b.put(r, "k", k), b.put(r, "v", v)
        exps.append(quant_exp(v.to(BF16).float()))
    q = torch.full((b.cap, Hq, D), 3e38, dtype=BF16, device="cuda")
    check(b, q, b.attend(q, scale=0.1), exps, 0.1)


@pytest.mark.parametrize("name", [n for n, c in CASES.items() if max(c[0]) * (c[2] // c[3]) <= 32])
def test_weights_keep_fp16_s_bits(name):
    """The shapes of single tokens and drafts, whose weights are rounded to fp16 and not to bf16."""
    lengths, context, Hq, Hk, D, page = CASES[name]
    b = Batch(lengths, context, Hq, Hk, D, "e4m3", page, seed=len(name))
    q = b.randn(b.cap, Hq, D).to(BF16)
    exps = []
    for r in range(len(lengths)):  # the exponents of what the cache holds
        amax = b.v[r].abs().amax(-1)
        exps.append(torch.ceil(torch.log2((amax / 448).clamp_min(2.0 ** -60))))
    err = check(b, q, b.attend(q), exps, D ** -0.5)
    assert err <= 2.3e-3, err
