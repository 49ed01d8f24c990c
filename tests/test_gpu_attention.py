"""The paged cache and the attention over it on the GPU, against plain 64-bit
implementations.

Tolerances, fixed before the first run.  Each value's own bound, with
A = sum_j p_j |v_j| (p the softmax weights):
* y's one rounding to bf16: 2^-8 |y|;
* weights rounded to bf16: 2^-8 A (8-bit caches of few rows: to fp16, 2^-11 A);
* scores: a sum of at most 128 fp32 products, 2^-24 each of scale sum |q k| (below
  128 here), and the same again for the exponent's argument: 2^-24 (2^7 + 2^7) = 2^-16,
  times as many terms at worst but 2^-10 A in all allowed, for weights and their sum.
The 2-norm over all rows: values of random signs, so the two roundings (1.7e-3
each, the root of a third of 2^-8 squared, a quarter less on average) add in squares: 3e-3.
What is moved or quantised is compared for equality: codes are exact quotients by
powers of two, rounded once.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.attention import KVCache
from rs_decode_gb300.prefill import Ragged, qk_norm

pytestmark = pytest.mark.gpu

F64, BF16, I32, E4M3 = torch.float64, torch.bfloat16, torch.int32, torch.float8_e4m3fn


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=I32).cuda()


class Batch:
    """A planned batch, a cache with something in every page, and a page table."""

    def __init__(self, lengths, context, Hq, Hk, D, type="bf16", page=64, cap=None, seed=0, spare=3, garbage=True, extra_pages=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.lengths, self.context = g, list(lengths), list(context)
        self.Hq, self.Hk, self.D, self.type, self.page = Hq, Hk, D, type, page
        R = len(lengths)
        need = [(n + c + page - 1) // page for n, c in zip(lengths, context)]
        self.n_pages, self.max_pages = sum(need) + spare, max(1, max(need)) + extra_pages
        order = torch.randperm(self.n_pages, generator=g, device="cuda").to(I32)
        self.pages = torch.full((R, self.max_pages), -1, dtype=I32, device="cuda")
        at = 0
        for r, n in enumerate(need):
            self.pages[r, :n] = order[at: at + n]
            at += n
        self.cu = [0]
        for n in lengths:
            self.cu.append(self.cu[-1] + n)
        self.cap = cap or max(1, self.cu[-1])
        self.ragged = Ragged(R, self.cap)
        self.ragged.plan(i32(lengths), i32(context))
        self.cache = KVCache(Hq, Hk, D, self.n_pages, self.max_pages, page=page, type=type)
        # every request's keys and values, and garbage everywhere else
        self.k, self.v = [], []
        if garbage:
            for t in (self.cache.k, self.cache.v):
                t.view(torch.uint8).fill_(0xff)  # NaN in either type
            if type == "e4m3":
                self.cache.k_exp.fill_(255)
                self.cache.v_exp.fill_(255)
        for r in range(R):
            n = lengths[r] + context[r]
            size = torch.exp2(torch.randint(-2, 2, (2, Hk, 1, 1), generator=g, device="cuda").float())
            k, v = torch.randn(2, Hk, n, D, generator=g, device="cuda") * size
            self.k.append(self.put(r, "k", k))
            self.v.append(self.put(r, "v", v))
        self.max_len = max(1, max(lengths))

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def put(self, r, name, x):
        """x [Hk, n, D] as the cache's first n keys or values of request r; what is then there, in 64 bits."""
        arr, exp = getattr(self.cache, name), getattr(self.cache, name + "_exp")
        n = x.shape[1]
        if self.type == "e4m3":
            e = quant_exp(x.to(BF16).float())
            codes = torch.ldexp(x.to(BF16).float(), -e[..., None]).to(E4M3)
            kept = torch.ldexp(codes.to(F64), e[..., None])
        else:
            kept = x.to(BF16).to(F64)
        for j in range((n + self.page - 1) // self.page):
            a, b = j * self.page, min(n, (j + 1) * self.page)
            at = int(self.pages[r, j])
            if self.type == "e4m3":
                arr[at, :, : b - a] = codes[:, a:b].view(torch.uint8)
                exp[at, :, : b - a] = (e[:, a:b] + 127).to(torch.uint8)
            else:
                arr[at, :, : b - a] = x[:, a:b].to(BF16)
        return kept

    def attend(self, q, max_len=None, scale=None, stream=None, **kw):
        m = max_len or self.max_len
        plan = self.cache.plan(self.ragged, m, stream=stream)
        return self.cache.attend(self.ragged, q, self.pages, plan, max_len=m, scale=scale, stream=stream, **kw)

    def reference(self, q, scale=None, r=None):
        """y and the bound's A, in 64 bits, [rows, Hq, D]."""
        g, scale = self.Hq // self.Hk, scale if scale is not None else self.D ** -0.5
        y = torch.zeros(self.cap, self.Hq, self.D, dtype=F64, device="cuda")
        mag = torch.zeros_like(y)
        for r in range(len(self.lengths)) if r is None else [r]:
            n, c, row = self.lengths[r], self.context[r], self.cu[r]
            if not n:
                continue
            step = max(1, (1 << 25) // (self.Hq * (n + c)))
            for a in range(0, n, step):
                m = min(step, n - a)
                qq = q[row + a: row + a + m].to(F64).view(m, self.Hk, g, self.D)
                s = torch.einsum("mhgd,hkd->hgmk", qq, self.k[r]) * scale
                hidden = torch.arange(n + c, device="cuda")[None] > c + a + torch.arange(m, device="cuda")[:, None]
                p = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
                y[row + a: row + a + m] = torch.einsum("hgmk,hkd->mhgd", p, self.v[r]).reshape(m, self.Hq, self.D)
                mag[row + a: row + a + m] = torch.einsum("hgmk,hkd->mhgd", p, self.v[r].abs()).reshape(m, self.Hq, self.D)
        return y, mag

    def check(self, q, y, scale=None, rows=None):
        ref, mag = self.reference(q, scale)
        rows = slice(0, self.cu[-1]) if rows is None else rows
        y, ref, mag = y[rows].to(F64), ref[rows], mag[rows]
        over = (y - ref).abs() - (2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag)
        assert not torch.isnan(y).any()
        assert float(over.max()) <= 0, f"{float(over.max()):.3e} past the bound at {np.unravel_index(int(over.argmax()), over.shape)}"
        err = float((y - ref).norm() / ref.norm())
        assert err <= 3e-3, err
        assert self.cache.status() == 0


def quant_exp(x):
    a = x.abs().amax(-1).double()
    e = torch.ceil(torch.log2(a / 448)).nan_to_num(neginf=-60.0)
    # the least power of two, whatever the logarithm's rounding
    e = torch.where(a <= 448 * torch.exp2(e - 1), e - 1, torch.where(a > 448 * torch.exp2(e), e + 1, e))
    return e.clamp_min(-60).to(I32)


# ----------------------------------------------------------------------------- the cache
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hk,D,page", [(1, 64, 16), (3, 128, 32), (4, 128, 64), (8, 64, 256), (5, 128, 128)])
def test_write_then_read(type, Hk, D, page):
    b = Batch([1, 0, 70, 17, 1], [0, 9, 33, 255, 64], 2 * Hk, Hk, D, type, page, cap=97)
    g = b.g
    fused = torch.randn(97, 3 * Hk * D + 8, generator=g, device="cuda", dtype=BF16)  # one projection's rows
    k, v = fused[:, 8: 8 + Hk * D].unflatten(1, (Hk, D)), fused[:, 8 + 2 * Hk * D:].unflatten(1, (Hk, D))
    before = [t.clone() for t in (b.cache.k, b.cache.v)]
    b.cache.write(b.ragged, k, v, b.pages)
    out = tuple(torch.full((97, Hk, D), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    b.cache.read(b.ragged, b.pages, out=out)
    T = b.cu[-1]
    touched = torch.zeros(b.n_pages, page, dtype=torch.bool, device="cuda")
    for r, (n, c) in enumerate(zip(b.lengths, b.context)):
        for t in range(c, c + n):
            touched[b.pages[r, t // page].long(), t % page] = True
    for x, got, arr, old in ((k, out[0], b.cache.k, before[0]), (v, out[1], b.cache.v, before[1])):
        if type == "e4m3":
            e = quant_exp(x.float())
            want = torch.ldexp(torch.ldexp(x.float(), -e[..., None]).to(E4M3).float(), e[..., None]).to(BF16)
        else:
            want = x
        assert torch.equal(got[:T], want[:T])
        assert torch.equal(got[T:], torch.full_like(got[T:], 7.0))  # past the batch
        same = (arr.view(torch.uint8) == old.view(torch.uint8)).all(-1).transpose(1, 2)  # [page, slot, head]
        assert bool(same[~touched].all())
    assert b.cache.status() == 0


def test_eight_bit_edges():
    """Zeros, the ends of the range, exact powers, heads that are not finite."""
    D = 64
    rows = torch.zeros(12, 1, D, dtype=BF16, device="cuda")
    top = torch.finfo(BF16).max
    rows[1, 0, 3] = 448.0
    rows[2, 0, 3] = 450.0
    rows[3, 0, :2] = torch.tensor([top, -top / 4])
    rows[4, 0, :2] = torch.tensor([1e-30, -1e-38])
    rows[5, 0, 0], rows[5, 0, 1] = math.inf, 1.0
    rows[6, 0, 0], rows[6, 0, 1] = math.nan, 1.0
    rows[7, 0] = torch.linspace(-448, 448, D)
    rows[8, 0, 0] = 2.0 ** -60 * 448
    rows[9, 0, 0] = 2.0 ** -61 * 448
    rows[10, 0, :2] = torch.tensor([-0.0, 2.0 ** -133])
    rows[11, 0] = 2.0 ** 100
    b = Batch([12], [0], 1, 1, D, "e4m3", 16)
    b.cache.write(b.ragged, rows, rows, b.pages)
    k, v = b.cache.read(b.ragged, b.pages)
    exp = b.cache.k_exp[b.pages[0, 0].long(), 0, :12].tolist()
    assert exp == [67, 127, 128, 246, 67, 255, 255, 127, 67, 67, 67, 127 + 92]
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    want = rows.clone()
    for r in range(12):
        if r in (5, 6):
            want[r] = math.nan
        elif exp[r] == 246:  # the largest value is past the codes' range by a little
            want[r, 0, 0] = 448 * 2.0 ** 119
            want[r, 0, 1] = -(112 * 2.0 ** 119 if top / 4 > 112 * 2.0 ** 119 else top / 4)
        else:
            e = exp[r] - 127
            want[r] = torch.ldexp(torch.ldexp(rows[r].float(), torch.tensor(-e, device="cuda")).to(E4M3).float(), torch.tensor(e, device="cuda")).to(BF16)
    keep = [r for r in range(12) if r != 3]
    torch.testing.assert_close(k[keep], want[keep], rtol=0, atol=0, equal_nan=True)
    assert float(k[3, 0, 0]) == 448 * 2.0 ** 119 and abs(float(k[3, 0, 1]) / (-top / 4) - 1) <= 2.0 ** -4
    assert b.cache.status() == 0


def test_pages_that_do_not_exist():
    b = Batch([40, 30, 20], [0, 10, 0], 4, 2, 64, page=16)
    k = b.randn(90, 2, 64).to(BF16)
    b.pages[1, 1] = b.n_pages
    b.pages[2, 0] = -1
    b.cache.write(b.ragged, k, k, b.pages)
    assert b.cache.status() == rb.DEV_SLOT
    out = tuple(torch.full((90, 2, 64), 3.0, dtype=BF16, device="cuda") for _ in range(2))
    b.cache.read(b.ragged, b.pages, out=out)
    assert b.cache.status() == rb.DEV_SLOT
    lost = [*range(46, 62), *range(70, 86)]
    kept = [r for r in range(90) if r not in lost]
    assert torch.equal(out[0][kept], k[kept])
    assert bool((out[0][lost] == 3.0).all())
    # positions past the table's row
    short = KVCache(4, 2, 64, b.n_pages, 1, page=16)
    short.write(b.ragged, k, k, b.pages[:, :1].contiguous())
    assert short.status() & rb.DEV_LENGTH


# ----------------------------------------------------------------------------- the shares
def shares(b, max_len):
    """The plan as plain lists: requests of either form, and where the shares begin."""
    raw = b.cache.plan(b.ragged, max_len).cpu().numpy()
    head = raw[:64].view(np.int32)
    n_short, n_long, short_rows, ctas, R = head[0], head[1], head[2], head[3], len(b.lengths)
    at = 64
    lists = raw[at: at + 32 * R].view(np.int32).reshape(2, R, 4)
    at += 32 * R
    starts = raw[at: at + 32 * (ctas + 1)].view(np.int32).reshape(2, ctas + 1, 4)
    return lists[0][:n_short], lists[1][:n_long], short_rows, starts[0], starts[1]


@pytest.mark.parametrize("lengths,context,Hq,Hk", [
    ([1] * 300, list(range(0, 3000, 10)), 8, 2),
    ([1, 500, 0, 3, 77, 2, 1, 1300], [5, 0, 9, 1000, 4097, 63, 64, 127], 32, 4),
    ([9], [100_000], 6, 2), ([1], [200_000], 16, 1), ([4000, 33], [0, 10], 3, 1), ([257] * 40, [0] * 40, 10, 2),
    ([1], [0], 1, 1), ([2000], [77], 4, 4), ([5] * 1500, [3] * 1500, 160, 4)])
def test_shares_cover_the_work_once(lengths, context, Hq, Hk):
    b = Batch.__new__(Batch)
    R, g = len(lengths), Hq // Hk
    b.lengths = lengths
    b.ragged = Ragged(R, sum(lengths))
    b.ragged.plan(i32(lengths), i32(context))
    b.cache = KVCache(Hq, Hk, 64, 10, 20_000, page=16)
    shorts, longs, short_rows, s_start, l_start = shares(b, max(lengths))
    assert b.cache.status() == 0
    cu = np.concatenate([[0], np.cumsum(lengths)])
    rows = [(r, int(cu[r]), lengths[r], context[r]) for r in range(R) if lengths[r]]
    assert [tuple(x) for x in shorts] == [x for x in rows if x[2] * g <= short_rows]
    assert [tuple(x) for x in longs] == [x for x in rows if x[2] * g > short_rows]
    tq = 2 * (128 // g)
    for starts, lst, items_of, parts_of in (
            (s_start, shorts, lambda n: 1, lambda n, c, i: (n + c + 63) // 64),
            (l_start, longs, lambda n: -(-n // tq), lambda n, c, i: (c + min(n, (i + 1) * tq) + 127) // 128)):
        if not len(lst):
            continue
        # the places of all parts, in order
        places, sizes = [], []
        for idx, (_, _, n, c) in enumerate(lst):
            for i in range(items_of(n)):
                for h in range(Hk):
                    places += [(idx, i, h, p) for p in range(parts_of(n, c, i))]
        index = {p: k for k, p in enumerate(places)}
        index[(len(lst), 0, 0, 0)] = len(places)
        at = [index[tuple(int(v) for v in s)] for s in starts]
        assert at[0] == 0 and at[-1] == len(places) and all(a <= c for a, c in zip(at, at[1:]))
        biggest = max(c - a for a, c in zip(at, at[1:]))
        assert biggest <= 2 * (len(places) + 4 * len(lst) * Hk * max(items_of(n) for _, _, n, _ in lst)) // 152 + 4


@pytest.mark.parametrize("lengths,context,Hq,Hk", [
    ([1], [0], 4, 4), ([1], [9000], 8, 2), ([1] * 7, [0, 5000, 3, 640, 64, 2000, 1], 32, 4), ([3000, 40, 1], [0, 700, 9], 6, 2),
    ([33] * 3, [20_000, 10, 4000], 16, 1), ([1] * 200, list(range(0, 2000, 10)), 16, 2)])
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_cut_heads_are_listed_once(lengths, context, Hq, Hk, type):
    b = Batch.__new__(Batch)
    R, g = len(lengths), Hq // Hk
    b.lengths = lengths
    b.ragged = Ragged(R, sum(lengths))
    b.ragged.plan(i32(lengths), i32(context))
    b.cache = KVCache(Hq, Hk, 64, 10, 20_000, page=16, type=type)
    shorts, longs, _, s_start, l_start = shares(b, max(lengths))
    raw = b.cache.plan(b.ragged, max(lengths)).cpu().numpy()
    ctas = len(s_start) - 1
    at = 64 + 32 * R + 32 * (ctas + 1)
    joins = raw[at: at + 32 * ctas].view(np.int32).reshape(2, ctas, 4)
    tq = 2 * (128 // g)
    for starts, lst, got, is_long in ((s_start, shorts, joins[0], False), (l_start, longs, joins[1], True)):
        heads = {}  # of each head that a share begins within: the shares that do
        for c in range(ctas):
            idx, item, head, part = (int(x) for x in starts[c])
            if idx < len(lst) and part:
                heads.setdefault((idx, item, head), []).append(c)
        want = np.zeros((ctas, 4), np.int32)
        for (idx, item, head), cs in heads.items():
            assert cs == list(range(cs[0], cs[-1] + 1)) and len({int(starts[c][3]) for c in cs}) == len(cs)
            _, row, n, _ = (int(x) for x in lst[idx])
            want[cs[0]] = (1 + len(cs), head, row + item * tq, min(tq, n - item * tq) if is_long else n)
        assert np.array_equal(got[:, 0], want[:, 0])
        assert np.array_equal(got[got[:, 0] > 0], want[want[:, 0] > 0])


# ----------------------------------------------------------------------------- attention
CASES = {  # lengths, context, Hq, Hk, D, page
    "one token of one": ([1], [0], 1, 1, 64, 16),
    "first tokens": ([1, 1, 1], [0, 0, 0], 8, 2, 128, 64),
    "tokens": ([1, 1, 0, 1, 1, 1, 1], [0, 1, 9, 15, 63, 64, 1000], 32, 4, 128, 64),
    "tokens, small pages": ([1] * 5, [16, 500, 31, 77, 250], 8, 1, 64, 16),
    "tokens, one head each": ([1] * 6, [100, 2, 3000, 64, 127, 128], 4, 4, 128, 128),
    "tokens of 16 heads": ([1, 1, 1], [700, 33, 2], 16, 1, 128, 32),
    "tokens of 24 heads": ([1, 1, 1], [700, 33, 2], 48, 2, 64, 64),
    "tokens of 40 heads": ([1, 1, 1], [700, 33, 2], 40, 1, 128, 64),
    "tokens of 128 heads": ([1, 3], [200, 5], 128, 1, 64, 64),
    "one long": ([1], [20_000], 16, 2, 128, 256),
    "drafts": ([4, 4, 2, 1, 4], [0, 61, 300, 1000, 127], 32, 4, 128, 32),
    "drafts of 3 heads": ([5, 8, 3], [60, 7, 1200], 6, 2, 64, 64),
    "two drafts": ([2, 2], [500, 62], 40, 5, 128, 16),
    "a short prompt": ([50], [0], 8, 1, 128, 64),
    "edges": ([127, 128, 129, 1, 255, 16, 17], [0, 0, 0, 5, 1, 128, 111], 8, 2, 128, 64),
    "prompts, one head each": ([300, 128, 1, 129, 600], [0] * 5, 2, 2, 64, 128),
    "prompts of 3 heads": ([300, 84, 85, 43], [0, 10, 128, 1000], 6, 2, 128, 32),
    "prompts of 5 heads": ([70, 400], [3, 200], 10, 2, 64, 16),
    "prompts of 16 heads": ([100, 9], [0, 2000], 16, 1, 128, 64),
    "turns": ([1, 40, 200, 3, 90, 1, 2], [900, 1500, 64, 2000, 127, 4000, 129], 32, 4, 128, 64),
    "many small prompts": ([9, 10, 11, 12, 13, 14, 15, 16] * 8, [0, 100, 7, 64] * 16, 16, 2, 64, 64),
    "a long turn": ([33], [9000], 8, 2, 128, 256),
    "a prompt": ([3000], [0], 4, 2, 128, 64),
}


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", CASES)
def test_attend(name, type):
    lengths, context, Hq, Hk, D, page = CASES[name]
    b = Batch(lengths, context, Hq, Hk, D, type, page, cap=sum(lengths) + 5, seed=len(name))
    rows = b.randn(b.cap, (Hq + 3) * D).to(BF16)  # queries among other things
    q = rows[:, D: (Hq + 1) * D].unflatten(1, (Hq, D))
    y = torch.full((b.cap, Hq, D), 9.0, dtype=BF16, device="cuda")
    out = b.attend(q, y=y)
    assert out.data_ptr() == y.data_ptr()
    b.check(q, y)
    assert bool((y[b.cu[-1]:] == 9.0).all())  # past the batch
    again = b.attend(q)
    assert torch.equal(again[: b.cu[-1]], y[: b.cu[-1]])
