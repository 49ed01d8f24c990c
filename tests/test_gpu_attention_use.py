"""The paged cache and its attention as a serving loop uses them, and the calls that
its documentation allows but that are easy to get wrong: values that are not
finite, plans of another shape, requests that do not fit, far offsets, captured
and replayed calls, several streams, workspaces with anything in them.

Tolerances are those of test_gpu_attention.py (Batch.check), which derives them.
"""
from __future__ import annotations

import math

import pytest
import torch

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.attention import KVCache
from rs_decode_gb300.prefill import Ragged, qk_norm
from test_gpu_attention import BF16, F64, I32, Batch, i32

pytestmark = pytest.mark.gpu

MIXED = dict(lengths=[1, 70, 3, 0, 200, 1, 40], context=[300, 65, 1000, 9, 0, 2000, 130])


def mixed(type="bf16", Hq=16, Hk=4, D=128, page=32, **kw):
    b = Batch(MIXED["lengths"], MIXED["context"], Hq, Hk, D, type, page, **kw)
    return b, b.randn(b.cap, Hq, D).to(BF16)


# ----------------------------------------------------------------------------- what is not finite
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("form", ["tokens", "mixed"])
@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_nan_stays_where_it_is_seen(type, form, which):
    if form == "tokens":
        b = Batch([1, 1, 1, 1], [300, 77, 1000, 5], 16, 4, 128, type, 32)
        q = b.randn(b.cap, 16, 128).to(BF16)
    else:
        b, q = mixed(type)
    before = b.attend(q).clone()
    r = 2 if form == "tokens" else 4                      # the request that gets one
    n, c, row = b.lengths[r], b.context[r], b.cu[r]
    at = c + n - 1 if form == "tokens" else 150            # its position
    if which == "q":
        q[row + at - c, 5] = math.nan
    else:
        arr, exp = getattr(b.cache, which), getattr(b.cache, which + "_exp")
        page, slot = b.pages[r, at // b.page].long(), at % b.page
        if type == "e4m3":
            arr[page, 1, slot], exp[page, 1, slot] = 0x7f, 255
        else:
            arr[page, 1, slot, 7] = math.nan
    y = b.attend(q)
    assert b.cache.status() == 0
    bad = torch.isnan(y).flatten(2).any(-1)               # [row, head]
    want = torch.zeros_like(bad)
    maybe = torch.zeros_like(bad)
    if which == "q":
        want[row + at - c, 5] = True
    else:
        want[row + at - c: row + n, 4:8] = True            # the rows that see it, the heads on key head 1
        if which == "v":
            maybe[max(row, row + at - c - 127): row + at - c, 4:8] = True
    assert bool((bad == want)[~maybe].all())
    assert torch.equal(y[~(want | maybe)], before[~(want | maybe)])


def test_infinite_and_huge_scores():
    """One key far above the rest takes all the weight; -inf scores take none."""
    b = Batch([1, 9], [200, 300], 8, 2, 64, "bf16", 64)
    for r in range(2):
        b.k[r][:, 5] = 100.0
        b.put(r, "k", b.k[r].float())
    q = torch.full((10, 8, 64), 100.0, dtype=BF16, device="cuda")
    y = b.attend(q, scale=10.0)
    for r in range(2):
        want = b.v[r][:, 5].repeat_interleave(4, 0).expand(b.lengths[r], 8, 64)
        # Not equal: c s of 9.2 million is 2^23 and more, so its fp32 product is off by up to a half and the one
        # weight is 2^d with |d| <= 1/2, in the sum of weights as it is and before the values rounded
        # to bf16, 2^-8 of itself at most; then y's rounding, 2^-8 of the result.
        assert bool(((y[b.cu[r]: b.cu[r + 1]].to(F64) - want).abs() <= (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -16) * want.abs()).all())
    k = torch.zeros(2, 201, 64, device="cuda")
    k[:, 7] = -3e38  # times 3e38: a score of minus infinity
    b.put(0, "k", k)
    q[0] = 3e38
    y = b.attend(q, scale=0.1)
    v = b.v[0][:, [i for i in range(201) if i != 7]].repeat_interleave(4, 0)
    assert bool(((y[0].to(F64) - v.mean(1)).abs() <= 2.0 ** -8 * v.mean(1).abs() + 2.0 ** -8 * v.abs().mean(1)).all())
    assert not torch.isnan(y).any()


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_a_tiny_scale_is_the_mean(type):
    """Down to scales whose products with a score are below fp32's normal range."""
    b, q = mixed(type)
    for scale in (1e-9, 1e-38):
        b.check(q, b.attend(q, scale=scale), scale=scale)


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4, 24])
def test_one_heavy_key_beside_many_light_ones(type, n):
    """20,000 equal weights of 2^-20 of the largest: each alone is nothing, together they are 2 %."""
    b = Batch([n], [20_000], 8, 1, 64, type, 64)
    k = torch.zeros(1, 20_000 + n, 64, device="cuda")
    k[:, 0] = 1.0
    b.k[0] = b.put(0, "k", k)
    v = torch.full((1, 20_000 + n, 64), 5.0, device="cuda")
    v[:, 0] = 0.0
    b.v[0] = b.put(0, "v", v)
    q = torch.full((n, 8, 64), 1.0, dtype=BF16, device="cuda")
    scale = 20 * math.log(2) / 64
    y = b.attend(q, scale=scale)
    ref, _ = b.reference(q, scale)
    assert float(((y.to(F64) - ref) / ref).abs().max()) <= 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10


def test_values_of_very_different_sizes():
    """8 bits: a token's values 2^30 above the others', with a weight of 2^-30: both parts count."""
    b = Batch([1], [700], 4, 1, 128, "e4m3", 16)
    k = torch.zeros(1, 701, 128, device="cuda")
    k[:, 400] = -1.0
    b.k[0] = b.put(0, "k", k)
    v = b.randn(1, 701, 128)
    v[:, 400] *= 2.0 ** 30
    b.v[0] = b.put(0, "v", v)
    q = torch.ones(1, 4, 128, dtype=BF16, device="cuda")
    scale = 30 * math.log(2) / 128
    b.check(q, b.attend(q, scale=scale), scale=scale)


# ----------------------------------------------------------------------------- what does not fit
def test_plan_of_another_shape_is_refused():
    b, q = mixed()
    y = torch.full((b.cap, 16, 128), 4.0, dtype=BF16, device="cuda")
    plan = b.cache.plan(b.ragged, 200)
    b.cache.attend(b.ragged, q, b.pages, plan, max_len=201, y=y)
    assert b.cache.status() == rb.DEV_LENGTH and bool((y == 4.0).all())
    b.cache.attend(b.ragged, q, b.pages, torch.zeros_like(plan), max_len=200, y=y)
    assert b.cache.status() == rb.DEV_LENGTH and bool((y == 4.0).all())
    wider = Ragged(len(b.lengths), b.cap + 100)  # as many requests, more rows
    wider.plan(i32([min(200, n + 10) for n in b.lengths]), i32([0] * len(b.lengths)))
    b.cache.attend(b.ragged, q, b.pages, b.cache.plan(wider, 200), max_len=200, y=y)
    assert b.cache.status() == rb.DEV_LENGTH and bool((y == 4.0).all())
    b.cache.attend(b.ragged, q, b.pages, plan, max_len=200, y=y)
    b.check(q, y)


def test_requests_that_do_not_fit():
    b, q = mixed()
    y = torch.full((b.cap, 16, 128), 4.0, dtype=BF16, device="cuda")
    plan = b.cache.plan(b.ragged, 70)  # 200 rows are too many
    assert b.cache.status() == rb.DEV_LENGTH
    b.cache.attend(b.ragged, q, b.pages, plan, max_len=70, y=y)
    gone = slice(b.cu[4], b.cu[5])
    kept = [i for i in range(b.cu[-1]) if not gone.start <= i < gone.stop]
    b.check(q, y, rows=kept)
    assert bool((y[gone] == 4.0).all())
    # an end past the page table's row: request 5 has 2,001 positions in 63 entries
    narrow = KVCache(16, 4, 128, b.n_pages, 62, page=32)
    narrow.k.copy_(b.cache.k), narrow.v.copy_(b.cache.v)
    y.fill_(4.0)
    plan = narrow.plan(b.ragged, 200)
    assert narrow.status() == rb.DEV_LENGTH
    narrow.attend(b.ragged, q, b.pages[:, :62].contiguous(), plan, max_len=200, y=y)
    b.check(q, y, rows=[i for i in range(b.cu[-1]) if i != b.cu[5]])
    assert bool((y[b.cu[5]] == 4.0).all())


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_entries_that_name_no_page(type):
    b, q = mixed(type)
    b.pages[1, 2], b.pages[5, 0] = -5, b.n_pages
    plan = b.cache.plan(b.ragged, b.max_len)
    y = b.cache.attend(b.ragged, q, b.pages, plan, max_len=b.max_len)
    assert b.cache.status() == rb.DEV_SLOT
    kept = [i for r in (0, 2, 4, 6) for i in range(b.cu[r], b.cu[r + 1])]
    b.check(q, y, rows=kept)


def test_nothing_to_do():
    b = Batch([0, 0], [5, 0], 8, 2, 64, cap=7)
    y = torch.full((7, 8, 64), 4.0, dtype=BF16, device="cuda")
    for n in (1, 50):
        b.attend(b.randn(7, 8, 64).to(BF16), max_len=n, y=y)
    b.cache.write(b.ragged, b.randn(7, 2, 64).to(BF16), b.randn(7, 2, 64).to(BF16), b.pages)
    assert bool((y == 4.0).all()) and b.cache.status() == 0


# ----------------------------------------------------------------------------- large
def test_far_pages():
    """Pages past 2^32 bytes, and past 2^31 elements."""
    Hk, page, n_pages = 8, 256, 20_000
    c = KVCache(16, Hk, 128, n_pages, 8, page=page)
    lengths, context = [1, 300, 3], [511, 0, 700]
    r = Ragged(3, sum(lengths))
    table = torch.tensor([[n_pages - 1 - 3 * j - i for j in range(8)] for i in range(3)], dtype=I32, device="cuda")
    full = [a + b for a, b in zip(lengths, context)]
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(sum(full), Hk, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
    fill = Ragged(3, sum(full))
    fill.plan(i32(full))
    c.write(fill, k, v, table)
    a, b = c.read(fill, table)
    assert torch.equal(a, k) and torch.equal(b, v)
    r.plan(i32(lengths), i32(context))
    q = torch.randn(sum(lengths), 16, 128, generator=g, device="cuda").to(BF16)
    y = c.attend(r, q, table, c.plan(r, 300), max_len=300)
    row = at = 0
    for n, ctx in zip(lengths, context):
        s = torch.einsum("thd,khd->htk", q[row: row + n].to(F64), k[at: at + n + ctx].to(F64).repeat_interleave(2, 1)) / math.sqrt(128)
        s.masked_fill_(torch.arange(n + ctx, device="cuda")[None] > ctx + torch.arange(n, device="cuda")[:, None], -math.inf)
        vv = v[at: at + n + ctx].to(F64).repeat_interleave(2, 1)
        p = torch.softmax(s, -1)
        ref, mag = torch.einsum("htk,khd->thd", p, vv), torch.einsum("htk,khd->thd", p, vv.abs())
        assert bool(((y[row: row + n].to(F64) - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag).all())
        row, at = row + n, at + n + ctx
    assert c.status() == 0


@pytest.mark.parametrize("n", [1, 5])
def test_rows_past_32_bits(n):
    """65,535 requests; with 5 rows each the packed rows' bytes pass 2^32."""
    R, Hq = 65_535, 64
    c = KVCache(Hq, 1, 128, 300, 1, page=16)
    g = torch.Generator(device="cuda").manual_seed(0)
    c.k.copy_(torch.randn(c.k.shape, generator=g, device="cuda"))
    c.v.copy_(torch.randn(c.v.shape, generator=g, device="cuda"))
    r = Ragged(R, R * n)
    lengths = torch.full((R,), n, dtype=I32, device="cuda")
    context = (torch.arange(R, device="cuda") % 11).to(I32)
    table = (torch.arange(R, device="cuda") % 300).to(I32)[:, None].contiguous()
    r.plan(lengths, context)
    q = torch.empty(R * n, Hq, 128, dtype=BF16, device="cuda").normal_(generator=g)
    y = c.attend(r, q, table, c.plan(r, n), max_len=n)
    for i in (0, 1, 31_000, 52_428, 52_429, R - 2, R - 1):
        ctx, page = i % 11, i % 300
        kk, vv = (t[page, 0, : ctx + n].to(F64) for t in (c.k, c.v))
        s = q[i * n: (i + 1) * n].to(F64) @ kk.T / math.sqrt(128)  # [row, head, key]
        s.masked_fill_(torch.arange(ctx + n, device="cuda") > ctx + torch.arange(n, device="cuda")[:, None, None], -math.inf)
        p = torch.softmax(s, -1)
        ref, mag = p @ vv, p @ vv.abs()
        got = y[i * n: (i + 1) * n].to(F64)
        assert bool(((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag).all()), i
    assert c.status() == 0


# ----------------------------------------------------------------------------- workspaces, streams, graphs
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_workspace_with_anything_in_it(type):
    b, q = mixed(type)
    first = b.attend(q)
    work = b.cache.workspace(b.ragged, b.max_len)
    work.fill_(0xff)
    assert torch.equal(b.attend(q, work=work), first)
    assert torch.equal(b.attend(q, work=work), first)  # as the last call left it


def test_two_layers_on_two_streams():
    """One plan, two caches, a workspace each, at the same time."""
    layers = [mixed(seed=s) for s in (1, 2)]
    (b0, _), (b1, _) = layers
    want = [b.attend(q).clone() for b, q in layers]
    plan = b0.cache.plan(b0.ragged, b0.max_len)
    work = [b.cache.workspace(b.ragged, b.max_len) for b, _ in layers]
    ys = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(20):
        for (b, q), w, y, s in zip(layers, work, ys, streams):
            b.cache.attend(b0.ragged, q, b.pages, plan, max_len=b0.max_len, y=y, work=w, stream=s)
    torch.cuda.synchronize()
    for y, w in zip(ys, want):
        assert torch.equal(y, w)


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_captured_decode_steps(type):
    """One step of a layer captured and replayed as the contexts grow, against 64 bits at each
    step; two such graphs of two layers, in turns, with a workspace that they share."""
    R, Hq, Hk, D, page, steps = 5, 8, 2, 64, 16, 24
    g = torch.Generator(device="cuda").manual_seed(3)
    context = i32([0, 7, 15, 16, 40])
    lengths = torch.ones(R, dtype=I32, device="cuda")
    table = torch.randperm(R * 5, generator=g, device="cuda").to(I32).view(R, 5)
    ragged = Ragged(R, R)
    inv_freq = (10000.0 ** (-torch.arange(0, 32, 2, device="cuda", dtype=F64) / 32)).float()
    layers = []
    for _ in range(2):
        c = KVCache(Hq, Hk, D, R * 5, 5, page=page, type=type)
        full = Ragged(R, 40 * R)
        full.plan(i32([40] * R))
        c.write(full, torch.randn(40 * R, Hk, D, generator=g, device="cuda").to(BF16), torch.randn(40 * R, Hk, D, generator=g, device="cuda").to(BF16), table)
        layers.append(dict(c=c, rows=torch.zeros(R, (Hq + 2 * Hk) * D, dtype=BF16, device="cuda")))
    plan, work = layers[0]["c"].plan(ragged, 1), layers[0]["c"].workspace(ragged, 1)

    def step(x):
        rows, c = x["rows"], x["c"]
        ragged.plan(lengths, context)
        c.plan(ragged, 1, out=plan)
        q, k = qk_norm(rows[:, :Hq * D].unflatten(1, (Hq, D)), rows[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)), norm="rms",
                       positions=ragged.token_pos, inv_freq=inv_freq)
        c.write(ragged, k, rows[:, (Hq + Hk) * D:].unflatten(1, (Hk, D)), table)
        x["q"], x["y"] = q, c.attend(ragged, q, table, plan, max_len=1, work=work)

    for x in layers:
        step(x)
        torch.cuda.synchronize()
        x["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(x["graph"]):
            step(x)
    whole = Ragged(R, 5 * page * R)
    for _ in range(steps):
        for x in layers:
            x["rows"].normal_(generator=g)
            x["graph"].replay()
        for x in layers:
            n = (context + 1).tolist()
            whole.plan(context + 1)
            k, v = x["c"].read(whole, table)
            at = 0
            for r in range(R):
                kk, vv = (t[at: at + n[r]].to(F64).repeat_interleave(Hq // Hk, 1) for t in (k, v))
                p = torch.softmax(torch.einsum("hd,khd->hk", x["q"][r].to(F64), kk) / math.sqrt(D), -1)
                ref, mag = torch.einsum("hk,khd->hd", p, vv), torch.einsum("hk,khd->hd", p, vv.abs())
                assert bool(((x["y"][r].to(F64) - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag).all())
                at += n[r]
            assert x["c"].status() == 0
        context += 1


# ----------------------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("type", ["bf16", "e4m3"])
def test_a_prompt_in_pieces(type):
    """Two conversations cached in turns of 130, 4, 1, 300, 17, 1 and 1 rows: every row's attention
    against one 64-bit pass over all of them."""
    Hq, Hk, D, page = 12, 3, 128, 32
    turns = [(130, 1), (4, 90), (1, 1), (300, 2), (17, 0), (1, 33), (1, 1)]
    total = [sum(t[i] for t in turns) for i in (0, 1)]
    b = Batch(total, [0, 0], Hq, Hk, D, type, page, garbage=True)
    rows = [[b.randn(n, h, D).to(BF16) for n in total] for h in (Hq, Hk, Hk)]
    done, out = [0, 0], [[], []]
    for turn in turns:
        ragged = Ragged(2, sum(turn) + 3)
        ragged.plan(i32(turn), i32(done))
        q, k, v = (torch.cat([x[i][done[i]: done[i] + turn[i]] for i in (0, 1)] + [torch.full((3, *x[0].shape[1:]), math.nan, device="cuda", dtype=BF16)])
                   for x in rows)
        b.cache.write(ragged, k, v, b.pages)
        y = b.cache.attend(ragged, q, b.pages, b.cache.plan(ragged, max(turn)), max_len=max(turn))
        out[0].append(y[: turn[0]].clone()), out[1].append(y[turn[0]: sum(turn)].clone())
        done = [a + n for a, n in zip(done, turn)]
    whole = Ragged(2, sum(total))
    whole.plan(i32(total))
    k, v = b.cache.read(whole, b.pages)
    b.k = [k[a: a + n].to(F64).transpose(0, 1) for a, n in zip((0, total[0]), total)]
    b.v = [v[a: a + n].to(F64).transpose(0, 1) for a, n in zip((0, total[0]), total)]
    b.check(torch.cat(rows[0]), torch.cat([torch.cat(o) for o in out]))


def test_the_example_s_attention_layer():
    """Ten tokens after a prompt, one at a time and in one pass: two results within 3e-3 of the same values."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prefill_decode.py")
    spec = importlib.util.spec_from_file_location("prefill_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main()["attention"] <= 2 * 3e-3
