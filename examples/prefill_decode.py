"""Prompts into the decode state, then decoding, then a second batch that reuses
a cached prefix: the calls of one Gated DeltaNet layer in a serving loop, and of
one attention layer beside it.

    python examples/prefill_decode.py

Per batch of requests: one plan (``Ragged.plan``, on the GPU, from lengths that
only the GPU needs to know), then per layer the norms of q and k (``qk_norm``)
and the delta rule over all packed rows (``Layer.prefill``), which leaves each
request's state where ``Layer.decode`` continues it and keeps the state after
every ``BLOCK`` tokens in a pool.  A later request that starts with the same
tokens begins from such a state instead of from nothing.

The attention layer takes the same batches: the norms with rotation, the new rows'
keys and values into the pages of a cache (``KVCache.write``), and the attention over
it (``KVCache.attend``), for prompts and single tokens alike.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from rs_decode_gb300 import build  # noqa: E402
from rs_decode_gb300.attention import KVCache  # noqa: E402
from rs_decode_gb300.layer import Layer  # noqa: E402
from rs_decode_gb300.prefill import Ragged, qk_norm  # noqa: E402

H, G, D, WINDOW, BLOCK = 32, 16, 128, 16, 256
HQ, HK, ROT, PAGE = 32, 4, 64, 64  # the attention layer: query heads, key heads, rotated channels, tokens of a page


def project(tokens: torch.Tensor, seed: int = 0) -> dict:
    """Stands in for a layer's projections: rows that depend on the token alone,
    queries, keys and values side by side, and the gates alpha, beta."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randn(1000, (2 * G + H) * D, generator=g, device="cuda", dtype=torch.bfloat16)
    gates = torch.randn(2, 1000, H, generator=g, device="cuda")
    rows = table[tokens]
    return dict(q=rows[:, :G * D].unflatten(1, (G, D)), k=rows[:, G * D:2 * G * D].unflatten(1, (G, D)),
                v=rows[:, 2 * G * D:].unflatten(1, (H, D)),
                alpha=torch.exp(-0.05 * torch.nn.functional.softplus(gates[0][tokens])),
                beta=torch.sigmoid(gates[1][tokens]))


def prefill(layer: Layer, requests: list, context: list, start: list, rows: list, pool: torch.Tensor, free: list):
    """One batch: requests' new tokens, the tokens before them, the pool slots
    (or -1) that they start from, their state rows.  Returns y and the plan."""
    lengths = [len(t) for t in requests]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ragged = Ragged(len(requests), sum(lengths), block=BLOCK,
                    max_blocks=max(1, max((c + n) // BLOCK for c, n in zip(context, lengths))), n_free=len(free))
    ragged.plan(i32(lengths), i32(context), i32(free))
    p = project(torch.cat(requests))
    q, k = qk_norm(p["q"], p["k"], norm="l2", scale_q=D ** -0.5)
    y = layer.prefill(ragged, q, k, p["v"], p["alpha"], p["beta"], max_len=max(lengths), rows=i32(rows), start=i32(start),
                      pool=pool)
    return y, ragged


def decode(layer: Layer, tokens: torch.Tensor) -> torch.Tensor:
    """One step for all rows of the layer."""
    p = project(tokens)
    q, k = qk_norm(p["q"], p["k"], norm="l2", scale_q=D ** -0.5)
    d = dict(q=q, k=k, v=p["v"].contiguous(), alpha=p["alpha"], beta=p["beta"])
    return layer.decode({n: t.view(torch.int16) if t.dtype == torch.bfloat16 else t for n, t in d.items()}, {})


def attend(cache: KVCache, pages: torch.Tensor, requests: list, context: list) -> torch.Tensor:
    """One batch of the attention layer: requests' new tokens behind the tokens before them."""
    lengths = [len(t) for t in requests]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = torch.randn(1000, (HQ + 2 * HK) * D, generator=g, device="cuda", dtype=torch.bfloat16)[torch.cat(requests)]
    inv_freq = 10000.0 ** (-torch.arange(0, ROT, 2, device="cuda", dtype=torch.float32) / ROT)
    ragged = Ragged(len(requests), sum(lengths))
    ragged.plan(i32(lengths), i32(context))
    plan = cache.plan(ragged, max(lengths))  # serves all attention layers of the batch
    q, k = qk_norm(rows[:, :HQ * D].unflatten(1, (HQ, D)), rows[:, HQ * D:(HQ + HK) * D].unflatten(1, (HK, D)), norm="rms",
                   positions=ragged.token_pos, inv_freq=inv_freq)
    cache.write(ragged, k, rows[:, (HQ + HK) * D:].unflatten(1, (HK, D)), pages)
    return cache.attend(ragged, q, pages, plan, max_len=max(lengths))


def main() -> dict:
    build.build()
    g = torch.Generator(device="cuda").manual_seed(1)
    text = lambda n: torch.randint(0, 1000, (n,), generator=g, device="cuda")
    layer = Layer("gdn", 4, H, G, D, D, WINDOW)
    layer.init()
    pool = torch.zeros(32, H, D, D, device="cuda")

    # four prompts of different lengths, packed
    prompts = [text(n) for n in (700, 33, 1500, 256)]
    y, plan = prefill(layer, prompts, [0] * 4, [-1] * 4, [0, 1, 2, 3], pool, list(range(32)))
    taken = plan.counts.tolist()[2]
    table = plan.block_table.tolist()
    print(f"prefill: {y.shape[0]} rows, {taken} states kept: {table}")

    # ten tokens each, from the same states
    steps = [text(4) for _ in range(10)]
    for t in steps:
        out = decode(layer, t)
    print("decoded 10 tokens for each request; |y| =", [round(float(o.norm()), 3) for o in out])

    # a new request that shares request 2's first 1280 tokens: it starts from the state
    # kept there; the same one from nothing gives the same state
    prefix, rest = prompts[2][:1280], text(90)
    again, _ = prefill(layer, [rest, torch.cat([prefix, rest])], [1280, 0], [table[2][1280 // BLOCK - 1], -1], [1, 3], pool,
                       list(range(taken, 32)))
    a, b = layer.checkpoint_hp()[1], layer.checkpoint_hp()[3]
    apart = float((a - b).norm() / b.norm())
    print(f"prefix reuse: 90 rows instead of 1370; the states differ by {apart:.1e}")
    assert layer.status() == 0
    # the steps above by prefill instead of decoding: one request's ten tokens as a continuation
    layer2 = Layer("gdn", 1, H, G, D, D, WINDOW)
    layer2.init()
    ten = torch.stack([t[0] for t in steps])
    y2, _ = prefill(layer2, [torch.cat([prompts[0], ten])], [0], [-1], [0], pool, list(range(24, 32)))
    step_apart = float((y2[-1].float() - out[0]).norm() / out[0].norm())
    print(f"the last decoded row against the same row of a prefill: {step_apart:.1e}")

    # the attention layer: the same prompts, then the same ten tokens each, one at a time; the last of
    # them against the same row of one pass over the whole request
    cache = KVCache(HQ, HK, D, 100, 30, page=PAGE)
    pages = torch.randperm(100, generator=g, device="cuda").to(torch.int32)
    table = torch.full((4, 30), -1, dtype=torch.int32, device="cuda")
    used = 0
    for r, p in enumerate(prompts):
        need = (len(p) + len(steps) + PAGE - 1) // PAGE
        table[r, :need] = pages[used:used + need]
        used += need
    attend(cache, table, prompts, [0] * 4)
    for i, t in enumerate(steps):
        last = attend(cache, table, list(t.view(4, 1)), [len(p) + i for p in prompts])
    whole = attend(cache, table, [torch.cat([p, torch.stack([t[r] for t in steps])]) for r, p in enumerate(prompts)], [0] * 4)
    ends = torch.tensor([len(p) + len(steps) for p in prompts], device="cuda").cumsum(0) - 1
    attention_apart = float((whole[ends].float() - last.float()).norm() / last.float().norm())
    print(f"attention: {used} pages; the last token's rows against those of one pass over the prompts: {attention_apart:.1e}")
    assert cache.status() == 0
    return {"prefix": apart, "step": step_apart, "taken": taken, "attention": attention_apart}


if __name__ == "__main__":
    main()
