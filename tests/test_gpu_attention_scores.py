"""Scores far from zero, from 2^8 to 2^100 in the exponent: products of queries and keys are exact in fp32, so that
which keys share the weight is known.  Equal scores have equal weights wherever their keys lie (another tile, another
CTA's part), and the largest takes all from those below it.

Scores are equal or at least 1/16 of the largest apart, 2^4 in the exponent: in 64 bits and in 32 all weights but the equal
ones are 2^-16 at most, and off by 2^-24 of the largest score at 2^8, 2^-16 of themselves; above, they vanish.  So the bound
of each value is Batch.check's: the weights' rounding to bf16 (2^-8 A), y's own (2^-8 |y|), and 2^-10 A.  Its 2-norm is not asked
for: it takes the roundings of weights for independent, and equal weights have the same one."""
from __future__ import annotations

import pytest
import torch

from test_gpu_attention import BF16, Batch

pytestmark = pytest.mark.gpu

BATCHES = {  # new rows and keys before them of each request
    "tokens": ([1, 1, 1], [3000, 70, 900]),
    "drafts": ([4, 3, 4], [5000, 70, 300]),
    "a turn": ([40], [9000]),
    "turns": ([90, 40, 3, 130], [700, 3000, 1000, 0]),
    "a prompt": ([1500], [0]),
}


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (2, 2, 64)])
@pytest.mark.parametrize("size", [8, 24, 28, 30, 60, 100])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_scores_share_the_weight(type, name, Hq, Hk, D, size, sign):
    lengths, context = BATCHES[name]
    b = Batch(lengths, context, Hq, Hk, D, type, 64)
    for r, (n, c) in enumerate(zip(lengths, context)):
        # levels 1, 1.125 .. 1.875 that rise along the keys, so that later keys take the weight from earlier ones; the
        # keys of a level's last eighth and every 37th are equal, the others a level lower
        j = torch.arange(n + c, device="cuda")
        part = j * 8 // (n + c)
        level = part if sign > 0 else 7 - part
        even = (j % 37 == 0) | (j * 64 // (n + c) % 8 == 7)
        k = (1 + level / 8) * torch.where(even, 1.0, 0.5) * sign
        k = k[None, :, None].expand(Hk, -1, D)
        b.put(r, "k", k)
        b.k[r] = k.double()  # exact in either type
    q = torch.full((b.cap, Hq, D), 2.0 ** (size // 2), dtype=BF16, device="cuda")
    scale = 0.83 * 2.0 ** (size - size // 2) / D  # a score of k = 1: 1.2 * 2^size in the exponent
    y = b.attend(q, scale=scale).double()
    ref, mag = b.reference(q, scale)
    assert bool(((y - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * mag).all())
    assert b.cache.status() == 0
