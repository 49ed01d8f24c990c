"""Ragged prefill on the GPU where a request's chunks run in segments: every
width of the columns that join them, every precision, states kept inside
segments; and rows past 2^31 elements on the chunked path.

The tolerances are those of test_gpu_prefill.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from rs_decode_gb300 import binding as rb
from test_gpu_prefill import Case, dev

pytestmark = pytest.mark.gpu


def segments(c):
    """Segments that the workspace has room for, beyond what the same plan needs without any."""
    one, n = (rb.rs_prefill_bytes_for(c.layer.desc, c.rg.desc, m) for m in (13, max(c.lengths)))
    slabs, rest = divmod(n - one, 2 * len(c.lengths) * c.H * c.d * c.d * 4)
    assert rest == 0
    return slabs


# joined by 8 columns a CTA up to 152 x 8 / d chains, by 16 up to twice as many, by 32 above
@pytest.mark.parametrize("d,H,G,lengths,width", [
    (128, 9, 3, [2700], 8), (128, 12, 6, [2700], 16), (128, 19, 19, [3000], 16), (128, 32, 16, [3100], 32),
    (128, 30, 15, [2800, 90], 32), (64, 19, 19, [2700], 8), (64, 24, 12, [2700], 16), (64, 15, 5, [2900, 3, 2650], 32)])
def test_segments_of_every_width(d, H, G, lengths, width):
    chains = H * len(lengths)
    assert width == (8 if chains * d // 8 <= 152 else 16 if chains * d // 16 <= 152 else 32)
    c = Case(lengths, H, G, d, context=[29] + [0] * (len(lengths) - 1), seed=H, alpha="slow")
    assert segments(c) == min(304 // chains, (max(lengths) // 64 + 2) // 8) >= 5
    c.run([-1, 0, -2][:len(lengths)])
    c.check()
    assert c.layer.status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("prec", ["shared_bf16", "two"])
@pytest.mark.parametrize("start", [0, -2])
def test_segments_of_other_precisions(d, prec, start):
    """A pool or a checkpoint of the layer's precision to start from, a state kept every chunk."""
    c = Case([2750], 4, 2, d, prec, context=[64], block=64, seed=d, alpha="slow")
    assert segments(c) >= 5
    c.run([start])
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_chunked_rows_past_32_bits(d):
    """The long request's own rows, of q, k and v, lie on both sides of 2^31 elements."""
    H, G, ld = 2, 2, 1 << 24
    c = Case([2, 190], H, G, d, fused=False, seed=1)
    T = c.cap
    assert (T - 1) * ld > 1 << 31 > 2 * ld
    for name, heads in (("q", G), ("k", G), ("v", H)):
        x = getattr(c, name)
        big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, :heads * d].unflatten(1, (heads, d))
        big.copy_(x)
        setattr(c, name, big)
    slots = (1 << 31) // (H * d * d) + 2
    small = c.pool
    c.pool = torch.empty(slots, H, d, d, device="cuda")
    c.pool[0], c.pool[-1] = small[0], small[1]
    y = c.layer.prefill(c.rg, c.q, c.k, c.v, c.alpha, c.beta, max_len=T, rows=c.rows, start=dev(np.array([0, slots - 1], np.int32)),
                        pool=c.pool)
    c.pool0, c.pool, c.start, c.y = small, small, [0, 1], y
    c.check()
