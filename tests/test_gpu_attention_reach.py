"""How far a value that is not finite reaches: the rows that see it, and of the request's
own rows before it those of tiles that meet it with weights of zero.  A tile of T = 128 // g tokens (g query
heads on a key head) meets keys up to the end of the 128 that its last token is among: 126 + T past its first row
at most.  Everything else has to come out bit for bit as without it."""
from __future__ import annotations

import math

import pytest
import torch

from test_gpu_attention import BF16, Batch

pytestmark = pytest.mark.gpu


def reach(g):
    return 126 + 128 // g


def spoil(b, r, head, at, what):
    """Position ``at`` of request r, one channel of a key head's values."""
    page, slot = b.pages[r, at // b.page].long(), at % b.page
    if b.type == "e4m3":
        b.cache.v[page, head, slot], b.cache.v_exp[page, head, slot] = 0x7f, 255
    else:
        b.cache.v[page, head, slot, 11] = what


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("what", [math.nan, -math.inf])
@pytest.mark.parametrize("g,context,at", [
    (1, 1, 255), (1, 1, 256), (1, 0, 255), (1, 129, 383), (2, 1, 191), (2, 65, 255), (2, 0, 150), (3, 87, 255), (4, 97, 255), (4, 0, 150),
    (8, 113, 255), (16, 121, 255), (128, 128, 255), (1, 50, 399)])
def test_values_that_are_not_finite(type, what, g, context, at):
    lengths = [30, 350, 200]
    b = Batch(lengths, [200, context, 0], 2 * g, 2, 64, type, 32)
    q = b.randn(b.cap, 2 * g, 64).to(BF16)
    before = b.attend(q).clone()
    spoil(b, 1, 1, at, what)
    y = b.attend(q)
    assert b.cache.status() == 0
    row = b.cu[1] + at - context  # of the position, if the batch brings it
    sees = torch.zeros(b.cap, 2 * g, dtype=torch.bool, device="cuda")
    sees[max(row, b.cu[1]): b.cu[2], g:] = True
    may = torch.zeros_like(sees)
    may[max(row - reach(g), b.cu[1]): max(row, b.cu[1]), g:] = True
    assert bool((~torch.isfinite(y)).any(-1)[sees].all())
    rest = ~(sees | may)
    assert bool(rest[b.cu[1]: b.cu[1] + 1, :g].all())
    assert torch.equal(y[rest], before[rest])


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,g", [(8, 4), (32, 1), (2, 16)])
def test_drafts(type, n, g):
    """Few rows reach no further: among the rows of the same request."""
    b = Batch([n] * 5, [0, 40, 64, 100, 128 - n], 2 * g, 2, 128, type, 16)
    q = b.randn(b.cap, 2 * g, 128).to(BF16)
    before = b.attend(q).clone()
    for r in (1, 3):
        spoil(b, r, 0, b.context[r] + n - 1, math.nan)
    y = b.attend(q)
    for r in range(5):
        rows = slice(b.cu[r], b.cu[r + 1])
        if r in (1, 3):
            assert bool(torch.isnan(y[b.cu[r + 1] - 1, :g]).any(-1).all())
            assert torch.equal(y[rows, g:], before[rows, g:])
        else:
            assert torch.equal(y[rows], before[rows])
