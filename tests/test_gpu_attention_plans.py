"""Plans that were made for another call than the one they are given to: refused,
whatever the plan's buffer holds behind them, and y is left as it was."""
from __future__ import annotations

import pytest
import torch

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.prefill import Ragged
from test_gpu_attention import BF16, Batch, i32

pytestmark = pytest.mark.gpu


def attend(b, plan, q, y, max_len):
    """The C call: a plan's size is not checked there."""
    c = b.cache
    work = c.workspace(b.ragged, max_len)
    attn = rb.Attn(q.data_ptr(), b.Hq * b.D, b.pages.data_ptr(), b.D ** -0.5, max_len)
    rb.rs_attend(c.desc, c.kv, b.ragged.desc, b.ragged.arrays, attn, plan, y, work, c.status_word)


@pytest.mark.parametrize("type", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("small,large", [(1, 2), (3, 4), (3, 3000), (3000, 2999)])
def test_plan_of_another_number_of_requests(type, n, small, large):
    b = Batch([n] * 2 + [0] * (large - 2), [70, 70] + [0] * (large - 2), 8, 2, 64, type, 64, cap=100)
    q = b.randn(b.cap, 8, 64).to(BF16)
    y = torch.full((b.cap, 8, 64), 4.0, dtype=BF16, device="cuda")
    other = Ragged(small, b.cap)
    other.plan(i32([n] * min(2, small) + [0] * (small - 2)), i32([70] * small))
    plan = b.cache.plan(other, n)
    # alone, and where the call's own plan lay before
    attend(b, plan, q, y, n)
    assert b.cache.status() == rb.DEV_LENGTH and bool((y == 4.0).all())
    if small < large:
        own = b.cache.plan(b.ragged, n)
        own[: plan.numel()] = plan
        attend(b, own, q, y, n)
        assert b.cache.status() == rb.DEV_LENGTH and bool((y == 4.0).all())
    b.check(q, b.attend(q, y=y))
