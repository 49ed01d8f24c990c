"""Plans that were made for another call than the one they are given to: refused,
whatever the plan's buffer holds behind them, and y is left as it was."""
from __future__ import annotations

import pytest
import torch

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.attention import KVCache
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


@pytest.mark.parametrize("type,other", [("bf16", "e4m3"), ("e4m3", "bf16")])
@pytest.mark.parametrize("Hq,Hk,n", [(8, 2, 1), (8, 2, 8), (8, 2, 9), (16, 1, 2), (40, 1, 1), (128, 2, 30)])
def test_plan_for_a_cache_of_another_type(type, other, Hq, Hk, n):
    """Also where both types run the same form: up to 32 rows of a group, or more than 32 heads in it."""
    b = Batch([n, 1, 0], [300, 5, 0], Hq, Hk, 64, type, 16)
    q = b.randn(b.cap, Hq, 64).to(BF16)
    y = torch.full((b.cap, Hq, 64), 4.0, dtype=BF16, device="cuda")
    plan = KVCache(Hq, Hk, 64, b.n_pages, b.max_pages, page=16, type=other).plan(b.ragged, n)
    b.cache.attend(b.ragged, q, b.pages, plan, max_len=n, y=y)
    assert b.cache.status() == rb.DEV_LENGTH and bool((y == 4.0).all())
    b.check(q, b.attend(q, y=y))
