"""Ragged prefill on the GPU at the ends of its inputs' ranges, against the
64-bit recurrence: large states, chunks that write nothing, outputs far smaller
than what enters them.

Tolerances, fixed before the first run, are those of test_gpu_prefill.py where
not said otherwise at a test.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from rs_decode_gb300 import binding as rb
from rs_decode_gb300.prefill import qk_norm
from test_gpu_prefill import TOL_BF16, Case, gdn_ref

pytestmark = pytest.mark.gpu


def scaled(c, scale):
    """The case with a checkpoint `scale` times as large."""
    c.S0 *= scale
    c.layer.init(c.S0)
    return c


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["no writes", "reset at the end", "no keys", "one written row"])
def test_large_states_where_nothing_is_written(d, what):
    """Chunks whose rows all have beta = 0, or end with a reset, or have no keys, with states and
    values of 2^16 times the keys: finite inputs give finite results."""
    c = scaled(Case([200, 64, 65, 3, 70], 4, 2, d, alpha="slow", seed=21), 1e5)
    c.v.copy_((c.v.float() * 2.0 ** 20).bfloat16())
    at = np.cumsum([0] + c.lengths)
    if what == "no writes":
        c.beta.zero_()
    elif what == "reset at the end":
        for a, n in zip(at, c.lengths):
            c.alpha[a + n - 1], c.beta[a + n - 1] = 0, 0
            if n > 64:
                c.alpha[a + 63], c.beta[a + 63] = 0, 0
    elif what == "no keys":
        c.k.zero_()
    else:
        keep = c.beta[at[:-1] + 1].clone()
        c.beta.zero_()
        c.beta[at[:-1] + 1] = keep
    c.run()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_states_near_the_end_of_fp32(d):
    """The bound of |S k| passes what fp32 holds, the products themselves do not."""
    c = scaled(Case([200, 13], 4, 2, d, alpha="slow", seed=22), 2e38)
    c.run()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k,rows", [(12, 1), (16, 1), (20, 1), (12, 8), (16, 8)])
def test_states_that_replace_far_larger_ones(d, k, rows):
    """A state 2^k times the values, forgotten in the middle of a chunk, at once or over eight rows:
    what is written behind it is as accurate as ever."""
    c = scaled(Case([64, 150], 4, 2, d, alpha="slow", seed=3), 10 * 2.0 ** k)
    for at in (20, 64 + 20, 64 + 100):
        c.alpha[at:at + rows] = 0 if rows == 1 else 2.0 ** (-2 * k / rows)
    c.run()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k,rows", [(13, 8), (14, 8), (14, 30), (18, 12)])
def test_large_states_that_fade(d, k, rows):
    """A state 2^k times the values that fades by 2^-2k within a chunk: rows on the way down are sums of
    small multiples of large values."""
    c = scaled(Case([64], 4, 2, d, alpha="slow", seed=3), 10 * 2.0 ** k)
    c.alpha[20:20 + rows] = 2.0 ** (-2 * k / rows)
    c.run()
    row = int(c.rows[0])
    x = [t.double() for t in (c.q.repeat_interleave(2, 1), c.k.repeat_interleave(2, 1), c.v, c.alpha, c.beta)]
    c.near(c.state()[row].double(), gdn_ref(c.first_state(0), *x)[1], 5e-6, "state")


# ----------------------------------------------------------------------------- outputs beside what enters them
# An output is a sum of terms of S q and P u.  Its error besides the rounding to
# bf16 is that of fp32 sums and of operands held to 22 bits, 5e-6 of the terms'
# magnitudes in the 2-norm as for the states, times 4 for the largest of a row
# against its mean.
TOL_TERMS = 2e-5


def rows_near(c):
    """Every output for itself, beside the magnitudes of the terms that it is the sum of."""
    rep, at = c.H // c.G, 0
    for r, n in enumerate(c.lengths):
        s = slice(at, at + n)
        q, k = (x[s].double().repeat_interleave(rep, 1) for x in (c.q, c.k))
        v, alpha, beta = c.v[s].double(), c.alpha[s].double(), c.beta[s].double()
        y = gdn_ref(c.first_state(r), q, k, v, alpha, beta)[0]
        S, A, terms = c.first_state(r), c.first_state(r).abs(), []
        for t in range(n):
            S, A = alpha[t][:, None, None] * S, alpha[t][:, None, None] * A
            u = beta[t][:, None] * (v[t] - torch.einsum("hn,hnp->hp", k[t], S))
            S, A = S + k[t][:, :, None] * u[:, None, :], A + k[t].abs()[:, :, None] * u.abs()[:, None, :]
            terms.append(torch.einsum("hn,hnp->hp", q[t].abs(), A))
        err = (c.y[s].double() - y).abs()
        over = (err - TOL_BF16 * y.abs()) / torch.stack(terms)
        assert bool(err.isfinite().all()) and float(over.max()) <= TOL_TERMS, f"request {r}: {float(over.max()):.1e}"
        at += n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[5, 12], [13, 64, 200], [2200]])
def test_queries_that_meet_little_of_a_large_state(d, lengths):
    """The state's largest part, on two keys, is at right angles to every query."""
    c = Case(lengths, 2, 1, d, alpha="one", beta="zero", seed=23)
    w = torch.randn(c.S0.shape[0], 2, d, device="cuda")
    c.S0[:, :, 0] -= 3000 * w
    c.S0[:, :, 1] += 1000 * w
    c.layer.init(c.S0)
    c.q[..., 0], c.q[..., 1] = 0.125, 0.375
    c.run()
    rows_near(c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[12], [13, 64, 200], [2200]])
def test_large_values_overwritten_by_small_ones(d, lengths):
    """One key all along, written in full: every other row takes a value a thousand times its own out again."""
    c = Case(lengths, 2, 1, d, alpha="one", beta="one", keys="same", seed=24)
    c.v[::2] = (c.v[::2].float() * 1000).bfloat16()
    c.run()
    rows_near(c)


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_are_not_biased(d):
    """Roundings to bf16 cancel over 2.6 million outputs (2^-9 / sqrt(2.6e6), 1.2e-6); 3e-5 leaves the sums' own."""
    c = Case([640] * 8, 4, 2, d, alpha="slow", seed=25)
    c.run()
    at, dot, square = 0, 0.0, 0.0
    for r, n in enumerate(c.lengths):
        s = slice(at, at + n)
        q, k = (x[s].double().repeat_interleave(2, 1) for x in (c.q, c.k))
        y = gdn_ref(c.first_state(r), q, k, c.v[s].double(), c.alpha[s].double(), c.beta[s].double())[0]
        dot, square, at = dot + float((c.y[s].double() * y).sum()), square + float(y.square().sum()), at + n
    assert abs(dot / square - 1) <= 3e-5


# ----------------------------------------------------------------------------- growing states
def growing(lengths, d, alpha):
    c = Case(lengths, 4, 2, d, seed=26)
    if alpha == "steps":  # up and down by 2^3, twice up in a row
        c.alpha.copy_(torch.tensor([8, 8, 1 / 64], device="cuda").repeat(c.cap // 3 + 1)[:c.cap, None].expand_as(c.alpha))
    elif alpha == "runs":  # 2^-52 down, 2^47 up
        c.alpha.copy_(torch.where((torch.arange(c.cap, device="cuda") // 30 % 2 == 0)[:, None], 0.3, 3.0).expand_as(c.alpha))
    else:
        c.alpha.fill_(alpha)
    c.q.copy_(c.k)
    c.run()
    return c


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("alpha", [1.0001, 1.05, "steps"])
def test_growth_within_a_chunk(d, alpha):
    c = growing([100, 12, 64, 13], d, alpha)
    c.check()
    rows_near(c)
    assert c.layer.status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("alpha", [1.2, 2.0, "runs"])
def test_too_much_growth_within_a_chunk_is_reported(d, alpha):
    c = growing([90, 64], d, alpha)
    assert c.layer.status() == rb.DEV_GATE


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("alpha", [1.2, 4.0, "runs"])
def test_growth_in_short_requests(d, alpha):
    """The recurrence has no such limit, also beside a chunk that does not grow."""
    c = growing([12, 5, 1], d, alpha)
    c.check()
    rows_near(c)
    c = Case([12, 64], 4, 2, d, seed=27)
    c.alpha[:12] = 4
    c.run()
    c.check()
    assert c.layer.status() == 0


# ----------------------------------------------------------------------------- norms
@pytest.mark.parametrize("eps", [1e-39, 0.0])
def test_norm_of_a_zero_head_with_the_smallest_eps(eps):
    q = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    q[1, 0] = 2.0
    out, _ = qk_norm(q, None, norm="l2", eps=eps, scale_q=3.0)
    ref = torch.zeros_like(q)
    ref[1, 0] = 3.0 * 128 ** -0.5
    assert torch.equal(out, ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("k,rows", [(8, 8), (12, 8), (12, 30)])
def test_outputs_while_a_large_state_fades(d, k, rows):
    """Every output for itself, beside its terms, while a state 2^k times the values fades by 2^-2k."""
    c = scaled(Case([64, 150], 4, 2, d, alpha="slow", seed=3), 10 * 2.0 ** k)
    for at in (20, 64 + 20, 64 + 80):
        c.alpha[at:at + rows] = 2.0 ** (-2 * k / rows)
    c.run()
    rows_near(c)
