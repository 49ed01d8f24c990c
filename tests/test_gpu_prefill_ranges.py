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

from test_gpu_prefill import Case

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
