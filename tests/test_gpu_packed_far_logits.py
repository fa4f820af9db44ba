"""Attention over packed and 16-bit pages with logits far below zero."""
import math

import numpy as np
import pytest
import torch

from tests.packed_reference import PAGE
from tests.test_gpu_packed_attention import KINDS, Cache
from tests.test_gpu_packed_range import _attend, _params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", ["packed", "sixteen", "mixed"])
def test_logits_far_below_zero(kap, kinds):
    """Every token has the logit -2^113: all are seen, so the output is the mean of the values."""
    n, d = 300, 64
    c = Cache(kap, [n], 1, 2, d, KINDS[kinds], seed=6)
    # the first dim alone meets the query: -2^56 in every key (as a packed group: code 0 of that lowest value)
    c.K[:, :, :, 0] = -(2.0 ** 56)
    c.packed[:, :, 0:512].view(c.P4, 1, PAGE, 32)[..., 0] &= 0xF0
    _params(c)[:, :, 0, :, :, 1] = -(2.0 ** 56)
    q = torch.zeros(1, 2, d, dtype=torch.bfloat16)
    q[:, :, 0] = 2.0 ** 60
    out, lse = _attend(kap, c, n, q)
    vals = np.stack([c.page(int(c.bt[0, i // PAGE]), 0)[i % PAGE][1] for i in range(n)])
    vabs = np.stack([c.page(int(c.bt[0, i // PAGE]), 0)[i % PAGE][4] for i in range(n)])
    # fp32 sums of n terms, p * scale as fp16 (2^-11), the output to bf16
    mean, tol = vals.mean(0), vabs.mean(0) * (n * 2.0 ** -24 + 2.0 ** -11)
    for head in range(2):
        got = out[0, head].double().cpu().numpy()
        assert (np.abs(got - mean) <= tol + 2.0 ** -8 * np.abs(mean)).all()
        assert abs(float(lse[0, head]) + 2.0 ** 113) <= 2.0 ** 113 * 2.0 ** -21
        assert math.isfinite(float(lse[0, head]))
