"""The bound that the attention kernels' outputs are held to is one: exponentials and roundings
that are each off as far as they can be stay inside it."""

import os
import re

import numpy as np
import pytest

from oracle import attention as oa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_cubic_is_as_good_as_the_bound_says():
    """The prompt kernel's 2^x, step by step in fp32."""
    text = open(os.path.join(ROOT, "rank_bit_residual_b200", "csrc", "prompt_attention.cu")).read()
    body = text[text.index("uint64_t exp2_poly"):]
    body = body[:body.index("\n}")]
    c = [float(x) for x in re.findall(r"pk2\((0\.\d+)f, \1f\)", body)]
    assert len(c) == 4
    x = np.concatenate([np.linspace(-126, 8, 2000001), np.linspace(-1, 1, 200001)]).astype(np.float32)
    shift = np.float32(12582912.0)
    n = (x + shift) - shift
    f = (x - n).astype(np.float64)
    p = np.float32(c[0])
    for k in c[1:]:
        p = (p.astype(np.float64) * f + np.float64(np.float32(k))).astype(np.float32)
    err = p.astype(np.float64) * 2.0 ** n.astype(np.float64) / 2.0 ** x.astype(np.float64) - 1
    assert np.max(np.abs(err)) <= oa.EXP2_CUBIC


@pytest.mark.parametrize("center", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("exp2", [0.0, oa.EXP2_CUBIC])
def test_the_worst_errors_stay_inside(exp2, center):
    """Two equal weights, v = center +- 1, all errors on the same side."""
    v = center + np.array([1.0, -1.0])
    e = np.array([0.5 * (1 + exp2), 0.5 * (1 - exp2)])               # in fp32, as the total takes them
    r = 2.0 ** -8 / (1 + 2.0 ** -8)
    p = e * np.where(v > 0, 1 + r, 1 - r)
    got = np.sum(p * v) / np.sum(e)
    got += 2.0 ** -8 * abs(got)
    out, spread = np.mean(v), np.mean(np.abs(v))
    assert abs(got - out) <= oa.attention_tolerance(out, spread, 0.0, 64, 2, exp2)
