"""GPU tests of decode attention over the 4-bit cache at the ends of its number
ranges.  Inputs, oracle, metric and bound as in test_kv4_attn_gpu.py.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
import oracle
from test_kv4_attn_gpu import Case, TOL, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()


@pytest.mark.parametrize("rep", [1, 5])
def test_fp32_queries_up_to_the_largest_number(rep):
    """Elements of +-FLT_MAX beside others of a few 2^124, with the scale that brings the scores back to a few units."""
    c = Case([60, 300], 2 * rep, 2, 1, 64, dtype="f32", seed=4)
    top = torch.finfo(torch.float32).max
    base = c.q * 2.0 ** 124
    for at, sign in ((3, 1.0), (40, -1.0)):
        c.q = base.clone()
        c.q[..., at] = sign * top
        got, _ = c.check(scale=2.0 ** -128)
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("e", [-111, -113, -124, -126])
def test_queries_down_to_the_least_normal_number(dtype, e):
    """Rows whose largest elements are near 2^(e + 2), their small ones subnormal, with the scale that brings them back."""
    c = Case([60, 300], 8, 2, 1, 64, dtype=dtype, seed=5)
    c.q = (c.q.double() * 2.0 ** e).to(c.q.dtype)
    c.check(scale=2.0 ** -e / 8)
