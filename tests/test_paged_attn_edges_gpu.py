"""GPU tests of decode attention over a paged cache of 16- and 32-bit rows where its arithmetic could go wrong.  Cases,
metric and tolerance are those of tests/test_paged_attn_gpu.py.
"""
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn  # noqa: F401
from test_paged_attn_gpu import DTYPES, Case, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,n_q", [(8, 1), (16, 1), (8, 5)])
def test_16_bit_outputs_are_the_rounded_32_bit_ones(dtype, H, n_q):
    """One rounding at the end: weights keep as many bits whatever the output's type."""
    c = Case([3000, 17, 0, 640], H, 2, n_q, 128, dtype=dtype, seed=41)
    assert torch.equal(c.run(out_dtype=DTYPES[dtype]), c.run().to(DTYPES[dtype]))
