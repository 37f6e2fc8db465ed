"""GPU tests of decode attention over the 4-bit cache at the ends of its number
ranges.  Inputs, oracle, metric and bound as in test_kv4_attn_gpu.py.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
import oracle
from oracle import kv4
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


@pytest.mark.parametrize("n_q,rep", [(2, 2), (5, 4)])
def test_f16_masks_of_the_lowest_value(n_q, rep):
    """A row hidden by -65504 throughout is the softmax of score - 65504 in fp32, whose unit there is 2^-8.  A score
    comes to lie at most half a unit, 2^-9, and what it is off itself (TOL) beside itself, a weight over the sum of the
    weights is off by twice that at most, and the output by as much of sum p |v|."""
    c = Case([50, 333], 2 * rep, 2, n_q, 128, dtype="f16", seed=3)
    low = torch.finfo(torch.float16).min
    m = torch.zeros((2, 1, n_q, c.cap), device="cuda", dtype=torch.float16)
    m[:, 0, 0] = low                                       # whole rows
    m[1, 0, 1, ::2] = low                                  # every other token of a row: as good as hidden
    got, ref, weight = np64(c.run(mask=m)), c.want(mask=m), c.want(mask=m, absolute=True)
    off = np.expm1(2 * (2.0 ** -9 + TOL)) * weight
    assert (np.abs(got - ref)[:, 0] <= off[:, 0]).all()
    rest = np.abs(got - ref)[:, 1:]
    assert rest.max() <= TOL * np.sqrt((ref[:, 1:] ** 2).mean())
    # the bound tells the row from one without weights: the mean of the values is further off
    plain = c.want(scale=0.0)[:, 0]
    assert (np.abs(plain - ref[:, 0]) > 2 * off[:, 0]).mean() > 0.5


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (256, 64)])
def test_many_rows_around_steps(dtype, dk, dv):
    """12 rows a kv head, two blocks; lengths around steps of 2 and 4 tiles and runs of several."""
    lens = [31, 32, 33, 47, 63, 64, 65, 95, 96, 97, 127, 128, 129, 191, 193, 0, 1]
    c = Case(lens, 8, 2, 3, dk, dv, page=16, dtype=dtype, seed=dk + dv)
    c.check()
    c.check(causal=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [1e5, 1e7, 1e8, 1e12, -1e20, 1e30])
def test_scores_up_to_the_largest_numbers(dtype, scale):
    """Scores of `scale` times a few units, far apart against their fp32 units: each row is its best token's values.
    Whole steps and a part of one, one CTA a unit and runs that are joined, one row and several a kv head."""
    for lens, H, n_q in (([64, 200], 4, 1), ([3000, 64, 900], 16, 3)):
        c = Case(lens, H, 2, n_q, 64, dtype=dtype, seed=6, page=64)
        q, k, v = np64(c.q), kv4.kept(np64(c.k)), kv4.kept(np64(c.v))
        got = np64(c.run(scale=scale))
        assert np.isfinite(got).all()
        for b, n in enumerate(lens):
            s = np.einsum("hid,hjd->hij", q[b], np.repeat(k[b, :, :n], H // 2, axis=0)) * np.sign(scale)
            order = np.sort(s, axis=-1)
            # the best token's lead, in natural units of the score, against what fp32 sums of 64 products are off by
            clear = (order[..., -1] - order[..., -2]) * abs(scale) > 30 + 2.0 ** -20 * 64 * abs(scale)
            assert clear.mean() > 0.5
            best = v[b, np.arange(H)[:, None] // (H // 2), s.argmax(-1)]           # (H, n_q, dv)
            off = np.abs(got[b].transpose(1, 0, 2) - best).max(-1)
            assert off[clear].max() <= TOL
