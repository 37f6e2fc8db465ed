"""GPU tests of decode attention over a paged cache of 16- and 32-bit rows where its arithmetic could go wrong.  Cases,
metric and tolerance are those of tests/test_paged_attn_gpu.py.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
import oracle
from test_paged_attn_gpu import DTYPES, TOL, Case, built, np64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H,n_q", [(8, 1), (16, 1), (8, 5)])
def test_16_bit_outputs_are_the_rounded_32_bit_ones(dtype, H, n_q):
    """One rounding at the end: weights keep as many bits whatever the output's type."""
    c = Case([3000, 17, 0, 640], H, 2, n_q, 128, dtype=dtype, seed=41)
    assert torch.equal(c.run(out_dtype=DTYPES[dtype]), c.run().to(DTYPES[dtype]))


# The largest finite numbers of each type; of fp32 also bf16's lowest twice over, and the first that rounds up to 2^128 at 11 bits.
BIG = [(t, x) for t in DTYPES for x in (torch.finfo(DTYPES[t]).max, torch.finfo(DTYPES[t]).min)] + \
    [("f32", np.array(x, dtype=np.uint32).view(np.float32).item()) for x in (0xff7fff7f, 0x7f7ff000)]


@pytest.mark.parametrize("dtype,big", BIG)
@pytest.mark.parametrize("heads,n_q", [(4, 1), (16, 1), (8, 5)])
def test_hidden_tokens_may_hold_the_largest_numbers(dtype, big, heads, n_q):
    """Behind a sequence's end, hidden by a mask, after a query's own place."""
    c = Case([50, 37, 64, 1], heads, 2, n_q, 128, dtype=dtype, seed=14)
    for x in (c.kc, c.vc):
        x.copy_(torch.where(x.isnan(), torch.full_like(x, big), x))
    c.check()
    c.check(causal=True)
    m = c.mask()
    m[0, 0, :, 5] = m[1, 0, :, 36] = m[2, 0, :, 20] = -float("inf")
    for b, tok in ((0, 5), (1, 36), (2, 20)):
        for x in (c.kc, c.vc):
            x[int(c.table[b, tok // 32]), :, tok % 32] = big
    c.check(mask=m)
    c.check(mask=m, causal=True)


@pytest.mark.parametrize("dtype,big", BIG)
@pytest.mark.parametrize("heads,n_q", [(4, 1), (8, 5)])
def test_the_largest_numbers_are_numbers(dtype, big, heads, n_q):
    """Values, keys and queries of that size that are seen: one of a row's each, so that no sum passes the type."""
    c = Case([64, 1, 640, 45], heads, 2, n_q, 128, dtype=dtype, seed=15)
    small = 32.0 / 2.0 ** np.round(np.log2(abs(big)))        # a power of two: scores of 32 scale = 2.8
    for b, tok in ((0, 20), (1, 0), (2, 333), (3, 44)):
        p = int(c.table[b, tok // 32])
        c.vc[p, :, tok % 32, 7] = big
        c.kc[p, :, tok % 32, 3] = big
    c.q[..., 3] = small
    used = c.table.flatten().long()
    c.kc[used, :, :, 9] = torch.where(c.kc[used, :, :, 9].isnan(), c.kc[used, :, :, 9], torch.full_like(c.kc[used, :, :, 9], small))
    c.q[..., 9] = big
    got, ref = np64(c.run()), c.want()
    torch.cuda.synchronize()
    assert gdn.device_status() == gdn.OK and np.isfinite(got).all()
    # a weight is off by no more of itself than the tolerance (the sums that its bound is for are the same here)
    assert (np.abs(got[..., 7] - ref[..., 7]) <= TOL * np.abs(ref[..., 7]) + 1e-3).all()
    rest = np.arange(128) != 7
    assert oracle.parity_error(got[..., rest], ref[..., rest]) <= TOL


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("heads,n_q", [(4, 1), (16, 1), (8, 5)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_seen_infinities_reach_their_element_only(dtype, heads, n_q, bad):
    """In the middle of a long sequence, at its end, in its only tile: not finite there, and everything else as before."""
    c = Case([3000, 41, 16, 64], heads, 2, n_q, 128, dtype=dtype, seed=16)
    want = c.run()
    for b, tok in ((0, 1501), (1, 40), (2, 3)):
        c.vc[int(c.table[b, tok // 32]), 1, tok % 32, 7] = bad
    got = c.run()
    torch.cuda.synchronize()
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[:3, :, heads // 2:, 7] = True
    assert not torch.isfinite(got[hit]).any()
    assert torch.equal(got[3], want[3]) and torch.equal(got[:, :, :heads // 2], want[:, :, :heads // 2])
    # (a tile with such a value may be summed in another order)
    assert oracle.parity_error(np64(got[~hit]), np64(want[~hit])) <= TOL
