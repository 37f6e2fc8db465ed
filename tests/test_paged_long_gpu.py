"""GPU tests of rotary positions and writes at numbers of tokens where warps share a token's rows in other ways, against the
oracle.  Bounds as in tests/test_paged_gpu.py.
"""
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
from oracle import paged
from test_paged_gpu import DTYPES, built, freqs_of, near, np64, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("T,H,Hk,d,r", [(150, 24, 3, 128, 128), (607, 8, 2, 128, 128), (609, 8, 2, 128, 64), (3647, 4, 2, 128, 32),
                                        (3700, 5, 3, 128, 128), (5001, 6, 1, 256, 64), (20011, 1, 1, 64, 32)])
def test_many_tokens(dtype, neighbours, T, H, Hk, d, r):
    q, k = randn((T, H, d), dtype, 1), randn((T, Hk, d), dtype, 2)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 5 - 9
    plan = gdn.rotary_plan(r, 1e5, neighbours=neighbours)
    for got, x in zip(gdn.rotary(q, k, pos, plan), (q, k)):
        near(got, paged.rotary(np64(x), np64(pos)[None], freqs_of(r, 1e5), [0] * (r // 2), neighbours), np64(x), r, neighbours)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [700, 6001])
@pytest.mark.parametrize("token_major", [False, True])
def test_turning_and_writing_prompts(dtype, T, token_major):
    """One call is the two that it stands for, bit for bit; rows of no slot are written nowhere."""
    H, Hk, d, page = 8, 2, 128, 64
    q, k, v = randn((T, H, d), dtype, 1), randn((T, Hk, d), dtype, 2), randn((T, Hk, d), dtype, 3)
    pos, plan = torch.arange(T, dtype=torch.int32, device="cuda"), gdn.rotary_plan(d)
    n_pages = -(-T // page) + 1
    slots = torch.randperm(n_pages * page, generator=torch.Generator("cuda").manual_seed(4), device="cuda")[:T].to(torch.int32)
    slots[::7] = -1
    caches = []
    for _ in range(2):
        shape = (n_pages, page, Hk, d) if token_major else (n_pages, Hk, page, d)
        pair = [torch.full(shape, 7.0, dtype=DTYPES[dtype], device="cuda") for _ in "kv"]
        caches.append([x.transpose(1, 2) if token_major else x for x in pair])
    got = gdn.rotary_write(q, k, v, pos, plan, *caches[0], slots)
    qo, ko = gdn.rotary(q, k, pos, plan)
    gdn.paged_write(ko, v, *caches[1], slots)
    torch.cuda.synchronize()
    assert torch.equal(got, qo) and all(torch.equal(x, y) for x, y in zip(*caches)) and gdn.device_status() == gdn.OK
    t = torch.nonzero(slots >= 0).flatten()
    at = slots[t].long()
    assert torch.equal(caches[0][0][at // page, :, at % page], ko[t]) and torch.equal(caches[0][1][at // page, :, at % page], v[t])
