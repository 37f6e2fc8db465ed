"""GPU test of what gdn_kv4_read writes for tokens that are not there: zeros with
a positive sign, whatever the cache's bytes say."""
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256)])
def test_absent_rows_are_positive_zeros(dtype, dk, dv):
    """Rows behind the counts, before the start and on pages that the cache does not have, over bytes of negative codes
    and of infinite scales; numbers that are there keep their signs."""
    B, Hkv, n = 4, 2, 70
    cache = torch.full((B * 5, Hkv, 1, 9 * (dk + dv)), 0xff, dtype=torch.uint8, device="cuda")
    table = torch.arange(B * 5, dtype=torch.int32, device="cuda").reshape(B, 5)
    lens = torch.tensor([n, 37, 16, 3], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((B, Hkv, n, d), device="cuda").to(dtype) for d in (dk, dv))
    gdn.kv4_write(k, v, cache, table, lens, lens)
    for count in (lens, lens - 2, None):
        back = gdn.kv4_read(cache, table, lens, n, dk, dv, lens=count, dtype=dtype)
        for x, y in zip((k, v), back):
            for b, have in enumerate(lens.tolist()):
                c = n if count is None else int(count[b])
                first = max(0, c - have)                   # rows before the sequence's start
                assert not (y[b, :, :first] != 0).any() and not torch.signbit(y[b, :, :first]).any()
                assert not (y[b, :, c:] != 0).any() and not torch.signbit(y[b, :, c:]).any()
                there, kept = x[b, :, have - (c - first):have], y[b, :, first:c]
                assert ((kept == 0) | (torch.signbit(kept) == torch.signbit(there))).all()
    assert gdn.device_status() == gdn.OK
    table[0, 1] = -1
    ky, vy = gdn.kv4_read(cache, table, lens, n, dk, dv, lens=lens, dtype=dtype)
    for y in (ky, vy):
        assert not (y[0, :, 16:32] != 0).any() and not torch.signbit(y[0, :, 16:32]).any()
        assert (y[0, :, :16] != 0).any() and (y[0, :, 32:] != 0).any()
    assert gdn.device_status() == gdn.ERR_PAGE
