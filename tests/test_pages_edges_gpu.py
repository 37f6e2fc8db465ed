"""GPU tests of page tables, slots and positions where calls could be misread, for equality with the oracle (oracle/paged.py).
"""
import random

import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
from oracle import paged
from test_pages_gpu import Pool, built, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 7, 1500])
def test_packed_prompts_need_no_bound(B):
    """Without n_new, a packed call takes as many of each sequence as new_lens says."""
    rng = random.Random(B)
    p = Pool(B, 12, B * 12, 16, seed=B)
    lens = [0] * B
    for _ in range(2):
        new = [rng.choice([0, 1, 15, 40, 90]) for _ in range(B)]
        lens = [a + n for a, n in zip(lens, new)]
        got = gdn.page_assign(p.table, i32(lens), p.free, p.count, 16, new_lens=i32(new), n_tokens=sum(new))
        want = paged.assign(p.h_table, lens, new, p.h_free, 16, sum(new), sum(new))
        assert want[3] and gdn.device_status() == gdn.OK
        assert [x.tolist() for x in got] == list(want[:3])
        p.same()


def test_default_of_new_tokens():
    """One each, but for packed calls with new_lens; a sequence takes no more than n_new, and that shows."""
    p = Pool(3, 12, 30, 16)
    s, _, none = gdn.page_assign(p.table, i32([1, 1, 1]), p.free, p.count, 16)
    assert tuple(s.shape) == (3, 1) and none is None
    s, q, _ = gdn.page_assign(p.table, i32([2, 2, 2]), p.free, p.count, 16, n_tokens=3)
    assert q.tolist() == [1, 1, 1] and gdn.device_status() == gdn.OK
    s, q, o = gdn.page_assign(p.table, i32([2, 2, 2]), p.free, p.count, 16, new_lens=i32([0, 0, 0]), n_tokens=0)
    assert o.tolist() == [0] * 4 and gdn.device_status() == gdn.OK


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B", [5, 5000])
def test_more_new_tokens_than_allowed_show(packed, B):
    p = Pool(B, 6, B * 6, 16, seed=3)
    new = [2] * B
    p.assign(new, 2, new, 2 * B if packed else None, ok=True)
    new[B // 2] = 3
    lens = [2 + n for n in new]
    p.assign(lens, 2, new, 2 * B + 1 if packed else None, ok=False)
    p.assign([n + 2 for n in lens], 2, ok=True)


def test_as_many_entries_as_a_full_stack_holds():
    """The stack's entries and those given back are 2^31 together: nothing fits, and nothing is written anywhere."""
    n = 1 << 30
    table = torch.zeros((1, n), dtype=torch.int32, device="cuda")
    both = torch.full((n + 1024,), -5, dtype=torch.int32, device="cuda")
    free, count = both[512:512 + n], i32([n])
    gdn.page_release(table, i32([n]), free, count, 1)
    assert gdn.device_status() == gdn.ERR_PAGE and int(count) == n
    assert all(bool((x == -5).all()) for x in both.split(1 << 28))


@pytest.mark.parametrize("gaps", [False, True])
def test_more_pages_back_than_a_cluster_holds_at_once(gaps):
    """Over 65536 entries a CTA takes its share in several turns; with entries that name no page among them."""
    rng = random.Random(4)
    lens = [rng.randint(0, 60000) for _ in range(9)] + [0, 40000]
    n = sum(lens)
    assert n > 3 * 65536
    p = Pool(len(lens), 60000, n + 5, 1, seed=5)
    p.assign(lens, 60000, lens, n, ok=True)
    if gaps:
        for b, j in ((0, 7), (4, 0), (10, 39999)):
            p.table[b, j] = p.h_table[b, j] = -1
    stay = [a // 5 for a in lens]
    p.release(lens, stay)
    p.release(stay)
