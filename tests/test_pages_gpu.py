"""GPU tests of page tables, slots and positions made on the device, for equality with the oracle
(oracle/paged.py).
"""
import random

import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
from oracle import paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """A pool of pages, tables and lengths on the device, and the same on the host."""

    def __init__(self, B, max_pages, n_pages, page, seed=0):
        rng = random.Random(seed)
        order = list(range(n_pages))
        rng.shuffle(order)
        self.page, self.n_pages = page, n_pages
        self.h_free, self.h_table = order, np.full((B, max_pages), -7, dtype=np.int64)
        self.free, self.count = i32(order + []).reshape(-1), i32([n_pages])
        self.table = torch.full((B, max_pages), -7, dtype=torch.int32, device="cuda")

    def assign(self, lens, n_new, new=None, n_tokens=None, ok=None):
        got = gdn.page_assign(self.table, i32(lens), self.free, self.count, self.page, n_new,
                              None if new is None else i32(new), n_tokens=n_tokens)
        want = paged.assign(self.h_table, lens, new, self.h_free, self.page, n_new, n_tokens)
        assert gdn.device_status() == (gdn.OK if want[3] else gdn.ERR_PAGE)
        assert ok is None or want[3] == ok
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1]
        assert got[2] is None if n_tokens is None else got[2].tolist() == want[2]
        self.same()
        return got

    def release(self, before, after=None):
        gdn.page_release(self.table, i32(before), self.free, self.count, self.page, None if after is None else i32(after))
        self.h_free, ok = paged.release(self.h_table, before, after, self.h_free, self.page, self.n_pages)
        assert gdn.device_status() == (gdn.OK if ok else gdn.ERR_PAGE)
        self.same()

    def same(self):
        assert self.table.tolist() == self.h_table.tolist()
        n = int(self.count)
        assert n == len(self.h_free) and self.free[:n].tolist() == self.h_free


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("packed", [False, True])
def test_steps_of_a_batch(page, packed):
    """Prompts, then steps of one and of several tokens, some sequences without any, some ended and begun again."""
    rng = random.Random(page)
    B = 9
    p = Pool(B, 400 // page + 2, B * (400 // page + 1) + 3, page, seed=page)
    lens = [0] * B
    for most in (100, 1, 1, 7, 40, 1, 3):
        new = [rng.randint(0, most) for _ in range(B)]
        lens = [a + b for a, b in zip(lens, new)]
        p.assign(lens, most, new, sum(new) + 2 if packed else None, ok=True)
        if most == 7:
            ended = [a if i % 3 == 0 else 0 for i, a in enumerate(lens)]
            p.release(ended)
            lens = [0 if i % 3 == 0 else a for i, a in enumerate(lens)]


def test_every_sequence_takes_n_new():
    p = Pool(4, 10, 40, 16)
    p.assign([5, 16, 17, 40], 5)
    p.assign([6, 17, 18, 41], 1)
    p.assign([6, 17, 18, 41], 0)


def test_a_step_called_off_leaves_the_stack_as_it_was():
    p = Pool(5, 30, 160, 8, seed=3)
    lens = [30, 0, 7, 8, 100]
    p.assign(lens, 100, lens)
    was, n = p.free.clone(), p.count.clone()
    more = [a + b for a, b in zip(lens, (9, 3, 1, 1, 60))]
    p.assign(more, 60, [9, 3, 1, 1, 60])
    p.release(more, lens)
    assert torch.equal(p.count, n) and torch.equal(p.free, was)


@pytest.mark.parametrize("B", [1, 31, 1024, 1025, 5000, 16384])
def test_many_sequences(B):
    """Sums over more sequences than a block has threads; clusters of CTAs."""
    rng = random.Random(B)
    p = Pool(B, 6, B * 4, 16, seed=B)
    new = [rng.choice([0, 1, 16, 17, 40]) for _ in range(B)]
    p.assign(new, 40, new, sum(new), ok=True)
    lens = [a + 1 for a in new]
    p.assign(lens, 1)
    p.release(lens, [a // 2 for a in lens])


def test_long_prompts():
    p = Pool(3, 9000, 20000, 16, seed=9)
    lens = [100003, 3, 60000]
    p.assign(lens, 100003, lens, sum(lens), ok=True)
    p.release(lens)


def test_the_stack_runs_out():
    """The pages that are left go to the first that need them; giving back what was handed out restores them."""
    p = Pool(4, 10, 6, 16, seed=5)
    p.assign([20, 40, 33, 10], 40, [20, 40, 33, 10], ok=False)
    assert int(p.count) == 0
    p.release([20, 40, 33, 10])
    assert int(p.count) == 6


def test_what_only_the_device_can_see():
    p = Pool(3, 4, 30, 16, seed=6)
    p.assign([64, 70, -5], 70, [64, 70, 3], ok=False)             # beyond the table; an empty one
    p.release([64, 70, -5])
    p.assign([3, 2, 0], 5, [5, -4, 2], n_tokens=10, ok=True)      # more new tokens than tokens, negative counts
    p.release([3, 2, 0])
    p.assign([3, 9, 4], 9, [3, 9, 4], n_tokens=10, ok=False)      # more than the packed tensors hold
    # a table that names no page where a sequence goes on, and one that names a page outside the pool
    p = Pool(2, 4, 8, 16, seed=7)
    p.table[1, 0] = 8
    s, _, _ = gdn.page_assign(p.table, i32([5, 5]), p.free, p.count, 16)
    assert s.tolist() == [[-1], [-1]] and gdn.device_status() == gdn.ERR_PAGE
    # counts outside the stack
    for bad in (-3, 9):
        p = Pool(1, 4, 8, 16)
        p.count.fill_(bad)
        s, _, _ = gdn.page_assign(p.table, i32([1]), p.free, p.count, 16)
        assert gdn.device_status() == gdn.ERR_PAGE
        assert int(p.count) == (0 if bad < 0 else 7) and int(s) == (-1 if bad < 0 else int(p.free[7]) * 16)
    # no room on the stack
    p = Pool(1, 4, 8, 16)
    p.table[0] = i32([1, 2, 3, 4])
    p.count.fill_(6)
    gdn.page_release(p.table, i32([64]), p.free, p.count, 16)
    assert gdn.device_status() == gdn.ERR_PAGE and int(p.count) == 8 and p.free[6:].tolist() == [4, 3]


def test_no_sequences():
    t = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    none, free, count = i32([]), i32([3, 4]), i32([2])
    s, q, o = gdn.page_assign(t, none, free, count, 16, n_tokens=3)
    assert s.tolist() == [-1] * 3 and q.tolist() == [0] * 3 and o.tolist() == [0] and int(count) == 2
    s, q, o = gdn.page_assign(t, none, free, count, 16)
    assert tuple(s.shape) == (0, 1) and o is None
    gdn.page_release(t, none, free, count, 16)
    assert int(count) == 2 and gdn.device_status() == gdn.OK


def test_captured_steps_follow_the_lengths():
    """A captured step is replayed on other lengths, tables and stacks, on another stream than the default."""
    p = Pool(40, 20, 900, 16, seed=8)
    lens = [3 * i for i in range(40)]
    p.assign(lens, 120, lens)
    d_lens = i32(lens)
    out = [torch.empty((40, 1), dtype=torch.int32, device="cuda") for _ in range(2)]
    was = p.table.clone(), p.count.clone(), d_lens.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d_lens += 1
        gdn.page_assign(p.table, d_lens, p.free, p.count, 16, slots=out[0], positions=out[1])
    for t, w in zip((p.table, p.count, d_lens), was):
        t.copy_(w)
    for _ in range(40):
        g.replay()
        lens = [a + 1 for a in lens]
        want = paged.assign(p.h_table, lens, None, p.h_free, 16, 1)
        assert out[0].tolist() == want[0] and out[1].tolist() == want[1]
        p.same()
    assert gdn.device_status() == gdn.OK
