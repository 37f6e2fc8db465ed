"""GPU tests of page tables, rotary positions, writes and attention as one program uses them: with the 4-bit cache
too, drafted tokens that are given up again, two programs' streams at once, a process whose first call is captured.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
import oracle
from oracle import kv4, paged
from oracle.attn import attention

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().double().cpu().numpy()


class Server:
    """A pool of pages and the tables of B sequences; the oracle of each kept on the host."""

    def __init__(self, B, n_pages, max_pages, page=16):
        self.page, self.B = page, B
        self.free, self.count = i32(list(range(n_pages))), i32([n_pages])
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def add(self, new, n_new):
        self.lens += new
        return gdn.page_assign(self.table, self.lens, self.free, self.count, self.page, n_new, new)


def test_tables_serve_the_4_bit_cache():
    """Prompts of unequal length and steps of one token over gdn_kv4_write and gdn_flash_attn_kv4."""
    B, H, Hkv, d = 3, 8, 2, 128
    s = Server(B, 60, 12)
    cache = gdn.kv4_cache(60, Hkv, 16, d)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda").bfloat16()  # noqa: E731
    prompt = [50, 7, 100]
    k, v = randn(B, Hkv, 100, d), randn(B, Hkv, 100, d)
    s.add(i32(prompt), 100)
    gdn.kv4_write(k, v, cache, s.table, s.lens, i32(prompt))
    ks = [[k[b, :, :n]] for b, n in enumerate(prompt)]
    vs = [[v[b, :, :n]] for b, n in enumerate(prompt)]
    one = i32([1] * B)
    for _ in range(20):
        k, v, q = randn(B, Hkv, 1, d), randn(B, Hkv, 1, d), randn(B, H, 1, d)
        s.add(one, 1)
        gdn.kv4_write(k, v, cache, s.table, s.lens)
        out = gdn.flash_attn_kv4(q, cache, s.table, s.lens)
        for b in range(B):
            ks[b].append(k[b])
            vs[b].append(v[b])
    assert gdn.device_status() == gdn.OK
    for b in range(B):
        kk, vv = (kv4.kept(np64(torch.cat(x, dim=1)))[None] for x in (ks[b], vs[b]))
        assert oracle.parity_error(np64(out[b:b + 1]), attention(np64(q[b:b + 1]), kk, vv)) <= 1e-4


def test_drafts_are_checked_and_given_up():
    """Steps of 4 drafted tokens of which some are kept: the others' pages go back, their rows stay without effect."""
    B, H, Hkv, d, n_q = 4, 8, 4, 64, 4
    s = Server(B, 100, 20)
    kc, vc = gdn.paged_cache(100, Hkv, 16, d, dtype=torch.float16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    rng = np.random.default_rng(3)
    rows = [[] for _ in range(B)]
    for step in range(12):
        q, k, v = (torch.randn((B, n_q, h, d), generator=gen, device="cuda").half() for h in (H, Hkv, Hkv))
        new = i32([n_q] * B)
        slots, _, _ = s.add(new, n_q)
        gdn.paged_write(k.flatten(0, 1), v.flatten(0, 1), kc, vc, slots.flatten())
        out = gdn.flash_attn_paged(q.transpose(1, 2), kc, vc, s.table, s.lens, causal=True)
        kept = rng.integers(0, n_q + 1, B)
        for b in range(B):
            kk = np.stack([r[0] for r in rows[b]] + list(np64(k[b])))
            vv = np.stack([r[1] for r in rows[b]] + list(np64(v[b])))
            n = len(kk)
            hide = np.where(np.arange(n)[None] > n - n_q + np.arange(n_q)[:, None], -np.inf, 0.0)[None, None]
            ref = attention(np64(q[b]).transpose(1, 0, 2)[None], kk.transpose(1, 0, 2)[None], vv.transpose(1, 0, 2)[None], hide)
            assert oracle.parity_error(np64(out[b:b + 1]), ref) <= 1e-4
            rows[b] += [(np64(k[b, i]), np64(v[b, i])) for i in range(kept[b])]
        before = s.lens.clone()
        s.lens -= i32(n_q - kept)
        gdn.page_release(s.table, before, s.free, s.count, 16, s.lens)
        held = sum(-(-len(r) // 16) for r in rows)
        assert int(s.count) == 100 - held and s.lens.tolist() == [len(r) for r in rows]
    assert gdn.device_status() == gdn.OK


def test_steps_of_two_programs_at_once():
    """Each on a stream of its own, with workspaces from the library and their own pools."""
    def program(stream, seed, steps):
        with torch.cuda.stream(stream):
            B, H, Hkv, d, n = 2, 16, 2, 128, 3000
            gen = torch.Generator(device="cuda")
            gen.manual_seed(seed)
            randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda").bfloat16()  # noqa: E731
            s, plan = Server(B, 500, 300), gdn.rotary_plan(d)
            kc, vc = gdn.paged_cache(500, Hkv, 16, d)
            outs = []
            for step in range(steps):
                m = n if step == 0 else 1
                slots, pos, _ = s.add(i32([m] * B), m)
                q = gdn.rotary_write(randn(B * m, H, d), randn(B * m, Hkv, d), randn(B * m, Hkv, d), pos.flatten(), plan,
                                     kc, vc, slots.flatten())
                outs.append(gdn.flash_attn_paged(q.view(B, m, H, d)[:, -1:].transpose(1, 2), kc, vc, s.table, s.lens))
            return outs
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    alone = []
    for x, seed in zip(streams, (5, 6)):
        alone.append(program(x, seed, 6))
        torch.cuda.synchronize()
    both = [program(x, seed, 6) for x, seed in zip(streams, (5, 6))]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(alone, both) for a, b in zip(x, y))
    assert gdn.device_status() == gdn.OK


FIRST = """
import torch
import linear_attention_sequence_gated_gb300 as gdn
B, H, Hkv, n, d, page = 2, 8, 2, 5000, 128, 64
pages = -(-n // page)
table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
free = torch.arange(2 * pages + 1, dtype=torch.int32, device="cuda")
count = torch.tensor([2 * pages + 1], dtype=torch.int32, device="cuda")
lens = torch.tensor([n, 77], dtype=torch.int32, device="cuda")
q, k, v = (torch.randn((n + 77, h, d), device="cuda").bfloat16() for h in (H, Hkv, Hkv))
kc, vc = gdn.paged_cache(2 * pages + 1, Hkv, page, d)
plan = gdn.rotary_plan(d)
torch.cuda.synchronize()
was = table.clone(), count.clone()


def call():
    slots, pos, _ = gdn.page_assign(table, lens, free, count, page, n, lens, n_tokens=n + 77)
    turned = gdn.rotary_write(q, k, v, pos, plan, kc, vc, slots)
    return gdn.flash_attn_paged(turned[-2:].unsqueeze(2), kc, vc, table, lens)


g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, capture_error_mode="MODE"):
    out = call()
g.replay()
torch.cuda.synchronize()
table.copy_(was[0])
count.copy_(was[1])
assert torch.isfinite(out).all() and torch.equal(out, call()) and gdn.device_status() == gdn.OK
"""


@pytest.mark.parametrize("mode", ["global", "thread_local"])
def test_the_first_calls_of_a_process_can_be_captured(mode):
    r = subprocess.run([sys.executable, "-c", FIRST.replace("MODE", mode)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.returncode == 0, r.stderr[-2000:]
