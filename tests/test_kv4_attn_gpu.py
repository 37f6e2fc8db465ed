"""GPU tests of decode attention over the 4-bit cache against the float64
oracle (oracle/attn.py) on the values that the cache keeps (oracle/kv4.py).

Metric, as for flash_attn: max |gpu - oracle| / RMS(oracle), bound 1e-4 for
fp32 outputs.  The cache's values enter exactly, q exactly or with 22 bits, the
softmax weights with 22 bits (11 where queries and outputs are 16-bit).  Scores accumulate in fp32 over at most 256
products, 16 at a time: an error of at most some 16 units of 2^-23 of
sum |q k| scale (below 16 for these inputs), 3e-5, if every rounding went one way, and a
hundredth of that as they do; a weight is off by as much of itself.  16-bit outputs may
be off by half a step more, and by what weights rounded to f16 (half a step: 2^-11 of
each) move the sum: at most 2^-11 sum p |v|, which is the oracle's output for |v|.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
import oracle
from oracle import kv4
from oracle.attn import attention

pytestmark = pytest.mark.gpu

TOL = 1e-4
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Case:
    """A written cache in pages of random order, over bytes that hold anything elsewhere."""

    def __init__(self, lens, H, Hkv, n_q, dk, dv=None, page=32, dtype="bf16", seed=0, room=0, held="f32"):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        dv = dv or dk
        B, n = len(lens), max(max(lens), 1)
        max_pages = -(-n // page) + room
        f = dict(generator=gen, device="cuda")
        self.cache = torch.randint(0, 256, (B * max_pages + 2, Hkv, page // 16, 9 * (dk + dv)), dtype=torch.uint8,
                                   **f)
        self.table = torch.randperm(B * max_pages + 2, **f)[:B * max_pages].to(torch.int32).reshape(B, max_pages)
        self.table = self.table.contiguous()
        self.lens, self.lens_l, self.dv, self.cap = i32(lens), lens, dv, max_pages * page
        self.k = torch.randn((B, Hkv, n, dk), **f).to(DTYPES[held])
        self.v = torch.randn((B, Hkv, n, dv), **f).to(DTYPES[held])
        gdn.kv4_write(self.k, self.v, self.cache, self.table, self.lens, self.lens)
        self.q = torch.randn((B, H, n_q, dk), **f).to(DTYPES[dtype])
        self.f = f

    def mask(self, std=0.5, hide=0.2):
        B, _, n_q, _ = self.q.shape
        m = torch.randn((B, 1, n_q, self.cap), **self.f) * std
        m[torch.rand(m.shape, **self.f) < hide] = -float("inf")
        return m.to(self.q.dtype)

    def run(self, mask=None, scale=None, **kw):
        return gdn.flash_attn_kv4(self.q, self.cache, self.table, self.lens, self.dv, mask, scale, **kw)

    def want(self, mask=None, scale=None, causal=False, absolute=False):
        q, m = np64(self.q), np64(mask)
        B, H, n_q, dk = q.shape
        scale = float(np.float32(1 / np.sqrt(dk) if scale is None else scale))
        k, v = kv4.kept(np64(self.k)), kv4.kept(np64(self.v))
        if absolute:
            v = np.abs(v)
        out = np.zeros((B, n_q, H, self.dv))
        for b, n in enumerate(self.lens_l):
            n = max(n, 0)
            add = np.zeros((1, 1, n_q, n)) if m is None else m[b:b + 1, :, :, :n].copy()
            if causal:
                j, i = np.arange(n)[None], np.arange(n_q)[:, None]
                add = np.where(j > n - n_q + i, -np.inf, add)
            out[b] = attention(q[b:b + 1], k[b:b + 1, :, :n], v[b:b + 1, :, :n], add, scale)[0]
        return out

    def check(self, tol=TOL, out_dtype=None, **kw):
        got = self.run(out_dtype=out_dtype, **kw)
        kw.pop("workspace", None)
        ref = self.want(**kw)
        torch.cuda.synchronize()
        assert gdn.device_status() == gdn.OK
        y = np64(got)
        assert y.shape == ref.shape and np.isfinite(y).all()
        if got.dtype == torch.float32:
            assert oracle.parity_error(y, ref) <= tol
        else:
            step = torch.finfo(got.dtype).eps / 2
            off = tol * np.sqrt((ref ** 2).mean()) + 2.0 ** -11 * self.want(absolute=True, **kw)
            assert (np.abs(y - ref) <= off + step * (np.abs(ref) + off) + 2.0 ** -25).all()
        return got, ref


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (64, 256), (256, 128), (128, 64), (64, 128),
                                   (128, 256), (256, 64)])
def test_widths_types_and_lengths(dtype, dk, dv):
    """Lengths of one token, inside, at and past tiles and pages, and an empty sequence."""
    c = Case([1, 0, 15, 16, 17, 31, 33, 100, 200, 64], 8, 2, 1, dk, dv, dtype=dtype, seed=dk + 3 * dv)
    got, _ = c.check()
    assert not got[1].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,n_q", [(1, 1, 1), (8, 8, 1), (16, 2, 1), (9, 1, 1), (32, 2, 1), (8, 2, 5), (10, 2, 19),
                                       (3, 3, 2), (24, 1, 3), (40, 1, 19)])
@pytest.mark.parametrize("causal", [False, True])
def test_head_groups_and_query_counts(dtype, H, Hkv, n_q, causal):
    """Rows from 1 to 760 a kv head, causal among the newest tokens; queries before the start of a short sequence."""
    c = Case([300, 3, 0, 77], H, Hkv, n_q, 128, dtype=dtype, seed=H + n_q)
    got, ref = c.check(causal=causal)
    if causal and n_q > 3:
        assert not ref[1, :n_q - 3].any() and not got[1, :n_q - 3].any()


@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_masks(page, dtype):
    """An additive mask with hidden tokens, whole rows hidden, and columns behind the sequences that hold anything."""
    c = Case([130, 17, 200], 4, 2, 3, 64, page=page, dtype=dtype, seed=page, room=1)
    m = c.mask()
    m[0, 0, 1] = -float("inf")
    m[1, 0, :, 17:] = float("nan")
    got, ref = c.check(mask=m)
    assert not got[0, 1].any()
    c.check(mask=m, causal=True)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_masks_of_the_lowest_value(dtype):
    """A row hidden by the type's lowest value is the softmax of what it says: all scores drown in it, weights are equal."""
    c = Case([50, 33], 4, 2, 2, 128, dtype=dtype, seed=3)
    low = torch.finfo(DTYPES[dtype]).min
    m = torch.zeros((2, 1, 2, c.cap), device="cuda", dtype=DTYPES[dtype])
    m[0, 0, 0] = low
    m[1, 0, :, ::2] = low
    got = c.run(mask=m)
    ref = c.want(mask=m)
    if dtype == "f16":       # scores do not drown in -65504 as an exact number; fp32 keeps 2^-7 of them
        ref[0, 0] = got[0, 0].double().cpu().numpy()
        spread = np.abs(np64(got[0, 0]))
        assert np.isfinite(spread).all() and spread.max() > 0
    if dtype != "f16":
        for h in range(4):
            mean = kv4.kept(np64(c.v))[0, h // 2, :50].mean(axis=0)
            assert np.abs(np64(got[0, 0, h]) - mean).max() < 1e-5
            ref[0, 0, h] = mean
    assert oracle.parity_error(np64(got), ref) <= TOL


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scale", [1.0, 0.0, -0.5, 20.0])
def test_scales(dtype, scale):
    """Uniform and very peaked weights.  At scale 20 scores reach 1e3: their fp32 units alone move a weight by 1e-4."""
    c = Case([100, 300], 4, 4, 2, 128, dtype=dtype, seed=8)
    c.check(scale=scale, tol=TOL if abs(scale) <= 1 else 1e-2)


def test_queries_of_many_magnitudes():
    """Rows of q from 2^-120 to 2^100, with the scale that brings them back, and zero rows."""
    c = Case([60], 8, 2, 1, 128, dtype="bf16", seed=9)
    base = c.q.clone()
    for e in (-120, -40, 40, 100):
        c.q = base * 2.0 ** e
        c.check(scale=2.0 ** -e / 11 if e > -120 else 2.0 ** 119 / 11)
    c.q = base * 0
    c.check()


def test_an_infinite_or_nan_query_spoils_its_own_row_only():
    c = Case([60, 20], 8, 2, 1, 64, dtype="f32", seed=10)
    want = c.run()
    c.q[0, 3, 0, 5] = float("nan")
    c.q[1, 6, 0, 7] = float("inf")
    got = c.run()
    torch.cuda.synchronize()
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 0, 3] = True
    bad[1, 0, 6] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dv", [64, 128, 256])
def test_16_bit_outputs(dtype, dv):
    c = Case([1, 40, 700, 0], 8, 2, 2, 128, dv, dtype=dtype, seed=11)
    got, _ = c.check(out_dtype=DTYPES[dtype])
    assert got.dtype == DTYPES[dtype] and not got[3].any()


@pytest.mark.parametrize("lens", [[20001], [9000, 1, 5], [1] * 70, [0, 0, 3000, 0] * 12, [40000, 41]])
def test_work_shared_unevenly(lens):
    """One long sequence over the whole GPU, many one-token ones, empty ones between."""
    H, Hkv = (4, 2) if max(lens) > 10000 else (8, 4)
    Case(lens, H, Hkv, 1, 64 if max(lens) > 10000 else 128, page=64, seed=len(lens)).check()


def test_more_sequences_than_a_warp_scans_at_once():
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 40, 150)]
    Case(lens, 4, 2, 1, 64, page=16, seed=12).check()


def test_values_of_cache_bytes_behind_the_end_do_not_matter():
    """Codes and scale bytes (infinities and NaN among them) of absent tokens, in the last tile and in unused pages."""
    c = Case([5, 21, 48], 4, 2, 2, 128, page=16, seed=13)
    want = c.run()
    other = Case([5, 21, 48], 4, 2, 2, 128, page=16, seed=13)
    keep = other.cache.clone()
    other.cache.fill_(0xff)
    gdn.kv4_write(other.k, other.v, other.cache, other.table, other.lens, other.lens)
    assert not torch.equal(keep, other.cache)
    assert torch.equal(other.run(), want)


def test_bad_pages_are_reported_and_left_out():
    c = Case([40, 40], 4, 2, 1, 64, page=16, seed=14)
    good = c.table.clone()
    c.table[0, 1], c.table[1, 2] = c.cache.shape[0], -7
    got = c.run()
    assert gdn.device_status() == gdn.ERR_PAGE and gdn.device_status() == gdn.OK
    m = torch.zeros((2, 1, 1, c.cap), dtype=c.q.dtype, device="cuda")
    m[0, ..., 16:32] = -float("inf")
    m[1, ..., 32:] = -float("inf")
    assert oracle.parity_error(np64(got), c.want(mask=m)) <= TOL
    c.table = good
    c.check()
    c.lens += 100                                          # past the table: what it reaches is attended to
    got = c.run()
    assert gdn.device_status() == gdn.ERR_PAGE
    c.lens = i32([c.cap, c.cap])
    again = c.run()                                        # (tokens 40 on were never written: any values, the same ones)
    assert torch.allclose(got, again, rtol=0, atol=0, equal_nan=True) and gdn.device_status() == gdn.OK
    c.lens = i32([-3, 40])
    assert not c.run()[0].any() and gdn.device_status() == gdn.OK


def test_a_length_past_the_table_is_reported_wherever_it_stands():
    """In the middle of a run over several short sequences, and as a CTA's own."""
    for B, at in ((200, 101), (200, 0), (9, 4)):
        c = Case([16] * B, 2, 2, 1, 64, page=16, seed=B)
        want = c.run()
        assert gdn.device_status() == gdn.OK
        c.lens[at] = 17
        got = c.run()
        assert gdn.device_status() == gdn.ERR_PAGE and torch.equal(got, want)


@pytest.mark.parametrize("B", [3, 200])
def test_a_table_without_pages(B):
    """Rows are zeros; a length above its room is reported."""
    cache, q = gdn.kv4_cache(0, 2, 16, 64), torch.randn((B, 4, 2, 64), device="cuda")
    table, lens = i32([[]] * B), i32([0] * B)
    for n, status in ((0, gdn.OK), (5, gdn.ERR_PAGE)):
        lens[B - 1] = n
        out = gdn.flash_attn_kv4(q, cache, table, lens, out=torch.ones((B, 2, 4, 64), device="cuda"))
        assert not out.any() and gdn.device_status() == status


def test_more_sequences_than_a_grid_has_rows():
    """70000 sequences of up to 3 tokens: written, read back, attended to."""
    B, d = 70000, 64
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 4, B)
    k, v = (torch.randn((B, 1, 3, d), device="cuda") for _ in range(2))
    cache = gdn.kv4_cache(B, 1, 16, d)
    table = torch.randperm(B, device="cuda").to(torch.int32).reshape(B, 1)
    n = i32(lens.tolist())
    gdn.kv4_write(k, v, cache, table, n, n)
    rk, rv = gdn.kv4_read(cache, table, n, 3, d, lens=n, dtype=torch.float32)
    there = np.arange(3)[None] < lens[:, None]
    kk, vk = (kv4.kept(np64(x)) * there[:, None, :, None] for x in (k, v))
    assert np.array_equal(np64(rk), kk) and np.array_equal(np64(rv), vk)
    q = torch.randn((B, 2, 1, d), device="cuda").to(torch.bfloat16)
    got = np64(gdn.flash_attn_kv4(q, cache, table, n))[:, 0]                   # (B, H, d)
    s = np.einsum("bhd,bnd->bhn", np64(q)[:, :, 0], kk[:, 0]) * float(np.float32(d ** -0.5))
    p = np.exp(s) * there[:, None]
    ref = np.einsum("bhn,bnd->bhd", p / np.maximum(p.sum(-1, keepdims=True), 1e-300), vk[:, 0])
    assert oracle.parity_error(got, ref) <= TOL and gdn.device_status() == gdn.OK


def test_shared_pages():
    """Two sequences that begin with the same pages."""
    c = Case([64, 64], 4, 2, 1, 128, page=32, seed=15)
    c.table[1, 0] = c.table[0, 0]
    c.k[1, :, :32], c.v[1, :, :32] = c.k[0, :, :32], c.v[0, :, :32]
    c.check()


def test_same_result_every_time_with_any_workspace_and_on_two_streams_at_once():
    c = Case([3000, 17, 1234], 8, 4, 2, 128, page=64, seed=16)
    want, _ = c.check()
    need = gdn.flash_attn_kv4_workspace_bytes(3, 8, 4, 2, 128, 128, 64, c.table.shape[1])
    ws = [torch.full((need,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s, w in zip(streams, ws):
            outs.append(c.run(workspace=w, stream=s))
            outs.append(c.run(stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with pytest.raises(gdn.GdnError) as e:
        c.run(workspace=ws[0][:need - 256])
    assert e.value.status == gdn.ERR_WORKSPACE


def test_a_decode_loop_captured_once():
    """Append, attend, repeat: the captured step against the oracle at every length; two graphs replayed in turn."""
    B, H, Hkv, d, page = 2, 4, 2, 128, 16
    total = 50
    c = Case([total, total - 9], H, Hkv, 1, d, page=page, seed=17)
    k, v = c.k.clone(), c.v.clone()
    c.cache.fill_(0xff)
    nk, nv, lens = k[:, :, :1].clone(), v[:, :, :1].clone(), i32([0, -9])
    qs = torch.randn((total, B, H, 1, d), device="cuda").to(torch.bfloat16)
    q = qs[0].clone()

    def step():
        lens.add_(1)
        gdn.kv4_write(nk, nv, c.cache, c.table, lens)
        return gdn.flash_attn_kv4(q, c.cache, c.table, lens)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    c.cache.fill_(0xff)
    lens.copy_(i32([0, -9]))
    for i in range(total):
        for b, first in ((0, 0), (1, 9)):
            if i >= first:
                nk[b], nv[b] = k[b, :, i - first:i - first + 1], v[b, :, i - first:i - first + 1]
        q.copy_(qs[i])
        g, out = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        c.q, c.lens_l = qs[i], [i + 1, i + 1 - 9]
        assert oracle.parity_error(np64(out), c.want()) <= TOL
    assert gdn.device_status() == gdn.OK


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("lens", [[40, 7], [3000, 900, 0, 2100]])
def test_inputs_made_just_before_and_overwritten_just_after(lens, captured):
    """By kernels, copies and another stream, eagerly and in a graph: one CTA a unit, and joined."""
    c = Case(lens, 8, 2, 2, 128, page=16, seed=7)
    want = c.run()
    busy = torch.randn((3000, 3000), device="cuda")
    cache, q, n = torch.zeros_like(c.cache), torch.zeros_like(c.q), torch.zeros_like(c.lens)
    k, v, out = torch.zeros_like(c.k), torch.zeros_like(c.v), torch.zeros_like(want)
    side = torch.cuda.Stream()

    def step(main):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            busy @ busy
            k.copy_(c.k)
            v.copy_(c.v)
        n.copy_(c.lens)
        main.wait_stream(side)
        gdn.kv4_write(k, v, cache, c.table, n, n)
        for x in (k, v):
            x.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            busy @ busy
            q.copy_(c.q)
        main.wait_stream(side)
        gdn.flash_attn_kv4(q, cache, c.table, n, out=out)
        for x in (q, n, cache):
            x.zero_()

    main = torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        step(main)
        torch.cuda.synchronize()
        run = lambda: step(main)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                step(main)
            run = graph.replay
        for _ in range(5):
            out.fill_(float("nan"))
            run()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
    assert gdn.device_status() == gdn.OK


def test_against_flash_attn_on_the_rows_read_back():
    """The path that it replaces: read back dense in f16 (exact), then dense attention."""
    c = Case([500, 500], 16, 4, 3, 256, dtype="f16", seed=18)
    k, v = gdn.kv4_read(c.cache, c.table, c.lens, 500, 256, lens=c.lens, dtype=torch.float16)
    assert oracle.parity_error(np64(c.run()), np64(gdn.flash_attn(c.q, k, v))) <= 2 * TOL


def test_a_cache_past_4_gib():
    n_pages, Hkv, page, d = 35000, 8, 64, 128
    cache = torch.zeros((n_pages, Hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
    c = Case([130], 16, 8, 1, d, page=page, seed=19)
    c.cache, c.table = cache, i32([[n_pages - 1, 5, n_pages - 3]])
    gdn.kv4_write(c.k, c.v, cache, c.table, c.lens, c.lens)
    c.check()


# ---------------------------------------------------------------- more than 8 rows a kv head, widths up to 128

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_many_rows_over_widths_and_lengths(dtype, dk, dv):
    """12 rows; lengths inside, at and past tiles and steps of 128 tokens, empty and one-token sequences."""
    c = Case([1, 0, 16, 127, 128, 129, 200, 255, 256, 257, 1000, 40], 8, 2, 3, dk, dv, dtype=dtype, seed=dk + 3 * dv)
    got, _ = c.check()
    assert not got[1].any()
    c.check(causal=True)


@pytest.mark.parametrize("page", [16, 48, 256])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_many_rows_with_masks(page, dtype):
    c = Case([300, 17, 140], 8, 2, 5, 64, page=page, dtype=dtype, seed=page, room=1)
    m = c.mask()
    m[0, 0, 1] = -float("inf")
    m[0, 0, 2, :150] = -float("inf")                       # nothing seen in the first step
    m[1, 0, :, 17:] = float("nan")
    got, _ = c.check(mask=m)
    assert not got[0, 1].any()
    c.check(mask=m, causal=True)
    low = torch.zeros_like(m)
    low[0, 0, 0] = low[1, 0, :, ::2] = torch.finfo(DTYPES[dtype]).min
    got, ref = c.run(mask=low), c.want(mask=low)
    if dtype == "f16":                                     # fp32 keeps 2^-7 of scores beside -65504
        ref[0, 0] = np64(got[0, 0])
        assert np.isfinite(ref).all()
    assert oracle.parity_error(np64(got), ref) <= TOL


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.5, 20.0])
def test_many_rows_at_scales(scale):
    """Uniform and very peaked weights: at scale 20 maxima move by hundreds between steps."""
    c = Case([600, 300], 12, 1, 2, 128, dtype="bf16", seed=8)
    c.check(scale=scale, tol=TOL if abs(scale) <= 1 else 1e-2)


def test_many_rows_whose_maxima_keep_rising():
    """Masks that rise by 3 a step of 128 tokens (below the slack) and by 40, and fall: every order of moves."""
    c = Case([1500], 8, 1, 4, 64, dtype="f32", seed=21)
    step = torch.arange(c.cap, device="cuda") // 128
    for slope in (3.0, 40.0, -40.0):
        m = (step * slope).float().expand(1, 1, 4, c.cap).contiguous()
        m = m * torch.tensor([1.0, -1.0, 0.0, 0.5], device="cuda")[None, None, :, None]
        c.check(mask=m.contiguous())
    # the same without a mask: keys that grow along the sequence
    c.k *= torch.exp(step[:1500].float() / 4)[None, None, :, None]
    gdn.kv4_write(c.k, c.v, c.cache, c.table, c.lens, c.lens)
    c.check(tol=1e-3)                                      # (scores near 200: their fp32 units reach 2^-16)


@pytest.mark.parametrize("lens", [[20001], [9000, 1, 5], [1] * 70, [0, 0, 3000, 0] * 12])
def test_many_rows_with_work_shared_unevenly(lens):
    H, Hkv, n_q = (8, 2, 3) if max(lens) > 10000 else (16, 4, 5)
    Case(lens, H, Hkv, n_q, 64 if max(lens) > 10000 else 128, page=64, seed=len(lens)).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_rows_to_16_bits(dtype):
    c = Case([1, 40, 700, 0], 8, 1, 5, 128, 64, dtype=dtype, seed=11)     # 40 rows: two blocks
    got, _ = c.check(out_dtype=DTYPES[dtype])
    assert not got[3].any()


def test_many_rows_with_bad_pages_and_anything_behind_the_end():
    c = Case([140, 300], 8, 1, 2, 64, page=16, seed=14)
    want = c.run()
    c.cache.fill_(0xff)
    gdn.kv4_write(c.k, c.v, c.cache, c.table, c.lens, c.lens)
    assert torch.equal(c.run(), want)
    c.table[0, 1], c.table[1, 2] = c.cache.shape[0], -7
    got = c.run()
    assert gdn.device_status() == gdn.ERR_PAGE and gdn.device_status() == gdn.OK
    m = torch.zeros((2, 1, 2, c.cap), dtype=c.q.dtype, device="cuda")
    m[0, ..., 16:32] = -float("inf")
    m[1, ..., 32:48] = -float("inf")
    assert oracle.parity_error(np64(got), c.want(mask=m)) <= TOL


def test_many_rows_queries_that_are_not_finite_and_streams():
    c = Case([260, 20], 10, 1, 1, 64, dtype="f32", seed=10)
    want = c.run()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [c.run(stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    c.q[0, 3, 0, 5] = float("nan")
    c.q[1, 6, 0, 7] = float("inf")
    got = c.run()
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 0, 3] = True
    bad[1, 0, 6] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])
