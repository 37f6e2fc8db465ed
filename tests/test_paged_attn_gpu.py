"""GPU tests of decode attention over a paged cache of 16- and 32-bit rows against the float64 oracle
(oracle/paged.py).

Metric, as for flash_attn: max |gpu - oracle| / RMS(oracle), bound 1e-4 for fp32 outputs.  16-bit rows enter
exactly, fp32 ones as 22 bits: a score is off by at most 3 * 2^-22 of sum |q k| scale (below 16 for these
inputs), 1.2e-5, and by its fp32 accumulation over at most 256 products, 16 (fp32: 8) at a time, some 16 units of
2^-23 of that sum, 3e-5, if every rounding went one way; a weight is off by as much of itself, and by 2^-18 (bf16: hi and lo
of 8 bits, each to nearest), 2^-22 (f16, fp32) of its rounding.  16-bit outputs may be off by half a step more.
The cache holds NaN wherever no row was written.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
import oracle
from oracle import paged

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


LAYOUTS = ["heads", "tokens", "joint", "pages_inner"]


def caches(layout, n_pages, Hkv, page, dk, dv, dtype):
    """NaN-filled (k_cache, v_cache) in one of several orders of pages, heads and tokens."""
    full = lambda *s: torch.full(s, float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    if layout == "heads":
        return full(n_pages, Hkv, page, dk), full(n_pages, Hkv, page, dv)
    if layout == "tokens":
        return full(n_pages, page, Hkv, dk).transpose(1, 2), full(n_pages, page, Hkv, dv).transpose(1, 2)
    if layout == "pages_inner":       # a head's pages lie together
        return full(Hkv, n_pages, page, dk).transpose(0, 1), full(Hkv, n_pages, page, dv).transpose(0, 1)
    both = full(n_pages, 2, Hkv, page, max(dk, dv))   # keys and values of a page together
    return both[:, 0, :, :, :dk], both[:, 1, :, :, :dv]


class Case:
    """Sequences written into pages of random order."""

    def __init__(self, lens, H, Hkv, n_q, dk, dv=None, page=32, dtype="bf16", seed=0, room=0, layout="heads"):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        dv = dv or dk
        B, n = len(lens), max(max(lens), 1)
        max_pages = -(-n // page) + room
        f = dict(generator=gen, device="cuda")
        self.table = torch.randperm(B * max_pages + 2, **f)[:B * max_pages].to(torch.int32).reshape(B, max_pages)
        self.table = self.table.contiguous()
        self.lens, self.lens_l, self.dv, self.cap = i32(lens), lens, dv, max_pages * page
        self.kc, self.vc = caches(layout, B * max_pages + 2, Hkv, page, dk, dv, DTYPES[dtype])
        slots = torch.cat([self.table[b, torch.arange(m, device="cuda") // page] * page + torch.arange(m, device="cuda") % page
                           for b, m in enumerate(lens)] + [i32([])]).to(torch.int32)
        k = torch.randn((sum(lens), Hkv, dk), **f).to(DTYPES[dtype])
        v = torch.randn((sum(lens), Hkv, dv), **f).to(DTYPES[dtype])
        gdn.paged_write(k, v, self.kc, self.vc, slots)
        self.q = torch.randn((B, H, n_q, dk), **f).to(DTYPES[dtype])
        self.f = f

    def mask(self, std=0.5, hide=0.2):
        B, _, n_q, _ = self.q.shape
        m = torch.randn((B, 1, n_q, self.cap), **self.f) * std
        m[torch.rand(m.shape, **self.f) < hide] = -float("inf")
        return m.to(self.q.dtype)

    def run(self, mask=None, scale=None, **kw):
        return gdn.flash_attn_paged(self.q, self.kc, self.vc, self.table, self.lens, mask, scale, **kw)

    def want(self, mask=None, scale=None, causal=False):
        dk = self.q.shape[3]
        scale = float(np.float32(1 / np.sqrt(dk) if scale is None else scale))
        return paged.attend(np64(self.q), np64(self.kc), np64(self.vc), self.table.cpu().numpy(), self.lens_l, np64(mask), scale,
                            causal)

    def check(self, tol=TOL, out_dtype=None, status=gdn.OK, **kw):
        got = self.run(out_dtype=out_dtype, **kw)
        kw.pop("workspace", None)
        ref = self.want(**kw)
        torch.cuda.synchronize()
        assert gdn.device_status() == status
        y = np64(got)
        assert y.shape == ref.shape and np.isfinite(y).all()
        if got.dtype == torch.float32:
            assert oracle.parity_error(y, ref) <= tol
        else:
            step = torch.finfo(got.dtype).eps / 2
            off = tol * np.sqrt((ref ** 2).mean())
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


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H,Hkv,n_q", [(1, 1, 1), (8, 8, 1), (16, 2, 1), (9, 1, 1), (32, 2, 1), (8, 2, 5), (10, 2, 19),
                                       (3, 3, 2), (24, 1, 3), (40, 1, 19), (17, 1, 1), (33, 1, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_head_groups_and_query_counts(dtype, H, Hkv, n_q, causal):
    """Rows from 1 to 760 a kv head, causal among the newest tokens; queries before the start of a short sequence."""
    c = Case([300, 3, 0, 77], H, Hkv, n_q, 128, dtype=dtype, seed=H + n_q)
    got, ref = c.check(causal=causal)
    if causal and n_q > 3:
        assert not ref[1, :n_q - 3].any() and not got[1, :n_q - 3].any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (256, 256), (64, 256)])
@pytest.mark.parametrize("n_q", [2, 3, 5, 9])
def test_blocks_of_rows_at_other_widths(dtype, dk, dv, n_q):
    c = Case([131, 40], 8, 2, n_q, dk, dv, dtype=dtype, seed=n_q)
    c.check(causal=True)
    c.check(mask=c.mask())


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_orders_of_a_cache(layout, dtype, page):
    """Heads before tokens, tokens before heads, keys and values in one buffer, heads outermost."""
    for dk, dv, Hkv in ((128, 128, 3), (64, 128, 1)):
        Case([130, 17, 200], 6, Hkv, 1, dk, dv, page=page, dtype=dtype, seed=page, layout=layout).check()


@pytest.mark.parametrize("n_q", [1, 4])
def test_queries_of_any_strides(n_q):
    c = Case([130, 17], 8, 2, n_q, 128, seed=2)
    want = c.run()
    token_major = c.q.transpose(1, 2).contiguous().transpose(1, 2)
    joint = torch.zeros((2, n_q, 12, 128), dtype=c.q.dtype, device="cuda")
    joint[:, :, 4:] = c.q.transpose(1, 2)
    for q in (token_major, joint[:, :, 4:].transpose(1, 2)):
        c.q = q
        assert torch.equal(c.run(), want)
    c.q = c.q[:1].expand(2, -1, -1, -1)      # a stride of 0: both sequences ask the same
    c.check()


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
    """A row hidden by the type's lowest value is the softmax of what it says: scores drown in it, weights are equal (in f16
    65504 leaves fp32 scores 2^-8: some 2^-9 of a weight is lost to that rounding alone)."""
    c = Case([50, 33], 4, 2, 2, 128, dtype=dtype, seed=3)
    m = torch.zeros((2, 1, 2, c.cap), device="cuda", dtype=DTYPES[dtype])
    m[0, 0, 0] = torch.finfo(DTYPES[dtype]).min
    m[1, 0, :, ::2] = torch.finfo(DTYPES[dtype]).min
    got, ref = np64(c.run(mask=m)), c.want(mask=m)
    if dtype == "f16":
        assert np.abs(got[0, 0] - ref[0, 0]).max() <= 2.0 ** -8 * np.abs(np64(c.vc)[np.isfinite(np64(c.vc))]).max()
    else:
        used = c.table[0, :2].long()
        v = np64(c.vc[used].transpose(0, 1).reshape(2, -1, 128)[:, :50])
        for h in range(4):
            assert np.abs(got[0, 0, h] - v[h // 2].mean(axis=0)).max() < 1e-5
    got[0, 0] = ref[0, 0]
    assert oracle.parity_error(got, ref) <= TOL


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scale", [1.0, 0.0, -0.5, 20.0])
def test_scales(dtype, scale):
    """Uniform and very peaked weights.  At scale 20 scores reach 1e3: their fp32 units alone move a weight by 1e-4."""
    c = Case([100, 300], 4, 4, 2, 128, dtype=dtype, seed=8)
    c.check(scale=scale, tol=TOL if abs(scale) <= 1 else 1e-2)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n_q,heads", [(1, 4), (1, 8), (3, 8), (5, 8)])
def test_hidden_tokens_may_hold_anything(dtype, n_q, heads):
    """Tokens that only some rows see hold infinities and NaN: those rows take them, the others are as without."""
    c = Case([50, 37, 64], heads, 2 if n_q > 1 else 1, n_q, 128, dtype=dtype, seed=12)
    m = torch.zeros((3, 1, n_q, c.cap), device="cuda", dtype=DTYPES[dtype])
    m[0, 0, :, 5] = m[1, 0, :, 36] = -float("inf")
    m[2, 0, 0, 20] = -float("inf")
    clean, ref = c.check(mask=m)

    def spoil(b, tok, key, value, page=32):
        p = int(c.table[b, tok // page])
        c.kc[p, :, tok % page, 3] = key
        c.vc[p, :, tok % page, 7] = value

    nan, inf = float("nan"), float("inf")
    spoil(0, 5, nan, inf)
    spoil(1, 36, 1.0, nan)
    spoil(2, 20, 1.0, inf)
    got = c.run(mask=m)
    torch.cuda.synchronize()
    assert torch.isfinite(got[:2]).all() and oracle.parity_error(np64(got[:2]), ref[:2]) <= TOL
    assert oracle.parity_error(np64(got[2, 0]), ref[2, 0]) <= TOL       # hidden from this row by its mask
    assert not torch.isfinite(got[2, 1:, :, 7]).any()                   # the rows that see it
    if n_q > 1:
        ok = torch.ones(128, dtype=torch.bool)
        ok[7] = False
        plain = c.want(mask=m)                    # (scores changed with that token's key)
        assert np.abs(np64(got[2, 1:])[..., ok.numpy()] - plain[2, 1:][..., ok.numpy()]).max() <= 1e-3


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_later_drafts_may_hold_anything(dtype):
    """causal: a query does not see the tokens after its own."""
    c = Case([40, 33], 4, 2, 4, 64, dtype=dtype, seed=13)
    _, ref = c.check(causal=True)
    for b, n in enumerate((40, 33)):
        for back, bad in ((1, float("nan")), (2, float("inf"))):
            tok = n - back
            c.vc[int(c.table[b, tok // 32]), :, tok % 32] = bad
    got = c.run(causal=True)
    torch.cuda.synchronize()
    assert oracle.parity_error(np64(got[:, :2]), ref[:, :2]) <= TOL
    assert torch.isinf(got[:, 2]).all() and torch.isnan(got[:, 3]).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_an_infinite_or_nan_query_spoils_its_own_row_only(dtype):
    c = Case([60, 20, 3000], 8, 2, 1, 64, dtype=dtype, seed=10)
    want = c.run()
    c.q[0, 3, 0, 5] = float("nan")
    c.q[1, 6, 0, 7] = float("inf")
    c.q[2, 1, 0, 7] = float("nan")
    got = c.run()
    torch.cuda.synchronize()
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 0, 3] = bad[1, 0, 6] = bad[2, 0, 1] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dv", [64, 128, 256])
def test_16_bit_outputs(dtype, dv):
    c = Case([1, 40, 700, 0], 8, 2, 2, 128, dv, dtype=dtype, seed=11)
    got, _ = c.check(out_dtype=DTYPES[dtype])
    assert got.dtype == DTYPES[dtype] and not got[3].any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n_q", [1, 3, 9])
def test_uneven_batches_and_runs(dtype, n_q):
    """Runs that begin and end inside units, units over many runs, empty sequences between, more sequences than a warp scans."""
    for lens in ([9000, 1, 0, 33, 2000, 0, 16, 500], [70000], [0, 0, 3000, 0], [40 + 17 * (i % 7) for i in range(70)]):
        c = Case(lens, 4, 2, n_q, 64, dtype=dtype, seed=len(lens), page=64)
        c.check(causal=n_q == 3)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (64, 256), (256, 128), (128, 64), (64, 128),
                                   (128, 256), (256, 64)])
@pytest.mark.parametrize("H", [4, 6, 20, 33])
def test_many_laps_of_the_ring(dtype, dk, dv, H):
    """Tiles enough for hundreds of uses of every stage, in runs and in clusters, of 1 to 5 blocks of rows."""
    Case([16000, 5, 9100], H, 1, 1, dk, dv, page=64, dtype=dtype, seed=dk + dv + H).check()
    Case([1900] * 40, H, 1, 1, dk, dv, page=256, dtype=dtype, seed=H).check()


@pytest.mark.parametrize("lens,room", [([7000, 300], 0), ([300, 3, 0], 2000), ([20000], 0)])
def test_one_call_is_the_next(lens, room):
    """Results do not depend on timing: the same bits again, and with a workspace of the caller's."""
    c = Case(lens, 16, 2, 1, 128, seed=4, room=room)
    want = c.run()
    size = gdn.flash_attn_paged_workspace_bytes(len(lens), 16, 2, 1, 128, 128, 32, c.table.shape[1])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(c.run(), want) and torch.equal(c.run(workspace=ws if size else None), want)
    c.check()


def test_bad_pages_and_lengths():
    """Tokens of pages outside the cache, and lengths beyond the table, count as absent."""
    c = Case([100, 64, 90], 8, 2, 1, 64, seed=5)
    c.table[0, 1] = c.kc.shape[0]
    c.table[1, 0] = -1
    c.table[1, 1] = 2 ** 31 - 1
    c.table[2, 2] = -2 ** 31
    got, _ = c.check(status=gdn.ERR_PAGE)
    assert not got[1].any()
    assert gdn.device_status() == gdn.OK
    c = Case([128, 50], 8, 2, 3, 64, seed=6)
    c.lens, c.lens_l = i32([130, 50]), [130, 50]
    c.check(status=gdn.ERR_PAGE, causal=True)
    c.lens, c.lens_l = i32([2 ** 31 - 1, -7]), [2 ** 31 - 1, -7]
    c.check(status=gdn.ERR_PAGE)
    c.lens, c.lens_l = i32([128, -2 ** 31]), [128, -2 ** 31]
    c.check(causal=True)


def test_caches_without_pages_and_tables_without_room():
    q = torch.ones((2, 4, 1, 64), device="cuda", dtype=torch.bfloat16)
    kc, vc = gdn.paged_cache(0, 2, 32, 64)
    for width in (0, 3):
        out = torch.full((2, 1, 4, 64), 7.0, device="cuda")
        gdn.flash_attn_paged(q, kc, vc, i32([[0] * width] * 2), i32([5, 0]), out=out)
        torch.cuda.synchronize()
        assert not out.any() and gdn.device_status() == gdn.ERR_PAGE


def test_pages_shared_by_sequences():
    c = Case([96, 96], 8, 2, 1, 128, seed=7)
    c.table[1, :2] = c.table[0, :2]
    c.check()


def test_two_streams_at_once():
    c, d = Case([5000, 3000], 16, 4, 1, 128, seed=20), Case([6000, 10], 16, 4, 2, 128, seed=21)
    want = c.run(), d.run()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [x.run(stream=y) for x, y in zip((c, d), s)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """Pages more than 2^32 bytes into the cache."""
    n_pages, Hkv, page, d = 5000 if dtype == "f32" else 9000, 8, 256, 128
    kc, vc = gdn.paged_cache(n_pages, Hkv, page, d, dtype=DTYPES[dtype])
    assert kc.numel() * kc.element_size() > 2 ** 32
    table = i32([[n_pages - 1, 0, n_pages - 2], [3, n_pages - 3, 1]])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for p in table.flatten().tolist():
        for x in (kc, vc):
            x[p] = torch.randn(x[p].shape, generator=gen, device="cuda").to(x.dtype)
    q = torch.randn((2, 16, 1, d), generator=gen, device="cuda").to(DTYPES[dtype])
    got = gdn.flash_attn_paged(q, kc, vc, table, i32([600, 700]))
    used = table.flatten().long()
    ref = paged.attend(np64(q), np64(kc[used]), np64(vc[used]), np.arange(6).reshape(2, 3), [600, 700])
    assert oracle.parity_error(np64(got), ref) <= TOL


@pytest.mark.parametrize("room", [0, 300])
def test_thousands_of_sequences(room):
    """Sums over more sequences than a CTA has threads, in runs (room) and in CTAs a unit."""
    lens = [(37 * b) % 90 if b % 5 else 0 for b in range(1500)] + [900, 0, 3]
    Case(lens, 4, 2, 2, 64, page=16, seed=31, room=room).check(causal=True)


def test_masks_past_32_bits():
    """Mask rows more than 2^31 elements into the mask of long tables."""
    B, room, page, d = 65, 1 << 21, 16, 64
    c = Case([40] * B, 4, 1, 1, d, page=page, seed=32)
    table = torch.full((B, room), -1, dtype=torch.int32, device="cuda")
    table[:, :3] = c.table
    mask = torch.zeros((B, 1, 1, room * page), dtype=torch.bfloat16, device="cuda")
    assert mask.numel() > 2 ** 31
    mask[:, :, :, :48] = c.mask()
    ref = paged.attend(np64(c.q), np64(c.kc), np64(c.vc), c.table.cpu().numpy(), c.lens_l, np64(mask[:, :, :, :48]))
    got = gdn.flash_attn_paged(c.q, c.kc, c.vc, table, c.lens, mask)
    torch.cuda.synchronize()
    assert gdn.device_status() == gdn.OK and oracle.parity_error(np64(got), ref) <= TOL


def test_captured_calls_follow_the_lengths():
    """Two graphs with the library's own workspace, replayed in turn (and both at once) while lengths grow."""
    c = Case([4000, 3000, 100, 2500], 16, 4, 1, 128, seed=33, room=200)
    lens = c.lens.clone()
    graphs = []
    for _ in range(2):
        c.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c.run()
        graphs.append((g, out))
    for step, now in enumerate(([1, 2, 3, 4], [0, 3000, 0, 1], [4000, 17, 100, 2500], [0, 0, 0, 0], [100, 2999, 64, 16])):
        c.lens.copy_(i32(now))
        want = c.run()
        g, out = graphs[step % 2]
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    c.lens.copy_(lens)
    want = c.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out in graphs)
    c.check()
