"""GPU tests of the 4-bit cache: writing it and reading it back.

The format defines every kept value exactly (oracle/kv4.py), and each is exact
in fp32, bf16 and f16, so all comparisons are for equality.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
from oracle import kv4

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_attention_sequence_gated_gb300 import _build
    _build.build()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A cache of random bytes (so that what must not be written shows), with pages in random order."""

    def __init__(self, B, Hkv, max_pages, page, dk, dv, seed=0, spare=2):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        n = B * max_pages + spare
        self.data = torch.randint(0, 256, (n, Hkv, page // 16, 9 * (dk + dv)), generator=gen, device="cuda",
                                  dtype=torch.uint8)
        self.table = torch.randperm(n, generator=gen, device="cuda")[:B * max_pages].to(torch.int32)
        self.table = self.table.reshape(B, max_pages).contiguous()
        self.gen, self.Hkv, self.dk, self.dv, self.page = gen, Hkv, dk, dv, page

    def rows(self, B, T, dtype):
        """Rows over many magnitudes, with zeros and exact multiples among them."""
        out = []
        for d in (self.dk, self.dv):
            x = torch.randn((B, self.Hkv, T, d), generator=self.gen, device="cuda")
            x *= torch.exp(2 * torch.randn((B, self.Hkv, T, 1), generator=self.gen, device="cuda"))
            x[torch.rand(x.shape, generator=self.gen, device="cuda") < 0.05] = 0
            tie = torch.rand(x.shape[:3], generator=self.gen, device="cuda") < 0.3
            x[tie] = torch.round(x[tie] * 4) / 4           # borders between codes, where the scale is a power of two
            out.append(x.to(DTYPES[dtype]))
        return out

    def read(self, lens, n, counts=None, dtype="f32"):
        return gdn.kv4_read(self.data, self.table, lens, n, self.dk, self.dv, lens=counts, dtype=DTYPES[dtype])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (64, 256), (256, 128), (128, 64)])
@pytest.mark.parametrize("page", [16, 48])
def test_write_then_read(dtype, dk, dv, page):
    """Ragged lengths and counts: what is read is what the format keeps, zeros elsewhere."""
    B, Hkv, T = 5, 3, 37
    lens, new = [37, 50, 1, 0, 96], [37, 20, 1, 0, 31]
    c = Cache(B, Hkv, 96 // page, page, dk, dv, seed=dk + dv + page)
    k, v = c.rows(B, T, dtype)
    gdn.kv4_write(k, v, c.data, c.table, i32(lens), i32(new))
    got = c.read(i32(lens), T, i32(new), dtype)
    torch.cuda.synchronize()
    assert gdn.device_status() == gdn.OK
    for x, y in zip((k, v), got):
        assert y.dtype == DTYPES[dtype]
        want = kv4.kept(np64(x))
        for b, n in enumerate(new):
            want[b, :, n:] = 0
        assert np.array_equal(np64(y), want)


@pytest.mark.parametrize("dk,dv", [(64, 128), (256, 64)])
def test_bytes_are_the_described_layout(dk, dv):
    c = Cache(1, 2, 1, 32, dk, dv, seed=3)
    k, v = c.rows(1, 32, "f32")
    gdn.kv4_write(k, v, c.data, c.table, i32([32]))
    tiles = c.data[c.table[0, 0].item()].cpu().numpy()
    for h in range(2):
        for t in range(2):
            tk, tv = kv4.unpack_tile(tiles[h, t], dk, dv)
            assert np.array_equal(tk, kv4.kept(np64(k[0, h, 16 * t:16 * t + 16])))
            assert np.array_equal(tv, kv4.kept(np64(v[0, h, 16 * t:16 * t + 16])))


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 256)])
def test_token_by_token_equals_one_run_and_nothing_else_changes(dk, dv):
    """Appending one at a time, in runs of odd lengths, or at once leaves the same bytes; other tiles and the
    tokens behind the end keep theirs."""
    B, Hkv, n, page = 2, 2, 41, 16
    first = Cache(B, Hkv, 4, page, dk, dv, seed=11)
    k, v = first.rows(B, n, "bf16")
    before, results = first.data.clone(), []
    for step in (1, 3, 16, n):
        c = Cache(B, Hkv, 4, page, dk, dv, seed=11)
        for at in range(0, n, step):
            end = min(n, at + step)
            gdn.kv4_write(k[:, :, at:end], v[:, :, at:end], c.data, c.table, i32([end, end]))
        results.append(c)
    want = results[0].data
    for c in results[1:]:
        assert torch.equal(c.data, want)
    touched = torch.zeros(want.shape[0], dtype=torch.bool, device="cuda")
    touched[first.table[:, :3].long().reshape(-1)] = True            # 41 tokens lie in three pages of 16
    assert torch.equal(want[~touched], before[~touched])
    # tokens 41 .. 47 of the last page, read as if the sequences had 48: as before the writes
    for x, y in zip(first.read(i32([48, 48]), 7), results[0].read(i32([48, 48]), 7)):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
    got = results[0].read(i32([n, n]), n)
    assert np.array_equal(np64(got[0]), kv4.kept(np64(k))) and np.array_equal(np64(got[1]), kv4.kept(np64(v)))


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_tokens_behind_the_run_keep_their_bytes(dk, dv):
    """A run that begins and ends inside tiles, written over older tokens: the older ones around it stay."""
    c = Cache(1, 2, 4, 16, dk, dv, seed=12)
    k, v = c.rows(1, 64, "bf16")
    gdn.kv4_write(k, v, c.data, c.table, i32([64]))
    k2, v2 = c.rows(1, 21, "bf16")
    gdn.kv4_write(k2, v2, c.data, c.table, i32([34]))                # positions 13 .. 33
    got = c.read(i32([64]), 64)
    for x, x2, y in ((k, k2, got[0]), (v, v2, got[1])):
        want = np64(x)
        want[:, :, 13:34] = np64(x2)
        assert np.array_equal(np64(y), kv4.kept(want))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_special_values(dtype):
    """NaN as 0, infinities and large values at 61440, tiny rows, signed zeros, borders between codes."""
    d, dt = 128, DTYPES[dtype]
    c = Cache(1, 1, 1, 16, d, d, seed=13)
    x = torch.zeros((1, 1, 16, d), device="cuda")
    x[..., 0, :] = float("nan")
    x[..., 1, 5], x[..., 1, 6], x[..., 1, 7] = float("nan"), 3.0, -1.0
    x[..., 2, 5], x[..., 2, 6] = float("inf"), 7.0
    x[..., 3, 5], x[..., 3, 6] = -float("inf"), float("nan")
    x[..., 4, :] = 60000.0
    x[..., 5, :] = -2.0 ** -18
    x[..., 6, :] = 2.0 ** -14
    x[..., 7, :] = -0.0
    x[..., 8, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5,
                                   -5.0, -6.0], device="cuda")
    x[..., 9, :16] = x[..., 8, :16] * 1.875
    x[..., 10, :16] = x[..., 8, :16] * 1.625
    x[..., 11, :16] = x[..., 8, :16] * 1.75
    if dtype != "f16":
        x[..., 12, :16] = x[..., 8, :16] * 2.0 ** 20
        x[..., 13, :16] = x[..., 8, :16] * 2.0 ** -30
    x = x.to(dt)
    gdn.kv4_write(x, x, c.data, c.table, i32([16]))
    got = c.read(i32([16]), 16, dtype=dtype)
    want = kv4.kept(np64(x))
    assert np.isfinite(want).all()
    for y in got:
        assert np.array_equal(np64(y), want)


def test_f32_inputs_beside_the_borders():
    """fp32 values one unit to either side of each border between codes, under every significand of the scale."""
    c = Cache(1, 1, 2, 16, 128, 128, seed=14)
    rows = []
    for sig in range(8, 16):
        s = np.float32(sig / 8)
        for m in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            b = np.float32(m * s)
            rows.append([np.nextafter(b, np.float32(0)), b, np.nextafter(b, np.float32(9)), -b, 6 * s] + [0] * 11)
    x = torch.zeros(32 * 8, 16)
    x[:len(rows)] = torch.tensor(np.array(rows, dtype=np.float32))
    x = x.reshape(1, 1, 32, 128).cuda()
    gdn.kv4_write(x, x, c.data, c.table, i32([32]))
    for y in c.read(i32([32]), 32):
        assert np.array_equal(np64(y), kv4.kept(np64(x)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows(dtype):
    """Token-major projections, a slice of a fused one (rows 16- but not 32-byte aligned), one row for all heads."""
    B, T, Hkv, d = 2, 19, 2, 128
    c = Cache(B, Hkv, 2, 32, d, d, seed=15)
    pad = 8 if dtype == "bf16" else 4
    fused = torch.randn((B, T, 2 * Hkv * d + 3 * pad), device="cuda").to(DTYPES[dtype])
    k = fused[..., pad:pad + Hkv * d].unflatten(2, (Hkv, d)).transpose(1, 2)
    v = fused[..., 2 * pad + Hkv * d:2 * pad + 2 * Hkv * d].unflatten(2, (Hkv, d)).transpose(1, 2)
    gdn.kv4_write(k, v, c.data, c.table, i32([T, T + 5]))
    got = c.read(i32([T, T + 5]), T)
    assert np.array_equal(np64(got[0]), kv4.kept(np64(k))) and np.array_equal(np64(got[1]), kv4.kept(np64(v)))
    one = torch.randn((B, 1, T, d), device="cuda").to(DTYPES[dtype]).expand(B, Hkv, T, d)
    gdn.kv4_write(one, k, c.data, c.table, i32([T, T]))
    got = c.read(i32([T, T]), T)
    assert np.array_equal(np64(got[0]), kv4.kept(np64(one))) and np.array_equal(np64(got[1]), kv4.kept(np64(k)))
    with pytest.raises(gdn.GdnError) as e:                           # rows off 16 bytes
        gdn.kv4_write(fused[..., 1:1 + Hkv * d].unflatten(2, (Hkv, d)).transpose(1, 2), v, c.data, c.table,
                      i32([T, T]))
    assert e.value.status == gdn.ERR_ALIGN


def test_read_into_an_output_off_32_bytes_and_zero_rows():
    c = Cache(2, 1, 2, 16, 64, 128, seed=16)
    k, v = c.rows(2, 20, "bf16")
    gdn.kv4_write(k, v, c.data, c.table, i32([20, 20]))
    hold = torch.full((2 * 25 * 64 + 2 * 25 * 128 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = hold[8:8 + 2 * 25 * 64].view(2, 1, 25, 64)
    vo = hold[8 + 2 * 25 * 64:8 + 2 * 25 * 192].view(2, 1, 25, 128)
    gdn.kv4_read(c.data, c.table, i32([20, 4]), 25, 64, 128, k_out=ko, v_out=vo)   # starts before position 0
    for x, y in ((k, ko), (v, vo)):
        want = np.zeros(y.shape)
        want[0, :, 5:] = kv4.kept(np64(x))[0]
        want[1, :, 21:] = kv4.kept(np64(x))[1, :, :4]
        assert np.array_equal(np64(y), want)
    assert (hold[:8] == 7).all() and (hold[-8:] == 7).all()


def test_bad_pages_and_lengths_are_reported_and_touch_nothing():
    c = Cache(3, 2, 2, 16, 64, 64, seed=17)
    n_pages = c.data.shape[0]
    k, v = c.rows(3, 32, "f32")
    table = c.table.clone()
    table[0, 1], table[1, 0] = n_pages, -1
    before = c.data.clone()
    assert gdn.device_status() == gdn.OK
    gdn.kv4_write(k, v, c.data, table, i32([32, 32, 32]))
    assert gdn.device_status() == gdn.ERR_PAGE and gdn.device_status() == gdn.OK
    good = torch.tensor([c.table[0, 0], c.table[1, 1], c.table[2, 0], c.table[2, 1]]).long()
    rest = torch.ones(n_pages, dtype=torch.bool)
    rest[good] = False
    assert torch.equal(c.data[rest.cuda()], before[rest.cuda()])
    got = gdn.kv4_read(c.data, table, i32([32, 32, 32]), 32, 64, dtype=torch.float32)
    assert gdn.device_status() == gdn.ERR_PAGE
    for x, y in zip((k, v), got):
        want = kv4.kept(np64(x))
        want[0, :, 16:] = 0
        want[1, :, :16] = 0
        assert np.array_equal(np64(y), want)
    # a length past the table: the part that the table reaches is written and read
    for length in (40, 2 ** 31 - 1):
        c = Cache(1, 2, 2, 16, 64, 64, seed=18)
        before = c.data.clone()
        gdn.kv4_write(k[:1], v[:1], c.data, c.table, i32([length]))
        assert gdn.device_status() == gdn.ERR_PAGE
        got = c.read(i32([length]), 32)
        assert gdn.device_status() == gdn.ERR_PAGE
        want = kv4.kept(np64(k[:1]))
        if length == 40:                                             # positions 8 .. 31 of 8 .. 39
            want[:, :, 24:] = 0
        else:
            want[:] = 0
            assert torch.equal(c.data, before)
        assert np.array_equal(np64(got[0]), want)
    # negative counts and lengths: nothing there
    before = c.data.clone()
    gdn.kv4_write(k[:1], v[:1], c.data, c.table, i32([-5]))
    gdn.kv4_write(k[:1], v[:1], c.data, c.table, i32([16]), i32([-1]))
    assert torch.equal(c.data, before) and gdn.device_status() == gdn.OK
    assert not c.read(i32([-5]), 8)[0].any()


def test_captured_steps_follow_the_lengths_in_memory():
    """A captured append and read-back, replayed with the lengths moved on the device."""
    B, Hkv, d = 2, 2, 128
    c = Cache(B, Hkv, 3, 16, d, d, seed=19)
    steps = [c.rows(B, 1, "bf16") for _ in range(40)]
    k, v = steps[0][0].clone(), steps[0][1].clone()
    lens = i32([0, 3])
    start = c.data.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        gdn.kv4_write(k, v, c.data, c.table, lens)
        back = c.read(lens, 1)
    c.data.copy_(start)
    lens.copy_(i32([0, 3]))
    for sk, sv in steps:
        k.copy_(sk)
        v.copy_(sv)
        graph.replay()
        assert np.array_equal(np64(back[0]), kv4.kept(np64(sk)))
    got = c.read(i32([40, 43]), 40)
    for i, y in enumerate(got):
        want = kv4.kept(np64(torch.cat([s[i] for s in steps], dim=2)))
        assert np.array_equal(np64(y), want)


def test_given_stream():
    c = Cache(1, 1, 2, 16, 64, 64, seed=20)
    k, v = c.rows(1, 20, "f16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lens = i32([20])
    s.wait_stream(torch.cuda.current_stream())
    gdn.kv4_write(k, v, c.data, c.table, lens, stream=s)
    got = gdn.kv4_read(c.data, c.table, lens, 20, 64, stream=s, dtype=torch.float32)
    s.synchronize()
    assert np.array_equal(np64(got[0]), kv4.kept(np64(k)))


def test_a_long_cache_past_32_bits():
    """Pages whose bytes lie beyond 4 GiB."""
    d, Hkv, page = 128, 8, 64
    n = (5 << 30) // (Hkv * page * 9 * 2 * d // 16)
    data = torch.empty((n, Hkv, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[n - 1, n - 7, 3]], dtype=torch.int32, device="cuda")
    k = torch.randn((1, Hkv, 150, d), device="cuda")
    v = torch.randn((1, Hkv, 150, d), device="cuda")
    gdn.kv4_write(k, v, data, table, i32([150]))
    got = gdn.kv4_read(data, table, i32([150]), 150, d, dtype=torch.float32)
    assert np.array_equal(np64(got[0]), kv4.kept(np64(k))) and np.array_equal(np64(got[1]), kv4.kept(np64(v)))
