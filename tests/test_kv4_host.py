"""The 4-bit cache without a GPU: its oracle's pins, the index and rounding
arithmetic compiled for the host, and the refusals of its entry points.

Calls that pass (made-up) device addresses are ones that the library must
refuse during host validation; none reaches a launch.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import linear_attention_sequence_gated_gb300 as gdn
from linear_attention_sequence_gated_gb300 import _build
from oracle import kv4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE, MB = 1 << 40, 1 << 20
ptr = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731


@pytest.fixture(scope="module")
def L():
    _build.build()
    return gdn.lib()


@pytest.fixture(scope="module")
def H(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("kv4") / "kv4_host.so")
    subprocess.check_call([_build.nvcc()] + _build.ARCH + ["-std=c++17", "-shared", "-Xcompiler", "-fPIC",
                                                          "-o", so, os.path.join(ROOT, "tests", "kv4_host.cu")])
    lib = ctypes.CDLL(so)
    lib.kv4_tile_offset.restype = ctypes.c_longlong
    return lib


# ------------------------------------------------------------ the oracle

def test_oracle_keeps_what_the_format_can_hold():
    """Rows that are codes times a scale, with the largest code among them, come back as they are."""
    rng = np.random.default_rng(0)
    for s in (kv4.SCALES[1], kv4.SCALES[9], kv4.SCALES[100], kv4.SCALES[-1]):
        x = kv4.LEVELS[rng.integers(0, 8, (50, 16))] * rng.choice([-1, 1], (50, 16)) * s
        x[:, 3] = 6 * s
        assert np.array_equal(kv4.kept(x), x)


def test_oracle_is_the_nearest_value():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((200, 16)) * np.exp(rng.standard_normal((200, 1)))
    y = kv4.kept(x)
    for row, got in zip(x, y):
        s = min(kv4.SCALES, key=lambda c: abs(c - np.abs(row).max() / 6))
        grid = np.concatenate([kv4.LEVELS, -kv4.LEVELS]) * s
        assert np.allclose(np.abs(got - row), np.abs(grid[None] - row[:, None]).min(axis=1), atol=1e-12)


def test_oracle_edges():
    x = np.zeros(16)
    assert not kv4.kept(x).any()
    x[0] = np.inf
    assert kv4.kept(x)[0] == 61440 and not kv4.kept(x)[1:].any()
    x[0], x[1] = np.nan, 3.0
    assert kv4.kept(x)[0] == 0 and kv4.kept(x)[1] == 3.0
    x[:] = 2.0 ** -17 * 2.9          # under half the least scale: nothing is kept
    assert not kv4.kept(x).any()


# ------------------------------------------------------------ index and rounding arithmetic

def test_scale_bytes_round_as_the_oracle(H):
    """Around every border between two scales, over all f16 and bf16 values, and at random."""
    rng = np.random.default_rng(2)
    border = (6 * (kv4.SCALES[1:] + kv4.SCALES[:-1]) / 2).astype(np.float32)
    near = (border.view(np.int32)[:, None] + np.arange(-30, 31)).astype(np.int32).view(np.float32).ravel()
    x16 = np.concatenate([np.arange(0x7c01, dtype=np.uint16).view(np.float16).astype(np.float32),
                          (np.arange(0x7f81, dtype=np.uint32) << 16).view(np.float32)])
    x32 = np.concatenate([near[near >= 0], x16, np.exp(rng.uniform(-14, 12, 100000)).astype(np.float32)])
    for wide, a in ((0, x16), (1, x32)):
        out = np.zeros(a.size, dtype=np.int32)
        H.kv4_scale_bytes(ctypes.c_void_p(a.ctypes.data), a.size, wide, ctypes.c_void_p(out.ctypes.data))
        want = kv4.nearest(np.minimum(a.astype(np.float64), 61440) / 6, kv4.SCALES)
        assert np.array_equal(out, want)


def fall(y, m, s):
    """On which side of the borders m (times s) the values y (or rows y * s) fall, as -1, 0, 1."""
    return np.sign(y[:, None].astype(np.float64) - np.asarray(m, dtype=np.float64) * s)


def test_quotients_fall_where_the_values_do(H):
    """Every f16 and bf16 value under every scale, and fp32 values around each border: the quotient is on the side of
    each border between codes where the value is of the border times the scale, and on it where it is."""
    borders = (kv4.LEVELS[1:] + kv4.LEVELS[:-1]) / 2
    x16 = np.concatenate([np.arange(1, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float32),
                          (np.arange(1, 0x7f80, dtype=np.uint32) << 16).view(np.float32)])
    for byte, s in enumerate(kv4.SCALES):
        if byte == 0:
            continue
        near = (borders * s).astype(np.float32)
        x32 = (near.view(np.int32)[:, None] + np.arange(-40, 41)).astype(np.int32).view(np.float32).ravel()
        for wide, x in ((0, x16[x16 < 7 * s]), (1, x32)):
            x = np.ascontiguousarray(x)
            y = np.zeros_like(x)
            H.kv4_ratios(ctypes.c_void_p(x.ctypes.data), x.size, byte, wide, ctypes.c_void_p(y.ctypes.data))
            assert np.array_equal(fall(y, borders, 1), fall(x, borders, s))


def test_pages_outside_the_cache_have_no_offset(H):
    assert H.kv4_tile_offset(0, 5, 3, 2, 4, 1, 2304) == (2 * 4 + 1) * 2304
    assert H.kv4_tile_offset(4, 5, 3, 2, 4, 3, 2304) == ((4 * 3 + 2) * 4 + 3) * 2304
    for page in (5, -1, 2 ** 31 - 1, -2 ** 31):
        assert H.kv4_tile_offset(page, 5, 3, 2, 4, 1, 2304) == -1
    assert H.kv4_tile_offset(0, 0, 3, 2, 4, 1, 2304) == -1
    # a long cache: the offset passes 32 bits
    assert H.kv4_tile_offset(10 ** 6, 10 ** 6 + 1, 8, 7, 4, 3, 2304) == ((10 ** 6 * 8 + 7) * 4 + 3) * 2304


@pytest.mark.parametrize("raw,cap,count", [(0, 64, 1), (1, 64, 1), (16, 64, 1), (17, 64, 5), (64, 64, 64),
                                           (3, 64, 7), (0, 64, 33), (70, 64, 10), (200, 64, 3), (50, 0, 20),
                                           (2 ** 31 - 1, 2 ** 31 - 65, 100), (40, 64, 0)])
def test_places_of_a_calls_tokens(H, raw, cap, count):
    """The tiles of a call together hold each of its tokens once, at its position, and no other."""
    seen = {}
    out = (ctypes.c_int * 19)()
    for j in range((max(count, 1) + 30) // 16):
        H.kv4_place(raw, cap, count, j, out)
        for i in range(16):
            if out[3 + i]:
                assert out[2]
                seen[out[1] + i] = out[0] * 16 + i
    want = {t: raw - count + t for t in range(count) if 0 <= raw - count + t < min(raw, cap)}
    assert seen == want


@pytest.mark.parametrize("units,most", [([1], 2432), ([9, 9, 9, 9], 2432), ([1, 0, 5000, 3, 0, 17, 1], 16),
                                        ([256] * 40, 97), ([6251, 0, 1], 2432), ([1] * 3000, 1216)])
def test_runs_share_out_every_tile_and_their_parts_join(H, units, most):
    """Every run is non-empty; together they cover each tile once; a unit's parts are found again by the runs of its
    first and last tile, no two parts share a slot, and a whole unit leaves none."""
    T = sum(units)
    W = min(T, most)
    begin = np.cumsum([0] + units)
    slots, parts = set(), {u: [] for u in range(len(units))}
    for w in range(W):
        at, stop = H.kv4_run_begin(T, W, w), H.kv4_run_begin(T, W, w + 1)
        assert at < stop and (w > 0 or at == 0) and (w < W - 1 or stop == T)
        while at < stop:
            u = int(np.searchsorted(begin, at, "right") - 1)
            end = min(stop, begin[u + 1])
            if not (at == begin[u] and end == begin[u + 1]):
                slot = H.kv4_partial_slot(w, int(at == begin[u]))
                assert slot not in slots and 0 <= slot < 2 * W
                slots.add(slot)
                parts[u].append((slot, end - at))
            at = end
    for u, n in enumerate(units):
        if n == 0:
            continue
        w0, w1 = H.kv4_run_of(T, W, int(begin[u])), H.kv4_run_of(T, W, int(begin[u + 1] - 1))
        if w0 == w1:
            assert not parts[u]
        else:
            assert [p[0] for p in parts[u]] == [H.kv4_partial_slot(w, int(w == w0)) for w in range(w0, w1 + 1)]
            assert sum(p[1] for p in parts[u]) == n


def test_runs_of_a_very_long_batch(H):
    T, W = 2 ** 31 - 1, 1824
    for w in (0, 1, 1000, W - 1):
        at = H.kv4_run_begin(T, W, w)
        assert at == T // W * w + min(w, T % W) and H.kv4_run_of(T, W, at) == w
        assert H.kv4_run_of(T, W, H.kv4_run_begin(T, W, w + 1) - 1) == w


# ------------------------------------------------------------ refusals

def test_supports_and_sizes(L):
    for dk in (64, 128, 256):
        for dv in (64, 128, 256):
            assert gdn.kv4_supports(dk, dv)
            assert L.gdn_kv4_cache_bytes(3, 2, 32, dk, dv) == 3 * 2 * 2 * 9 * (dk + dv)
    for d in (0, 16, 32, 96, 512, -64):
        assert not gdn.kv4_supports(d, 128) and not gdn.kv4_supports(128, d)
    for bad in ((-1, 2, 32, 64, 64), (3, -2, 32, 64, 64), (3, 2, 0, 64, 64), (3, 2, 24, 64, 64),
                (3, 2, 32, 96, 64), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 30, 256, 256)):
        assert L.gdn_kv4_cache_bytes(*bad) == 0
    assert gdn.status_string(gdn.ERR_PAGE) != "unknown status"
    with pytest.raises(gdn.GdnError):
        gdn.kv4_cache(4, 2, 24, 128, device="cpu")
    with pytest.raises(gdn.GdnError):
        gdn.kv4_cache(4, 2, 32, 96, device="cpu")
    assert tuple(gdn.kv4_cache(4, 2, 32, 64, 128, device="cpu").shape) == (4, 2, 2, 9 * 192)


COMMON = [
    (dict(B=-1), gdn.ERR_ARG), (dict(Hkv=-1), gdn.ERR_ARG), (dict(T=-1), gdn.ERR_ARG),
    (dict(n_pages=-1), gdn.ERR_ARG), (dict(max_pages=-1), gdn.ERR_ARG), (dict(dtype=3), gdn.ERR_ARG),
    (dict(dk=96), gdn.ERR_HEADDIM), (dict(dv=32), gdn.ERR_HEADDIM),
    (dict(page=24), gdn.ERR_SHAPE), (dict(page=0), gdn.ERR_SHAPE), (dict(page=-16), gdn.ERR_SHAPE),
    (dict(max_pages=1 << 27, page=16), gdn.ERR_ARG),                 # positions past 32 bits
    (dict(n_pages=2 ** 31 - 1, Hkv=2 ** 31 - 1, page=1 << 20, max_pages=1), gdn.ERR_ARG),
    (dict(cache=None), gdn.ERR_ARG), (dict(table=None), gdn.ERR_ARG), (dict(lens=None), gdn.ERR_ARG),
    (dict(k=None), gdn.ERR_ARG), (dict(v=None), gdn.ERR_ARG),
    (dict(k=BASE + 8), gdn.ERR_ALIGN), (dict(v=BASE + 64 * MB + 4), gdn.ERR_ALIGN),
    (dict(cache=BASE + 128 * MB + 8), gdn.ERR_ALIGN), (dict(table=BASE + 256 * MB + 2), gdn.ERR_ALIGN),
    (dict(lens=BASE + 260 * MB + 1), gdn.ERR_ALIGN), (dict(counts=BASE + 264 * MB + 2), gdn.ERR_ALIGN),
    (dict(k=BASE + 128 * MB), gdn.ERR_ALIAS), (dict(v=BASE + 128 * MB + 4096), gdn.ERR_ALIAS),
    (dict(B=1 << 30, T=1 << 30, Hkv=1 << 20), gdn.ERR_ARG),
]


def args(kw):
    a = dict(k=BASE, v=BASE + 64 * MB, cache=BASE + 128 * MB, table=BASE + 256 * MB, lens=BASE + 260 * MB,
             counts=None, strides=None, B=2, T=4, Hkv=2, dk=128, dv=128, n_pages=8, page=64, max_pages=4,
             dtype=1)
    a.update(kw)
    return a


def write(L, **kw):
    a = args(kw)
    st = None if a["strides"] is None else (ctypes.c_longlong * 6)(*a["strides"])
    return L.gdn_kv4_write(ptr(a["k"]), ptr(a["v"]), st, ptr(a["cache"]), ptr(a["table"]), ptr(a["lens"]),
                           ptr(a["counts"]), a["B"], a["T"], a["Hkv"], a["dk"], a["dv"], a["n_pages"],
                           a["page"], a["max_pages"], a["dtype"], None)


def read(L, **kw):
    a = args(kw)
    return L.gdn_kv4_read(ptr(a["cache"]), ptr(a["table"]), ptr(a["lens"]), ptr(a["counts"]), ptr(a["k"]),
                          ptr(a["v"]), a["B"], a["T"], a["Hkv"], a["dk"], a["dv"], a["n_pages"], a["page"],
                          a["max_pages"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", COMMON)
def test_write_and_read_refuse(L, kw, code):
    assert write(L, **kw) == code
    assert read(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(strides=(-1, 0, 128, 0, 0, 128)), gdn.ERR_ARG),
    (dict(strides=(1 << 62, 0, 128, 0, 0, 128)), gdn.ERR_ARG),
    (dict(strides=(1024, 512, 132, 1024, 512, 128)), gdn.ERR_ALIGN),
    (dict(table=BASE + 128 * MB + 64), gdn.ERR_ALIAS), (dict(lens=BASE + 128 * MB + 64), gdn.ERR_ALIAS),
    (dict(counts=BASE + 128 * MB + 64), gdn.ERR_ALIAS),
])
def test_write_refuses(L, kw, code):
    assert write(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(v=BASE + 1024), gdn.ERR_ALIAS), (dict(table=BASE + 64), gdn.ERR_ALIAS),
    (dict(lens=BASE + 64 * MB + 64), gdn.ERR_ALIAS), (dict(counts=BASE + 64), gdn.ERR_ALIAS),
])
def test_read_refuses(L, kw, code):
    assert read(L, **kw) == code


def test_empty_calls_do_nothing(L):
    none = dict(k=None, v=None, cache=None, table=None, lens=None)
    for f in (write, read):
        assert f(L, B=0, **none) == gdn.OK
        assert f(L, Hkv=0, **none) == gdn.OK
        assert f(L, T=0, k=None, v=None) == gdn.OK


def attend(L, **kw):
    a = dict(q=BASE, cache=BASE + 128 * MB, table=BASE + 256 * MB, lens=BASE + 260 * MB, mask=None,
             out=BASE + 264 * MB, B=2, H=8, Hkv=2, n_q=1, dk=128, dv=128, n_pages=8, page=64, max_pages=4,
             scale=0.1, causal=0, dtype=1, out_dtype=0, ws=None, ws_bytes=0)
    a.update(kw)
    return L.gdn_flash_attn_kv4(ptr(a["q"]), ptr(a["cache"]), ptr(a["table"]), ptr(a["lens"]), ptr(a["mask"]),
                                ptr(a["out"]), a["B"], a["H"], a["Hkv"], a["n_q"], a["dk"], a["dv"],
                                a["n_pages"], a["page"], a["max_pages"], ctypes.c_float(a["scale"]),
                                a["causal"], a["dtype"], a["out_dtype"], ptr(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), gdn.ERR_ARG), (dict(H=-1), gdn.ERR_ARG), (dict(n_q=-1), gdn.ERR_ARG), (dict(Hkv=3), gdn.ERR_ARG),
    (dict(Hkv=0), gdn.ERR_ARG), (dict(n_q=20), gdn.ERR_SHAPE), (dict(dk=96), gdn.ERR_HEADDIM),
    (dict(dv=512), gdn.ERR_HEADDIM), (dict(page=8), gdn.ERR_SHAPE), (dict(max_pages=1 << 26), gdn.ERR_ARG),
    (dict(scale=float("nan")), gdn.ERR_ARG), (dict(scale=float("inf")), gdn.ERR_ARG),
    (dict(causal=2), gdn.ERR_ARG), (dict(dtype=3), gdn.ERR_ARG), (dict(out_dtype=3), gdn.ERR_ARG),
    (dict(q=None), gdn.ERR_ARG), (dict(out=None), gdn.ERR_ARG), (dict(cache=None), gdn.ERR_ARG),
    (dict(table=None), gdn.ERR_ARG), (dict(lens=None), gdn.ERR_ARG),
    (dict(q=BASE + 8), gdn.ERR_ALIGN), (dict(out=BASE + 264 * MB + 8), gdn.ERR_ALIGN),
    (dict(mask=BASE + 300 * MB + 1), gdn.ERR_ALIGN), (dict(cache=BASE + 128 * MB + 4), gdn.ERR_ALIGN),
    (dict(out=BASE), gdn.ERR_ALIAS), (dict(out=BASE + 128 * MB + 64), gdn.ERR_ALIAS),
    (dict(out=BASE + 256 * MB), gdn.ERR_ALIAS), (dict(mask=BASE + 264 * MB), gdn.ERR_ALIAS),
    (dict(max_pages=100, ws=BASE + 512 * MB, ws_bytes=64), gdn.ERR_WORKSPACE),
    (dict(max_pages=100, ws=BASE + 512 * MB + 16, ws_bytes=1 << 30), gdn.ERR_WORKSPACE),
    (dict(max_pages=100, ws=BASE, ws_bytes=1 << 30), gdn.ERR_ALIAS),
    (dict(max_pages=100, ws=BASE + 264 * MB, ws_bytes=1 << 30), gdn.ERR_ALIAS),
    (dict(B=1 << 12, H=8, Hkv=8, page=16, max_pages=1 << 20, table=1 << 50), gdn.ERR_ARG),     # 2^35 tiles
    (dict(B=1 << 20, H=1 << 12, Hkv=1), gdn.ERR_ARG),                # more rows than the join has blocks
])
def test_attention_refuses(L, kw, code):
    assert attend(L, **kw) == code


def test_attention_with_nothing_to_do(L):
    none = dict(q=None, cache=None, table=None, lens=None, out=None)
    assert attend(L, B=0, **none) == gdn.OK
    assert attend(L, H=0, Hkv=0, **none) == gdn.OK
    assert attend(L, n_q=0, q=None, out=None) == gdn.OK


def test_attention_workspace_sizes(L):
    ok = (2, 8, 2, 1, 128, 128, 64, 40)
    assert L.gdn_flash_attn_kv4_workspace_bytes(*ok) > 0
    # few short sequences: one kernel, no workspace
    assert L.gdn_flash_attn_kv4_workspace_bytes(2, 8, 2, 1, 128, 128, 64, 4) == 0
    # never more than the grid's runs ask for, however long the cache
    assert L.gdn_flash_attn_kv4_workspace_bytes(64, 32, 8, 1, 128, 128, 64, 1 << 16) < 64 << 20
    for i, bad in ((0, 0), (0, -1), (1, 0), (2, 3), (3, 0), (3, 20), (4, 96), (5, 32), (6, 24), (7, 0), (7, 1 << 26)):
        a = list(ok)
        a[i] = bad
        assert L.gdn_flash_attn_kv4_workspace_bytes(*a) == 0


def test_binding_refuses():
    import torch
    cache = gdn.kv4_cache(4, 2, 32, 64, device="cpu")
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros((1, 2, 1, 64))
    with pytest.raises(ValueError):                                  # not on a GPU
        gdn.kv4_write(k, k, cache, table, lens)
    with pytest.raises(ValueError):
        gdn.kv4_write(k, k, cache, table.long(), lens)
    with pytest.raises(ValueError):
        gdn.kv4_write(k, k, cache, table, lens.repeat(2))
    with pytest.raises(ValueError):
        gdn.kv4_write(k, k[:, :1], cache, table, lens)
    with pytest.raises(TypeError):
        gdn.kv4_write(k.double(), k.double(), cache, table, lens)
    with pytest.raises(ValueError):                                  # another width than the cache's
        gdn.kv4_read(cache, table, lens, 1, 128)
    with pytest.raises(TypeError):
        gdn.kv4_read(cache, table, lens, 1, 64, dtype=torch.int8)
