"""Page tables, rotary positions and the paged cache of 16- and 32-bit rows without a GPU: pins of their
oracle, the plan's arithmetic, refusals of the entry points, and orderings in the sources.

Calls that pass (made-up) device addresses are ones that the library must refuse during host validation;
none reaches a launch.
"""
import ctypes
import math
import os
import re
import subprocess
from fractions import Fraction

import numpy as np
import pytest

import linear_attention_sequence_gated_gb300 as gdn
from linear_attention_sequence_gated_gb300 import _build
from oracle import paged
from oracle.attn import attention

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE, MB = 1 << 40, 1 << 20
ptr = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
host = lambda x: None if x is None else (ctypes.c_longlong * len(x))(*x)  # noqa: E731


@pytest.fixture(scope="module")
def L():
    _build.build()
    return gdn.lib()


# ------------------------------------------------------------ the oracle

def test_oracle_pages_and_slots():
    table, free = np.full((2, 3), -1), [9, 8, 7]
    slots, pos, offsets, ok = paged.assign(table, [5, 3], [5, 3], free, 4, 5)
    assert ok and free == [] and table.tolist() == [[7, 8, -1], [9, -1, -1]]
    assert slots == [[28, 29, 30, 31, 32], [36, 37, 38, -1, -1]] and offsets == [0, 5, 8]
    assert pos == [[0, 1, 2, 3, 4], [0, 1, 2, 0, 0]]
    assert paged.assign(table, [5, 4], [0, 1], free, 4, 1, 3) == ([39, -1, -1], [3, 0, 0], [0, 0, 1], True)
    assert paged.release(table, [5, 4], [0, 0], free, 4, 10) == ([9, 8, 7], True)
    assert paged.release(table, [5, 4], [4, 4], free, 4, 10) == ([8], True)
    assert not paged.assign(table, [9, 4], [4, 0], [], 4, 4)[3]       # no page left


def test_oracle_rotary():
    x = np.arange(8.0).reshape(1, 1, 8)
    y = paged.rotary(x, np.array([[math.pi / 2]]), [1.0, 1.0], [0, 0])
    assert np.allclose(y[0, 0], [-2, -3, 0, 1, 4, 5, 6, 7])
    y = paged.rotary(x, np.array([[math.pi / 2]]), [1.0, 1.0], [0, 0], neighbours=True)
    assert np.allclose(y[0, 0], [-1, 0, -3, 2, 4, 5, 6, 7])
    z = np.random.default_rng(0).standard_normal((5, 2, 8))
    pos = np.array([[0, 3, 5, 7, 9], [1, 1, 2, 2, 3]])
    y = paged.rotary(z, pos, [1.0, 0.3, 0.1], [0, 1, 0])
    assert np.allclose(paged.rotary(y, pos, [1.0, 0.3, 0.1], [0, 1, 0], inverse=True), z)
    assert np.allclose((y ** 2).sum(-1), (z ** 2).sum(-1)) and np.array_equal(y[..., 6:], z[..., 6:])


def test_oracle_attention_is_dense_attention_on_gathered_rows():
    rng = np.random.default_rng(1)
    kc, vc = rng.standard_normal((5, 2, 4, 8)), rng.standard_normal((5, 2, 4, 6))
    table, q = np.array([[3, 0], [1, 4]]), rng.standard_normal((2, 4, 2, 8))
    got = paged.attend(q, kc, vc, table, [6, 0])
    k = np.concatenate([kc[3], kc[0]], axis=1)[None, :, :6]
    v = np.concatenate([vc[3], vc[0]], axis=1)[None, :, :6]
    assert np.allclose(got[:1], attention(q[:1], k, v)) and not got[1].any()
    hide = np.where(np.arange(6)[None] > 4 + np.arange(2)[:, None], -np.inf, 0.0)[None, None]
    assert np.allclose(paged.attend(q, kc, vc, table, [6, 0], causal=True)[:1], attention(q[:1], k, v, hide))
    vc[0, :, 1:] = np.nan                # behind the end
    assert np.isfinite(paged.attend(q, kc, vc, table, [5, 0])).all()


# ------------------------------------------------------------ the plan

def test_plan_holds_the_turns_of_each_frequency():
    for base in (1e4, 5e5, 1e7):
        p = gdn.rotary_plan(128, base, sections=[16, 24, 24], device="cpu").data.numpy().view(np.uint64)
        for j in range(64):
            f = base ** (-2 * j / 128)
            # two fp64 roundings of a share of a turn, and what 64 bits cut off
            assert abs(int(p[j, 0]) / 2.0 ** 64 - f / (2 * math.pi)) <= 2.0 ** -52 * f + 2.0 ** -64
            assert p[j, 1] == (0 if j < 16 else 1 if j < 40 else 2)
    p = gdn.rotary_plan(16, freqs=[0, -1e-30, -0.25, 2 * math.pi, 100.5, 1e-9, 3.0, -7.0], device="cpu")
    turns = p.data.numpy().view(np.uint64)[:, 0].astype(np.float64) / 2.0 ** 64
    want = np.array([0, 0, 1 - 0.25 / (2 * math.pi), 0, (100.5 / (2 * math.pi)) % 1, 1e-9 / (2 * math.pi),
                     3 / (2 * math.pi), (-7 / (2 * math.pi)) % 1])
    off = np.abs(turns - want)
    assert (np.minimum(off, 1 - off) <= 2.0 ** -48).all()


def test_plan_is_exact_to_64_bits():
    """A 32-bit position multiplies what a frequency's share of a turn is off by."""
    turn = Fraction("0.1591549430918953357688837633725143620344596457404564487476673440588968")      # 1 / (2 pi)
    rng = np.random.default_rng(5)
    freqs = [0.0, 1.0, -1.0, 0.1, 1e-4, -3e-7, 1e-20, -1e-30, 5e-324, 2 * math.pi, -2 * math.pi, math.pi, 12345.678, -1e9] + \
        [1e6 ** (-j / 8) for j in range(8)] + list(rng.standard_normal(42))
    plan = gdn.rotary_plan(128, freqs=freqs, device="cpu").data.numpy().view(np.uint64)
    for f, p in zip(freqs, plan[:, 0]):
        off = (int(p) - turn * Fraction(f) * 2 ** 64) % 2 ** 64
        # two truncations; the second double's rounding, 2^-106 of the turns, and its product's are far below
        assert min(off, 2 ** 64 - off) <= 2 + abs(f) * 2.0 ** -40, f


def test_plan_deals_axes_and_refuses():
    axes = lambda **kw: gdn.rotary_plan(16, device="cpu", **kw).data[:, 1].tolist()  # noqa: E731
    assert axes() == [0] * 8
    assert axes(sections=[2, 3, 3]) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert axes(sections=[2, 3, 3], dealt=True) == [0, 1, 2, 0, 1, 2, 1, 2]
    assert axes(sections=[0, 8]) == [1] * 8 and axes(sections=[1, 0, 7], dealt=True) == [0] + [2] * 7
    for bad in (dict(sections=[3, 3]), dict(sections=[]), dict(sections=[9, -1]), dict(freqs=[1.0])):
        with pytest.raises(ValueError):
            gdn.rotary_plan(16, device="cpu", **bad)
    with pytest.raises(gdn.GdnError):
        gdn.rotary_plan(24, device="cpu")
    with pytest.raises(gdn.GdnError):
        gdn.rotary_plan(16, freqs=[float("nan")] + [1.0] * 7, device="cpu")
    assert gdn.lib().gdn_rotary_plan(None, None, -1, None) == gdn.ERR_ARG
    assert gdn.lib().gdn_rotary_plan(None, None, 2, None) == gdn.ERR_ARG
    assert gdn.lib().gdn_rotary_plan(None, None, 0, None) == gdn.OK
    neg = (ctypes.c_int * 1)(-1)
    assert gdn.lib().gdn_rotary_plan((ctypes.c_double * 1)(1.0), neg, 1, (ctypes.c_int * 4)()) == gdn.ERR_ARG


# ------------------------------------------------------------ how attention is shared out

@pytest.fixture(scope="module")
def H(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("paged") / "paged_host.so")
    subprocess.check_call([_build.nvcc()] + _build.ARCH + ["-std=c++17", "--expt-relaxed-constexpr", "-shared", "-Xcompiler", "-fPIC",
                                                          "-o", so, os.path.join(ROOT, "tests", "paged_host.cu")])
    return ctypes.CDLL(so)


@pytest.mark.parametrize("elt", [2, 4])
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("dv", [64, 128, 256])
def test_rings_are_a_whole_number_of_tiles_a_group(H, elt, dk, dv):
    """A barrier's parity tells a phase from the next only, so a stage belongs to one group; and all rows have a block."""
    out = (ctypes.c_int * 8)()
    for R in list(range(1, 200)) + [760, 5000]:
        H.paged_share(dk, dv, elt, R, out)
        warps, most, blocks, groups, units, ring, pool, queries = out
        assert ring % groups == 0 and groups <= ring <= 48 and 1 <= groups * blocks <= warps
        assert blocks <= most and 8 * blocks * units >= R and 8 * blocks * (units - 1) < R
        assert ring * 16 * (dk + dv) * elt + queries <= pool <= 224 << 10
        assert warps * 8 * (dv + 4) * 4 <= ring * 16 * (dk + dv) * elt       # the last unit is joined in the ring


def test_quotients_by_a_known_number(H):
    rng = np.random.default_rng(3)
    for d in list(range(1, 300)) + [2 ** k + e for k in range(9, 31) for e in (-1, 0, 1)] + [2 ** 31 - 1]:
        x = np.unique(np.concatenate([[0, 1, d - 1, min(d, 2 ** 31 - 1), 2 ** 31 - 1], rng.integers(0, 2 ** 31, 50),
                                      np.minimum(rng.integers(0, 2 ** 31 // d + 1, 50) * d, 2 ** 31 - 1)])).astype(np.int32)
        got = np.zeros_like(x)
        H.paged_quotients(d, ctypes.c_void_p(x.ctypes.data), x.size, ctypes.c_void_p(got.ctypes.data))
        assert np.array_equal(got, x // d)


# ------------------------------------------------------------ refusals

def assign(L, **kw):
    a = dict(table=BASE, lens=BASE + MB, new=None, free=BASE + 2 * MB, count=BASE + 3 * MB, slots=BASE + 4 * MB,
             positions=BASE + 5 * MB, offsets=None, B=4, n_new=2, n_tokens=0, page=16, max_pages=8, n_pages=100)
    a.update(kw)
    return L.gdn_page_assign(*(ptr(a[k]) for k in ("table", "lens", "new", "free", "count", "slots", "positions", "offsets")),
                             a["B"], a["n_new"], a["n_tokens"], a["page"], a["max_pages"], a["n_pages"], None)


def release(L, **kw):
    a = dict(table=BASE, lens=BASE + MB, to=None, free=BASE + 2 * MB, count=BASE + 3 * MB, B=4, page=16, max_pages=8,
             n_pages=100)
    a.update(kw)
    return L.gdn_page_release(ptr(a["table"]), ptr(a["lens"]), ptr(a["to"]), ptr(a["free"]), ptr(a["count"]), a["B"], a["page"],
                              a["max_pages"], a["n_pages"], None)


PAGES = [(dict(B=-1), gdn.ERR_ARG), (dict(max_pages=-1), gdn.ERR_ARG), (dict(n_pages=-1), gdn.ERR_ARG),
         (dict(page=0), gdn.ERR_SHAPE), (dict(B=16385), gdn.ERR_SHAPE), (dict(max_pages=1 << 28), gdn.ERR_ARG),
         (dict(n_pages=1 << 28), gdn.ERR_ARG), (dict(B=16384, max_pages=1 << 18, page=1), gdn.ERR_ARG),
         (dict(table=None), gdn.ERR_ARG), (dict(lens=None), gdn.ERR_ARG), (dict(free=None), gdn.ERR_ARG),
         (dict(count=None), gdn.ERR_ARG), (dict(table=BASE + 2), gdn.ERR_ALIGN), (dict(lens=BASE + MB + 1), gdn.ERR_ALIGN),
         (dict(free=BASE + 2 * MB + 2), gdn.ERR_ALIGN), (dict(count=BASE + 3 * MB + 3), gdn.ERR_ALIGN),
         (dict(free=BASE + 64), gdn.ERR_ALIAS), (dict(count=BASE + MB + 4), gdn.ERR_ALIAS),
         (dict(count=BASE + 2 * MB + 8), gdn.ERR_ALIAS)]


@pytest.mark.parametrize("kw,code", PAGES + [
    (dict(n_new=-1), gdn.ERR_ARG), (dict(n_tokens=-1), gdn.ERR_ARG), (dict(n_new=1 << 30), gdn.ERR_ARG),
    (dict(slots=None), gdn.ERR_ARG), (dict(new=BASE + 6 * MB + 2), gdn.ERR_ALIGN), (dict(slots=BASE + 4 * MB + 1), gdn.ERR_ALIGN),
    (dict(positions=BASE + 5 * MB + 2), gdn.ERR_ALIGN), (dict(offsets=BASE + 6 * MB + 2, n_tokens=8), gdn.ERR_ALIGN),
    (dict(offsets=BASE + 6 * MB, n_tokens=2 ** 31 - 1), gdn.ERR_ARG), (dict(table=BASE + MB - 16), gdn.ERR_ALIAS),
    (dict(slots=BASE + 5 * MB), gdn.ERR_ALIAS), (dict(slots=BASE + MB), gdn.ERR_ALIAS), (dict(positions=BASE + 3 * MB), gdn.ERR_ALIAS),
    (dict(offsets=BASE + 4 * MB, n_tokens=8), gdn.ERR_ALIAS), (dict(new=BASE + 4 * MB), gdn.ERR_ALIAS),
])
def test_page_assign_refuses(L, kw, code):
    assert assign(L, **kw) == code


@pytest.mark.parametrize("kw,code", PAGES + [(dict(to=BASE + 4 * MB + 1), gdn.ERR_ALIGN), (dict(to=BASE + 2 * MB + 4), gdn.ERR_ALIAS)])
def test_page_release_refuses(L, kw, code):
    assert release(L, **kw) == code


def test_no_sequences_nothing_done(L):
    assert assign(L, B=0, n_new=3, table=None, lens=None, free=None, count=None, slots=None, positions=None) == gdn.OK
    assert release(L, B=0, table=None, lens=None, free=None, count=None) == gdn.OK


def turn(L, **kw):
    a = dict(q=BASE, qo=BASE + 64 * MB, k=BASE + 128 * MB, ko=BASE + 192 * MB, strides=None, pos=BASE + 256 * MB,
             plan=BASE + 257 * MB, T=100, H=8, Hk=2, d=128, r=128, axes=1, flags=0, dtype=1)
    a.update(kw)
    return L.gdn_rotary(ptr(a["q"]), ptr(a["qo"]), ptr(a["k"]), ptr(a["ko"]), host(a["strides"]), ptr(a["pos"]), ptr(a["plan"]),
                        a["T"], a["H"], a["Hk"], a["d"], a["r"], a["axes"], a["flags"], a["dtype"], None)


DENSE = (1024, 128, 1024, 128, 256, 128, 256, 128)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), gdn.ERR_ARG), (dict(H=-1), gdn.ERR_ARG), (dict(Hk=-1), gdn.ERR_ARG), (dict(dtype=3), gdn.ERR_ARG),
    (dict(flags=4), gdn.ERR_ARG), (dict(axes=0), gdn.ERR_ARG), (dict(d=8), gdn.ERR_HEADDIM), (dict(d=120), gdn.ERR_HEADDIM),
    (dict(d=272), gdn.ERR_HEADDIM), (dict(r=-16), gdn.ERR_HEADDIM), (dict(r=24), gdn.ERR_HEADDIM), (dict(r=144), gdn.ERR_HEADDIM),
    (dict(q=None), gdn.ERR_ARG), (dict(qo=None), gdn.ERR_ARG), (dict(k=None), gdn.ERR_ARG), (dict(ko=None), gdn.ERR_ARG),
    (dict(pos=None), gdn.ERR_ARG), (dict(plan=None), gdn.ERR_ARG), (dict(q=BASE + 8), gdn.ERR_ALIGN),
    (dict(ko=BASE + 192 * MB + 4), gdn.ERR_ALIGN), (dict(pos=BASE + 256 * MB + 2), gdn.ERR_ALIGN),
    (dict(plan=BASE + 257 * MB + 8), gdn.ERR_ALIGN), (dict(qo=BASE + 16), gdn.ERR_ALIAS), (dict(qo=BASE + 128 * MB), gdn.ERR_ALIAS),
    (dict(ko=BASE + 64 * MB), gdn.ERR_ALIAS), (dict(ko=BASE + 256 * MB), gdn.ERR_ALIAS), (dict(qo=BASE + 257 * MB), gdn.ERR_ALIAS),
    (dict(strides=(-1024,) + DENSE[1:]), gdn.ERR_ARG), (dict(strides=(1 << 60,) + DENSE[1:]), gdn.ERR_ARG),
    (dict(strides=(1028,) + DENSE[1:]), gdn.ERR_ALIGN), (dict(strides=(1024, 128, 1024, 64, 256, 128, 256, 128)), gdn.ERR_ALIAS),
    (dict(strides=(1024, 128, 512, 128, 256, 128, 256, 128)), gdn.ERR_ALIAS),          # rows of an output share bytes
    (dict(strides=(1024, 128, 0, 128, 256, 128, 256, 128)), gdn.ERR_ALIAS),
    # turned in place with other strides, and joint rows whose heads overlap
    (dict(qo=BASE, strides=(1024, 128, 2048, 128, 256, 128, 256, 128)), gdn.ERR_ALIAS),
    (dict(qo=BASE, k=BASE + 1792, ko=BASE + 1792, strides=(1280, 128) * 4), gdn.ERR_ALIAS),
])
def test_rotary_refuses(L, kw, code):
    assert turn(L, **kw) == code


def test_rotary_with_nothing_to_do(L):
    none = dict(q=None, qo=None, k=None, ko=None, pos=None, plan=None)
    assert turn(L, T=0, **none) == gdn.OK
    assert turn(L, H=0, Hk=0, **none) == gdn.OK


def put(L, **kw):
    a = dict(q=BASE, qo=BASE + 64 * MB, k=BASE + 128 * MB, v=BASE + 160 * MB, qs=None, st=None, kc=BASE + 192 * MB,
             vc=BASE + 448 * MB, cs=None, pos=BASE + 900 * MB, plan=BASE + 901 * MB, slots=BASE + 902 * MB, T=100, H=8, Hk=2,
             dk=128, dv=128, r=128, axes=1, n_pages=50, page=16, flags=0, dtype=1)
    a.update(kw)
    return L.gdn_rotary_write(ptr(a["q"]), ptr(a["qo"]), ptr(a["k"]), ptr(a["v"]), host(a["qs"]), host(a["st"]), ptr(a["kc"]),
                              ptr(a["vc"]), host(a["cs"]), ptr(a["pos"]), ptr(a["plan"]), ptr(a["slots"]), a["T"], a["H"],
                              a["Hk"], a["dk"], a["dv"], a["r"], a["axes"], a["n_pages"], a["page"], a["flags"], a["dtype"], None)


CACHE = (4096, 2048, 128)


@pytest.mark.parametrize("kw,code", [
    (dict(n_pages=-1), gdn.ERR_ARG), (dict(page=0), gdn.ERR_SHAPE), (dict(n_pages=1 << 20, page=1 << 12), gdn.ERR_ARG),
    (dict(flags=2), gdn.ERR_ARG), (dict(dv=100), gdn.ERR_HEADDIM), (dict(dk=0), gdn.ERR_HEADDIM), (dict(slots=None), gdn.ERR_ARG),
    (dict(kc=None), gdn.ERR_ARG), (dict(vc=None), gdn.ERR_ARG), (dict(v=None), gdn.ERR_ARG),
    (dict(slots=BASE + 902 * MB + 2), gdn.ERR_ALIGN), (dict(kc=BASE + 192 * MB + 8), gdn.ERR_ALIGN),
    (dict(kc=BASE + 128 * MB), gdn.ERR_ALIAS), (dict(vc=BASE + 192 * MB), gdn.ERR_ALIAS), (dict(vc=BASE), gdn.ERR_ALIAS),
    (dict(kc=BASE + 902 * MB), gdn.ERR_ALIAS), (dict(qo=BASE + 192 * MB), gdn.ERR_ALIAS),
    (dict(cs=CACHE + (4096, 2048, 132)), gdn.ERR_ALIGN), (dict(cs=(0, 2048, 128) + CACHE), gdn.ERR_ALIAS),
    (dict(cs=(4096, 1024, 128) + CACHE), gdn.ERR_ALIAS), (dict(cs=(-4096, 2048, 128) + CACHE), gdn.ERR_ARG),
    # keys and values of one buffer, a page's values half inside its keys
    (dict(vc=BASE + 192 * MB + 4096, cs=(8192, 2048, 128) * 2), gdn.ERR_ALIAS),
])
def test_rotary_write_refuses(L, kw, code):
    assert put(L, **kw) == code


def test_paged_write_refuses(L):
    f = lambda **kw: (lambda a: L.gdn_paged_write(  # noqa: E731
        ptr(a["k"]), ptr(a["v"]), None, ptr(a["kc"]), ptr(a["vc"]), None, ptr(a["slots"]), a["T"], a["Hk"], a["dk"], a["dv"],
        a["n_pages"], 16, a["dtype"], None))(dict(dict(k=BASE, v=BASE + 64 * MB, kc=BASE + 128 * MB, vc=BASE + 256 * MB,
                                                      slots=BASE + 512 * MB, T=4, Hk=2, dk=128, dv=64, n_pages=9, dtype=0), **kw))
    for kw, code in ((dict(k=None), gdn.ERR_ARG), (dict(T=-1), gdn.ERR_ARG), (dict(Hk=-1), gdn.ERR_ARG), (dict(dk=24), gdn.ERR_HEADDIM),
                     (dict(dtype=7), gdn.ERR_ARG), (dict(slots=None), gdn.ERR_ARG), (dict(vc=BASE + 128 * MB + 64), gdn.ERR_ALIAS),
                     (dict(T=0, k=None, v=None, kc=None, vc=None, slots=None), gdn.OK), (dict(Hk=0, k=None, v=None), gdn.OK)):
        assert f(**kw) == code


def attend(L, **kw):
    a = dict(q=BASE, qs=None, kc=BASE + 128 * MB, vc=BASE + 192 * MB, cs=None, table=BASE + 256 * MB, lens=BASE + 260 * MB,
             mask=None, out=BASE + 264 * MB, B=2, H=8, Hkv=2, n_q=1, dk=128, dv=128, n_pages=8, page=64, max_pages=4,
             scale=0.1, causal=0, dtype=1, out_dtype=0, ws=None, ws_bytes=0)
    a.update(kw)
    return L.gdn_flash_attn_paged(ptr(a["q"]), host(a["qs"]), ptr(a["kc"]), ptr(a["vc"]), host(a["cs"]), ptr(a["table"]),
                                  ptr(a["lens"]), ptr(a["mask"]), ptr(a["out"]), a["B"], a["H"], a["Hkv"], a["n_q"], a["dk"],
                                  a["dv"], a["n_pages"], a["page"], a["max_pages"], ctypes.c_float(a["scale"]), a["causal"],
                                  a["dtype"], a["out_dtype"], ptr(a["ws"]), a["ws_bytes"], None)


NEST = (2 * 64 * 128, 64 * 128, 128)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), gdn.ERR_ARG), (dict(H=-1), gdn.ERR_ARG), (dict(n_q=-1), gdn.ERR_ARG), (dict(Hkv=3), gdn.ERR_ARG),
    (dict(Hkv=0), gdn.ERR_ARG), (dict(n_q=20), gdn.ERR_SHAPE), (dict(dk=96), gdn.ERR_HEADDIM),
    (dict(dv=512), gdn.ERR_HEADDIM), (dict(page=8), gdn.ERR_SHAPE), (dict(page=24), gdn.ERR_SHAPE),
    (dict(max_pages=1 << 26), gdn.ERR_ARG), (dict(n_pages=-1), gdn.ERR_ARG), (dict(max_pages=-1), gdn.ERR_ARG),
    (dict(scale=float("nan")), gdn.ERR_ARG), (dict(scale=float("inf")), gdn.ERR_ARG),
    (dict(causal=2), gdn.ERR_ARG), (dict(dtype=3), gdn.ERR_ARG), (dict(out_dtype=3), gdn.ERR_ARG),
    (dict(q=None), gdn.ERR_ARG), (dict(out=None), gdn.ERR_ARG), (dict(kc=None), gdn.ERR_ARG), (dict(vc=None), gdn.ERR_ARG),
    (dict(table=None), gdn.ERR_ARG), (dict(lens=None), gdn.ERR_ARG),
    (dict(q=BASE + 8), gdn.ERR_ALIGN), (dict(out=BASE + 264 * MB + 8), gdn.ERR_ALIGN),
    (dict(mask=BASE + 300 * MB + 1), gdn.ERR_ALIGN), (dict(kc=BASE + 128 * MB + 4), gdn.ERR_ALIGN),
    (dict(qs=(1024, 132, 128)), gdn.ERR_ALIGN), (dict(qs=(1024, -128, 128)), gdn.ERR_ARG), (dict(qs=(1 << 60, 128, 128)), gdn.ERR_ARG),
    (dict(out=BASE), gdn.ERR_ALIAS), (dict(out=BASE + 128 * MB + 64), gdn.ERR_ALIAS), (dict(out=BASE + 192 * MB), gdn.ERR_ALIAS),
    (dict(out=BASE + 256 * MB), gdn.ERR_ALIAS), (dict(mask=BASE + 264 * MB), gdn.ERR_ALIAS),
    (dict(max_pages=100, ws=BASE + 512 * MB, ws_bytes=64), gdn.ERR_WORKSPACE),
    (dict(max_pages=100, ws=BASE + 512 * MB + 16, ws_bytes=1 << 30), gdn.ERR_WORKSPACE),
    (dict(max_pages=100, ws=BASE, ws_bytes=1 << 30), gdn.ERR_ALIAS),
    (dict(max_pages=100, ws=BASE + 264 * MB, ws_bytes=1 << 30), gdn.ERR_ALIAS),
    (dict(B=1 << 12, H=8, Hkv=8, page=16, max_pages=1 << 20, table=1 << 50), gdn.ERR_ARG),     # 2^35 tiles
    (dict(cs=NEST + (2 * 64 * 128, 64 * 128, 120)), gdn.ERR_SHAPE),       # a token inside the one before
    (dict(cs=NEST + (2 * 64 * 128, 64 * 100, 128)), gdn.ERR_SHAPE),       # a head inside the one before
    (dict(cs=NEST + (2 * 64 * 128 + 64, 64 * 128, 128)), gdn.ERR_SHAPE),  # pages that hold no whole number of heads
    (dict(cs=NEST + (2 * 64 * 128, 64 * 128, 132)), gdn.ERR_ALIGN), (dict(cs=NEST + (0, 64 * 128, 128)), gdn.ERR_SHAPE),
    (dict(cs=NEST + (-8, 64 * 128, 128)), gdn.ERR_ARG), (dict(cs=NEST + (1 << 41, 64 * 128, 128)), gdn.ERR_ARG),
])
def test_attention_refuses(L, kw, code):
    assert attend(L, **kw) == code


def test_attention_with_nothing_to_do(L):
    none = dict(q=None, kc=None, vc=None, table=None, lens=None, out=None)
    assert attend(L, B=0, **none) == gdn.OK
    assert attend(L, H=0, Hkv=0, **none) == gdn.OK
    assert attend(L, n_q=0, q=None, out=None) == gdn.OK


def test_attention_supports_and_workspace_sizes(L):
    assert gdn.flash_attn_paged_supports(1, 64, 256) and gdn.flash_attn_paged_supports(19, 128, 128)
    for bad in ((0, 64, 64), (20, 64, 64), (1, 96, 64), (1, 64, 32)):
        assert not gdn.flash_attn_paged_supports(*bad)
    ok = (2, 8, 2, 1, 128, 128, 64, 100, 1)
    f = L.gdn_flash_attn_paged_workspace_bytes
    assert f(*ok) > 0
    assert f(2, 8, 2, 1, 128, 128, 64, 4, 1) == 0                         # few tiles: one launch, no workspace
    assert f(64, 32, 8, 1, 128, 128, 64, 1 << 16, 1) < 64 << 20           # never more than the grid's runs ask for
    for i, bad in ((0, 0), (0, -1), (1, 0), (2, 3), (3, 0), (3, 20), (4, 96), (5, 32), (6, 24), (7, 0), (7, 1 << 26), (8, 3)):
        a = list(ok)
        a[i] = bad
        assert f(*a) == 0


def test_binding_refuses():
    import torch
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kc, vc = gdn.paged_cache(4, 2, 32, 64, device="cpu")
    assert tuple(gdn.paged_cache(4, 2, 32, 64, 128, dtype=torch.float32, device="cpu")[1].shape) == (4, 2, 32, 128)
    with pytest.raises(TypeError):
        gdn.paged_cache(4, 2, 32, 64, dtype=torch.int8, device="cpu")
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    plan = gdn.rotary_plan(64, device="cpu")
    q = torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16)
    for call in (lambda: gdn.paged_write(k, k, kc, vc, i32(3)),                       # not on a GPU
                 lambda: gdn.rotary(k, k, i32(3), plan),
                 lambda: gdn.rotary_write(k, k, k, i32(3), plan, kc, vc, i32(3)),
                 lambda: gdn.flash_attn_paged(q, kc, vc, i32(3, 2), i32(3)),
                 lambda: gdn.page_assign(i32(3, 2), i32(3), i32(9), i32(1), 16),
                 lambda: gdn.page_release(i32(3, 2), i32(3), i32(9), i32(1), 16),
                 lambda: gdn.flash_attn_paged(q[..., :32], kc, vc, i32(3, 2), i32(3)),
                 lambda: gdn.paged_write(k, k, kc.float(), vc, i32(3)),
                 lambda: gdn.rotary(k, None, i32(3), plan, k_out=k)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gdn.paged_write(k.double(), k.double(), kc, vc, i32(3)),
                 lambda: gdn.rotary(k.int(), None, i32(3), plan),
                 lambda: gdn.flash_attn_paged(q.double(), kc, vc, i32(3, 2), i32(3)),
                 lambda: gdn.rotary_write(k, k, k, i32(3), None, kc, vc, i32(3)),
                 lambda: gdn.rotary_write(None, k, k, i32(3), plan, kc, vc, i32(3))):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------ the sources

CSRC = os.path.join(ROOT, "linear_attention_sequence_gated_gb300", "csrc")


@pytest.mark.parametrize("name", ["gdn_pages.cu", "gdn_paged.cu", "gdn_paged_attn.cuh"])
def test_kernels_that_start_early_read_with_ordinary_loads(name):
    """They run while the kernel before them still writes what they read, until they have waited for its end:
    non-coherent loads and the cache-hint intrinsics are not ordered behind that wait."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.findall(r"\b__ld(?:g|cg|ca|cs|lu|cv)\s*\(", text)
    assert not re.findall(r"ld\.global(?:\.\w+)*\.nc", text)
    assert len(re.findall(r"__global__", text)) == len(re.findall(r"after_the_kernel_before\(\);", text))
    # the thread that initialises barriers fences them: in its condition's block, behind the loop at most
    for init in re.finditer(r"\bmbar_init\s*\(", text):
        assert re.match(r"[^{}]*(?:\}\s*)?ptx::fence_mbar_init\(\);", text[init.start():]), text[init.start():][:200]
