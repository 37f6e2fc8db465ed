"""GPU tests of rotary positions and of writes into a paged cache against the oracle (oracle/paged.py).

Bounds.  A turned element is x c - y s in fp32: c and s are off by at most 2^-24 (their rounding) + 2^-23 (an fp32 unit of
the function at most) + 2 pi 2^-32 (the angle) < 2^-22 of 1, the product and the sum by 2^-24 each, so the result by 2^-21 of
|x| + |y|, and by half a step of its type.  Copies are exact.
"""
import math

import numpy as np
import pytest
import torch

import linear_attention_sequence_gated_gb300 as gdn
from oracle import paged

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


def randn(shape, dtype, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(DTYPES[dtype])


def freqs_of(r, base):
    return [base ** (-2 * j / r) for j in range(r // 2)]


def near(got, want, x, r, neighbours):
    """Within the bound above, and exact from element r on."""
    a, b = (slice(0, r, 2), slice(1, r, 2)) if neighbours else (slice(0, r // 2), slice(r // 2, r))
    size = np.abs(x[..., a]) + np.abs(x[..., b])
    room = np.zeros_like(x)
    room[..., a] = room[..., b] = 2.0 ** -21 * size
    step = torch.finfo(got.dtype).eps / 2
    y = np64(got)
    # (subnormal f16 results round to multiples of 2^-24)
    assert (np.abs(y - want) <= room + step * (np.abs(want) + room) * (room > 0) + (2.0 ** -25) * (room > 0)).all()
    assert np.array_equal(y[..., r:], x[..., r:])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("d,r", [(64, 64), (128, 128), (256, 256), (256, 64), (96, 96), (96, 48), (16, 16), (128, 32),
                                 (112, 16), (240, 208), (128, 0)])
def test_widths_and_types(dtype, neighbours, d, r):
    for T, H, Hk in ((1, 1, 1), (5, 8, 2), (67, 3, 5)):
        q, k = randn((T, H, d), dtype, T), randn((T, Hk, d), dtype, T + 1)
        pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3 - 2
        plan = gdn.rotary_plan(r, 1e4, neighbours=neighbours)
        axes = [0] * (r // 2)
        p = np64(pos)[None]
        for inverse in (False, True):
            qo, ko = gdn.rotary(q, k, pos, plan, inverse=inverse)
            for got, x in ((qo, q), (ko, k)):
                near(got, paged.rotary(np64(x), p, freqs_of(r, 1e4), axes, neighbours, inverse), np64(x), r, neighbours)
    assert gdn.device_status() == gdn.OK


@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("sections", [[16, 24, 24], [64], [0, 64], [10, 0, 54], [1, 2, 3, 58], [63, 1]])
def test_several_axes(dealt, sections):
    T, d, r = 50, 128, 128
    q = randn((T, 4, d), "f32", 1)
    rng = np.random.default_rng(0)
    pos = rng.integers(-100, 5000, (len(sections), T))
    left, axes = list(sections), []
    while sum(left):
        for a in range(len(left)):
            n = 1 if dealt else left[a]
            if left[a]:
                axes += [a] * n
                left[a] -= n
    plan = gdn.rotary_plan(r, 5e5, sections=sections, dealt=dealt)
    got, none = gdn.rotary(q, None, i32(pos), plan)
    assert none is None
    near(got, paged.rotary(np64(q), pos, freqs_of(r, 5e5), axes), np64(q), r, False)


@pytest.mark.parametrize("base", [1e4, 1e7])
def test_far_positions(base):
    """As accurate at 2^31 - 1 as at 1.  The frequencies are fp64 numbers of the user's: one unit of the first, 1, is
    2^-53 / (2 pi) of a turn, 2^-24 radians at the far end, which the bound takes on."""
    pos = [0, 1, 1000, 10 ** 6, 10 ** 9, 2 ** 31 - 1, -2 ** 31, -12345678]
    x = randn((len(pos), 2, 128), "f32", 2)
    f = freqs_of(128, base)
    # turns in exact integers: the fp64 frequency as a fraction, and pi to 50 digits
    from fractions import Fraction
    two_pi = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    want = np64(x)
    for t, p in enumerate(pos):
        turns = np.array([float((Fraction(v) * p / two_pi) % 1) for v in f])
        z = np.exp(2j * np.pi * turns)
        w = (want[t, :, :64] + 1j * want[t, :, 64:]) * z
        want[t, :, :64], want[t, :, 64:] = w.real, w.imag
    got, _ = gdn.rotary(x, None, i32(pos), gdn.rotary_plan(128, base))
    size = np.abs(np64(x))[..., :64] + np.abs(np64(x))[..., 64:]
    size = np.concatenate([size, size], -1)
    assert (np.abs(np64(got) - want) <= (2.0 ** -21 + 2.0 ** -24) * size + 2.0 ** -24 * np.abs(want)).all()


def test_given_frequencies():
    """Negative ones, none at all, more than a radian a position."""
    f = [0.0, -0.25, 3.0, 100.5, 1e-9, 2 * math.pi, 0.7, -7.0]
    x = randn((40, 2, 16), "f32", 3)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    got, _ = gdn.rotary(x, None, pos, gdn.rotary_plan(16, freqs=f))
    near(got, paged.rotary(np64(x), np64(pos)[None], f, [0] * 8), np64(x), 16, False)


@pytest.mark.parametrize("neighbours", [False, True])
def test_the_gradient(neighbours):
    """inverse=True against differences of the formula, and as the transpose: <rotary(x), y> = <x, inverse(y)>."""
    x, y = randn((6, 2, 32), "f32", 4), randn((6, 2, 32), "f32", 5)
    pos = i32([0, 1, 7, 100, 1000, -3])
    plan = gdn.rotary_plan(32, 100.0, neighbours=neighbours)
    out, _ = gdn.rotary(x, None, pos, plan)
    dx, _ = gdn.rotary(y, None, pos, plan, inverse=True)
    assert abs((np64(out) * np64(y)).sum() - (np64(x) * np64(dx)).sum()) <= 2.0 ** -20 * np.abs(np64(x) * np64(y)).sum()
    f, h = freqs_of(32, 100.0), 1e-4
    loss = lambda z: (paged.rotary(z, np64(pos)[None], f, [0] * 16, neighbours) * np64(y)).sum()  # noqa: E731
    for i in range(0, 384, 13):
        e = np.zeros(384)
        e[i] = h
        e = e.reshape(6, 2, 32)
        diff = (loss(np64(x) + e) - loss(np64(x) - e)) / (2 * h)
        assert abs(diff - np64(dx).ravel()[i]) <= 1e-5


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_in_place_and_strided(dtype):
    """Heads of one projection's rows turned where they are; a transposed view; outputs of other strides."""
    T, H, Hk, d = 23, 6, 2, 64
    joint = randn((T, H + 2 * Hk, d), dtype, 6)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 5
    plan = gdn.rotary_plan(d)
    q, k = joint[:, :H], joint[:, H:H + Hk]
    want = gdn.rotary(q.contiguous(), k.contiguous(), pos, plan)
    was = joint.clone()
    a, b = gdn.rotary(q, k, pos, plan, q_out=q, k_out=k)
    assert a is q and b is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(joint[:, H + Hk:], was[:, H + Hk:])
    heads_first = was[:, :H].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((H, T, d), dtype=DTYPES[dtype], device="cuda").transpose(0, 1)
    gdn.rotary(heads_first, None, pos, plan, q_out=out)
    assert torch.equal(out, want[0])
    one = was[:, :1, :].expand(T, H, d)                 # an input of stride 0
    assert torch.equal(gdn.rotary(one, None, pos, plan)[0], gdn.rotary(one.contiguous(), None, pos, plan)[0])


def test_non_finite_rows_stay_by_themselves():
    x = randn((4, 3, 64), "bf16", 7)
    want, _ = gdn.rotary(x, None, i32([1, 2, 3, 4]), gdn.rotary_plan(64))
    x[2, 1, 5] = float("inf")
    got, _ = gdn.rotary(x, None, i32([1, 2, 3, 4]), gdn.rotary_plan(64))
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[2, 1, 5] = bad[2, 1, 37] = True
    assert torch.equal(got[~bad], want[~bad]) and not torch.isfinite(got[bad]).any()


def pages(layout, n_pages, H, page, dk, dv, dtype):
    """Caches that hold a number everywhere, in one of several orders."""
    full = lambda *s: torch.full(s, 7.0, dtype=DTYPES[dtype], device="cuda")  # noqa: E731
    if layout == "heads":
        return full(n_pages, H, page, dk), full(n_pages, H, page, dv)
    if layout == "tokens":
        return full(n_pages, page, H, dk).transpose(1, 2), full(n_pages, page, H, dv).transpose(1, 2)
    both = full(n_pages, 2, H, page, max(dk, dv))
    return both[:, 0, :, :, :dk], both[:, 1, :, :, :dv]


@pytest.mark.parametrize("layout", ["heads", "tokens", "joint"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dk,dv,page", [(128, 128, 16), (64, 256, 5), (96, 16, 1), (256, 64, 64)])
def test_writes(layout, dtype, dk, dv, page):
    """Every row to its slot and nothing else: skipped tokens, one token, many; strided rows."""
    rng = np.random.default_rng(page)
    for T, H in ((1, 1), (37, 3), (300, 8)):
        n_pages = -(-T // page) + 4
        kc, vc = pages(layout, n_pages, H, page, dk, dv, dtype)
        slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
        if T > 1:
            slots[rng.random(T) < 0.2] = -1
            slots[0] = -2 ** 31
        joint = randn((T, H, dk + dv), dtype, T)
        k, v = joint[..., :dk], joint[..., dk:]
        a, b = np64(kc), np64(vc)
        gdn.paged_write(k, v, kc, vc, i32(slots))
        paged.write(a, np64(k), slots)
        paged.write(b, np64(v), slots)
        assert np.array_equal(np64(kc), a) and np.array_equal(np64(vc), b)
    assert gdn.device_status() == gdn.OK


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("T,H,Hk,dk,dv,r", [(1, 8, 2, 128, 128, 128), (70, 5, 1, 64, 128, 32), (9, 16, 4, 256, 256, 64),
                                            (400, 40, 8, 96, 64, 96), (3, 0, 2, 64, 64, 64), (4, 3, 2, 64, 64, 0)])
def test_rotary_write_is_rotary_and_write(dtype, neighbours, T, H, Hk, dk, dv, r):
    """The same bits as the two calls, axes and skipped slots among them."""
    q, k, v = (randn((T, h, d), dtype, s) for h, d, s in ((H, dk, 1), (Hk, dk, 2), (Hk, dv, 3)))
    n = r // 2
    plan = gdn.rotary_plan(r, sections=[n // 4, n - n // 4], neighbours=neighbours)
    pos = i32(np.random.default_rng(T).integers(0, 10 ** 6, (2, T)))
    slots = torch.randperm(32 * 16, device="cuda")[:T].to(torch.int32)
    slots[T // 2] = -1
    caches = [pages("heads", 32, Hk, 16, dk, dv, dtype) for _ in range(2)]
    want, turned = gdn.rotary(q, k, pos, plan)
    gdn.paged_write(turned, v, *caches[0], slots)
    got = gdn.rotary_write(q, k, v, pos, plan, *caches[1], slots)
    assert torch.equal(got, want)
    for a, b in zip(*caches):
        assert torch.equal(a, b)
    gdn.rotary_write(q, k, v, pos, plan, *caches[1], slots, q_out=q)     # in place
    assert torch.equal(q, want) and gdn.device_status() == gdn.OK


def test_slots_outside_the_cache():
    kc, vc = pages("heads", 3, 2, 16, 64, 64, "bf16")
    k, v = randn((4, 2, 64), "bf16", 1), randn((4, 2, 64), "bf16", 2)
    gdn.paged_write(k, v, kc, vc, i32([48, 2 ** 31 - 1, -1, 47]))
    assert gdn.device_status() == gdn.ERR_PAGE
    assert torch.equal(kc[2, :, 15], k[3]) and torch.equal(vc[2, :, 15], v[3])
    kc[2, :, 15] = vc[2, :, 15] = 7.0
    assert (kc == 7).all() and (vc == 7).all()
    none = gdn.paged_cache(0, 2, 16, 64)
    gdn.paged_write(k, v, *none, i32([-1, -1, -1, -1]))
    assert gdn.device_status() == gdn.OK
    gdn.paged_write(k, v, *none, i32([-1, -1, 0, -1]))
    assert gdn.device_status() == gdn.ERR_PAGE


def test_nothing_to_do():
    plan, none = gdn.rotary_plan(64), torch.empty(0, dtype=torch.int32, device="cuda")
    q, k = randn((0, 4, 64), "bf16", 1), randn((0, 2, 64), "bf16", 1)
    a, b = gdn.rotary(q, k, none, plan)
    assert a.shape == q.shape and b.shape == k.shape
    kc, vc = pages("heads", 2, 2, 16, 64, 64, "bf16")
    gdn.rotary_write(q, k, k, none, plan, kc, vc, none)
    assert (kc == 7).all()


def test_offsets_past_32_bits():
    """Slots more than 2^32 bytes into a cache, rows more than 2^32 bytes into a tensor."""
    n_pages = 9000
    kc, vc = gdn.paged_cache(n_pages, 8, 256, 128)
    far = n_pages * 256 - 5
    k, v = randn((2, 8, 128), "bf16", 1), randn((2, 8, 128), "bf16", 2)
    gdn.paged_write(k, v, kc, vc, i32([far, 3]))
    assert torch.equal(kc[far // 256, :, far % 256], k[0]) and torch.equal(vc[0, :, 3], v[1])
    T = 600000                          # 600000 x 32 x 128 x 2 bytes = 4.9e9
    x = torch.empty((T, 32, 128), dtype=torch.bfloat16, device="cuda")
    x[-3:] = randn((3, 32, 128), "bf16", 3)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-3:] = i32([1, 2, 3])
    plan = gdn.rotary_plan(128)
    gdn.rotary(x[-3:].contiguous(), None, i32([1, 2, 3]), plan, q_out=(want := torch.empty((3, 32, 128), dtype=torch.bfloat16,
                                                                                           device="cuda")))
    gdn.rotary(x, None, pos, plan, q_out=x)
    assert torch.equal(x[-3:], want)


@pytest.mark.parametrize("packed", [False, True])
def test_a_layers_steps_captured(packed):
    """Tables, rotary positions, writes and attention as a decode loop makes them: a prompt, then steps replayed from two
    graphs that share the pool, against the oracle on all rows so far."""
    B, H, Hkv, d, page, n = 3, 8, 2, 64, 16, 37
    gen = np.random.default_rng(1)
    free, count = i32(gen.permutation(40)), i32([40])
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    kc, vc = gdn.paged_cache(40, Hkv, page, d)
    plan = gdn.rotary_plan(d)
    lens = i32([0] * B)
    rows = []

    def layer(q, k, v, new, n_new, total):
        if packed:
            slots, pos, _ = gdn.page_assign(table, lens, free, count, page, n_new, new, n_tokens=total)
        else:
            slots, pos, _ = gdn.page_assign(table, lens, free, count, page, n_new, new)
        return gdn.rotary_write(q, k, v, pos.reshape(-1), plan, kc, vc, slots.reshape(-1))

    prompt = [n, 1, 20]
    tokens = sum(prompt) if packed else B * n
    at = [(b, i) for b in range(B) for i in range(n if not packed else prompt[b])]
    q, k, v = (randn((tokens, h, d), "bf16", s) for h, s in ((H, 1), (Hkv, 2), (Hkv, 3)))
    lens.copy_(i32(prompt))
    layer(q, k, v, i32(prompt), n, tokens)
    seqs = [[(np64(k)[t], np64(v)[t]) for t, (b, i) in enumerate(at) if b == s and i < prompt[s]] for s in range(B)]
    step_q, step_k, step_v = (torch.zeros((B, h, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    graphs = []
    state = [t.clone() for t in (table, free, count, lens, kc, vc)]
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lens += 1
            turned = layer(step_q, step_k, step_v, None, 1, B)
            out = gdn.flash_attn_paged(turned.unsqueeze(2), kc, vc, table, lens)
        graphs.append((g, out))
    for t, w in zip((table, free, count, lens, kc, vc), state):
        t.copy_(w)
    for step in range(30):
        for t, s in ((step_q, 10), (step_k, 11), (step_v, 12)):
            t.copy_(randn(tuple(t.shape), "bf16", s + 100 * step))
        g, out = graphs[step % 2]
        g.replay()
        torch.cuda.synchronize()
        assert gdn.device_status() == gdn.OK
        f = freqs_of(d, 1e4)
        for b in range(B):
            seqs[b].append((np64(step_k)[b], np64(step_v)[b]))
            m = len(seqs[b])
            ks = paged.rotary(np.stack([x[0] for x in seqs[b]]), np.arange(m)[None], f, [0] * (d // 2))
            qs = paged.rotary(np64(step_q)[b:b + 1], np.array([[m - 1]]), f, [0] * (d // 2))
            ks, qs = (torch.tensor(x).bfloat16().double().numpy() for x in (ks, qs))
            vs = np.stack([x[1] for x in seqs[b]])
            from oracle.attn import attention
            ref = attention(qs[None].transpose(0, 2, 1, 3), ks.transpose(1, 0, 2)[None], vs.transpose(1, 0, 2)[None])
            # a turned element beside a border may round the other way, one in 2^12: by a step of bf16, 2^-6 of an element
            # up to 4; times a query's (key's) element up to 4 and the scale 1/8 a score is off by 2^-7, and an output
            # by a quarter of that (p (1 - p)) times the values' spread of 6
            assert np.abs(np64(out)[b] - ref[0]).max() <= 2.0 ** -7 * 1.5
