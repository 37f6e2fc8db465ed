"""Workloads of the 4-bit key / value cache: writing it, reading it back, and decode attention over it.

``run`` computes each operator with elementary torch operations where ``own``
is false and through this package's entry points where it is true.

The cache holds, for every (sequence, kv head, token), a key row of ``dk`` and
a value row of ``dv`` numbers in 4 bits.  Sixteen neighbouring elements of a
row share a scale s, and element x is kept as the nearest of
+-{0, 0.5, 1, 1.5, 2, 3, 4, 6} to x / s (ties to the even code, larger values
to 6).  s is max|x| / 6 rounded to a significand of 4 bits (ties to even),
least step 2^-17, at most 10240.

Sixteen tokens of one kv head make a tile of 9 (dk + dv) bytes; pages of
``page`` tokens hold page / 16 tiles a head; a sequence finds its pages
through a page table.  The bytes of a tile, with nibbles low half first:
  keys    [dk / 128 or 1][16 tokens][bytes of that part of the row, in order]
  scales  [dk / 128 or 1][16 tokens][groups of that part]
  values  [dv / 64][8 g][4 t][4 w][4 b], nibble n: token 4t + 2(b / 2) + n and
          element 128 c + L g + 8 r + 2w + b % 2, where L = min(16, dv / 8) and
          c, r the quotient and remainder of the first index by 2
  scales  [dv / 16 groups][16 tokens]
A scale byte is bits 7 to 14 of the scale as a 16-bit float.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases

def listed():
    attn = dict(op="attn", n_q=1, dk=128, dv=128, page=64, dtype="bf16", out="f32", ragged=False,
                causal=False, mask=False)
    write = dict(op="write", new=1, dk=128, dv=128, page=64, dtype="bf16", ragged=False)
    read = dict(op="read", dk=128, dv=128, page=64, dtype="bf16", ragged=False)
    return [
        # one user's decode step on a short context: latency only
        dict(attn, name="attn_b1_h16_kv4_n141_d256", B=1, H=16, Hkv=4, n=141, dk=256, dv=256),
        # a serving batch's decode step: the cache streams from memory
        dict(attn, name="attn_b64_h32_kv8_n4096_d128", B=64, H=32, Hkv=8, n=4096),
        # two users on long contexts of unequal length, few heads to spread over the GPU
        dict(attn, name="attn_b2_h16_kv4_n100003_d128", B=2, H=16, Hkv=4, n=100003, page=256,
             ragged=True, out="bf16"),
        # drafted tokens checked together: five queries a sequence, each sees up to its own token
        dict(attn, name="attn_b16_h32_kv8_q5_n5001_d128_f16", B=16, H=32, Hkv=8, n=5001, n_q=5,
             page=16, dtype="f16", ragged=True, causal=True),
        # 32-bit queries, unequal widths and an additive mask
        dict(attn, name="attn_b3_h8_kv2_q3_n1000_d64_256_f32", B=3, H=8, Hkv=2, n=1000, n_q=3, dk=64,
             dv=256, page=32, dtype="f32", mask=True),
        # the same decode step's new token of every sequence
        dict(write, name="write_b64_kv8_d128_t1", B=64, Hkv=8, n=4096, ragged=True),
        # a long prompt's keys and values
        dict(write, name="write_b8_kv8_d128_t16384", B=8, Hkv=8, n=16384, new=16384),
        # prompts of unequal length behind what is there already, 32-bit rows
        dict(write, name="write_b5_kv3_d64_256_t301_f32", B=5, Hkv=3, n=777, new=301, dk=64, dv=256,
             page=16, dtype="f32", ragged=True),
        # one sequence's cache handed to an operator that wants dense keys and values
        dict(read, name="read_b1_kv4_n512_d256", B=1, Hkv=4, n=512, dk=256, dv=256),
        # a batch's whole cache
        dict(read, name="read_b32_kv8_n4096_d128", B=32, Hkv=8, n=4096, ragged=True, dtype="f16"),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["attn", "attn", "write", "read"])
    c = dict(op=op, Hkv=rng.choice([1, 2, 3, 4, 8]), dk=rng.choice([64, 128, 256]),
             page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=rng.choice(list(DTYPES)),
             ragged=rng.random() < 0.6)
    c["dv"] = c["dk"] if rng.random() < 0.7 else rng.choice([64, 128, 256])
    c["B"] = log(1, 64)
    c["n"] = log(1, 130000)
    rows = 1
    if op == "attn":
        c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 8])
        c["n_q"] = 1 if rng.random() < 0.6 else rng.randint(2, 19)
        c["out"] = "f32" if c["dtype"] == "f32" else rng.choice(["f32", c["dtype"]])
        c["causal"] = rng.random() < 0.5
        c["mask"] = rng.random() < 0.3
        rows = c["H"] // c["Hkv"] * c["n_q"]
    # at most what the largest listed case of the operator has
    most = {"attn": 64 * 8 * 4096 * 256, "write": 8 * 8 * 16384 * 256, "read": 32 * 8 * 4096 * 256}[op]
    each = c["B"] * c["Hkv"] * (c["dk"] + c["dv"]) * max(1.0, rows / 8)
    c["n"] = max(1, min(c["n"], int(most / each)))
    if op == "write":
        c["new"] = 1 if rng.random() < 0.4 else log(1, c["n"])
    return c


def _lens(case):
    """Tokens of each sequence, by the case alone: unequal ones spread from n down to about n / B."""
    B, n = case["B"], case["n"]
    return [max(1, n * ((b * 7) % B + 1) // B) if case["ragged"] else n for b in range(B)]


def _new(case):
    """New tokens of each sequence in a write: at most what it holds, and of unequal number where it is ragged."""
    most = case["new"]
    return [min(len_, most if most == 1 or not case["ragged"] else max(1, most - b * most // (2 * case["B"])))
            for b, len_ in enumerate(_lens(case))]


# ---------------------------------------------------------------- the format, in torch operations

def _split(x):
    """Codes (0 to 15), scale bytes and the values that they stand for, of x (..., d) in 32 bits."""
    x = x.float()
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    t = g.abs().amax(-1).double() / 6                       # exact to far beyond a step
    _, e = torch.frexp(t)
    power = torch.tensor([2.0 ** i for i in range(-17, 13)], dtype=torch.float64, device=x.device)
    step = power[torch.clamp(e - 1, -14, 15).long() + 14]
    s = torch.clamp(torch.round(t / step) * step, max=10240.0).float()
    a, u = g.abs(), s.unsqueeze(-1)
    code = torch.zeros_like(a, dtype=torch.uint8)
    # the borders between neighbouring values times s are exact in 32 bits; at a border the even code
    for i, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= m * u) if i % 2 else (a > m * u)
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    code = torch.where(u > 0, code, torch.zeros_like(code))
    value = torch.where(torch.signbit(g), -1.0, 1.0) * level[code.long()] * u
    byte = (s.half().view(torch.int16) >> 7).to(torch.uint8)
    return (code + 8 * torch.signbit(g)).to(torch.uint8).reshape(x.shape), byte, value.reshape(x.shape)


def _shape(d):
    """The first two extents of a tile's key part and its value part's order for width d."""
    return max(1, d // 128), d // 64


def _pack_keys(code, byte):
    """(..., 16, d) codes and (..., 16, d / 16) scale bytes -> the key bytes of a tile."""
    d, lead = code.shape[-1], code.shape[:-2]
    c, _ = _shape(d)
    b = code[..., 0::2] | (code[..., 1::2] << 4)
    b = b.reshape(*lead, 16, c, d // 2 // c).transpose(-3, -2).reshape(*lead, 8 * d)
    s = byte.reshape(*lead, 16, c, d // 16 // c).transpose(-3, -2).reshape(*lead, d)
    return torch.cat([b, s], -1)


def _unpack_keys(tile, d):
    lead = tile.shape[:-1]
    c, _ = _shape(d)
    b = tile[..., :8 * d].reshape(*lead, c, 16, d // 2 // c).transpose(-3, -2).reshape(*lead, 16, d // 2)
    code = torch.stack([b & 15, b >> 4], -1).reshape(*lead, 16, d)
    byte = tile[..., 8 * d:].reshape(*lead, c, 16, d // 16 // c).transpose(-3, -2)
    return code, byte.reshape(*lead, 16, d // 16)


def _pack_values(code, byte):
    d, lead = code.shape[-1], code.shape[:-2]
    q = d // 64
    c, r = (q + 1) // 2, min(q, 2)
    # tokens (t, pair, n), elements (c, g, r, w, half)
    x = code.reshape(*lead, 4, 2, 2, c, 8, r, 4, 2)
    x = x[..., 0, :, :, :, :, :] | (x[..., 1, :, :, :, :, :] << 4)      # t, pair, c, g, r, w, half
    k = len(lead)
    order = list(range(k)) + [k + i for i in (2, 4, 3, 0, 5, 1, 6)]      # c, r, g, t, w, pair, half
    return torch.cat([x.permute(order).reshape(*lead, 8 * d), byte.transpose(-2, -1).reshape(*lead, d)], -1)


def _unpack_values(tile, d):
    lead = tile.shape[:-1]
    q = d // 64
    c, r = (q + 1) // 2, min(q, 2)
    k = len(lead)
    x = tile[..., :8 * d].reshape(*lead, c, r, 8, 4, 4, 2, 2)            # c, r, g, t, w, pair, half
    x = x.permute(list(range(k)) + [k + i for i in (3, 5, 0, 2, 1, 4, 6)])  # t, pair, c, g, r, w, half
    code = torch.stack([x & 15, x >> 4], k + 2).reshape(*lead, 16, d)
    return code, tile[..., 8 * d:].reshape(*lead, d // 16, 16).transpose(-2, -1)


def _dense(code, byte):
    """The 32-bit values of codes (..., d) under scale bytes (..., d / 16)."""
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=code.device)
    level = torch.cat([level, -level])
    s = (byte.to(torch.int16) << 7).view(torch.float16).float()
    return (level[code.long()].reshape(*byte.shape, 16) * s.unsqueeze(-1)).reshape(code.shape)


# ---------------------------------------------------------------- inputs

def _rows(shape, dtype, gen, spread):
    """Rows as projections give them: normal, with some channels louder than others where `spread`."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if spread:
        x *= torch.exp(0.5 * torch.randn((1, shape[1], 1, shape[3]), generator=gen, device="cuda"))
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    """The cache, its table and lengths, as a serving program holds them, and this step's rows or queries."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    B, Hkv, n, dk, dv, page = (case[k] for k in ("B", "Hkv", "n", "dk", "dv", "page"))
    lens = _lens(case)
    pages = -(-n // page)
    table = torch.randperm(B * pages + 3, generator=gen, device="cuda")[:B * pages].to(torch.int32)
    table = table.reshape(B, pages).contiguous()
    state = dict(case=dict(case), table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    cache = torch.zeros((B * pages + 3, Hkv, page // 16, 9 * (dk + dv)), dtype=torch.uint8, device="cuda")
    held = "bf16" if case["dtype"] == "f32" and case["op"] == "attn" else case["dtype"]
    for b in range(B):  # a sequence at a time, for the room that the parts take
        m = pages * page
        tiles = torch.empty((Hkv, m // 16, 9 * (dk + dv)), dtype=torch.uint8, device="cuda")
        for w, lo, pack, spread in ((dk, 0, _pack_keys, True), (dv, 9 * dk, _pack_values, False)):
            code, byte, _ = _split(_rows((1, Hkv, m, w), held, gen, spread)[0])
            tiles[..., lo:lo + 9 * w] = pack(code.reshape(Hkv, m // 16, 16, w),
                                            byte.reshape(Hkv, m // 16, 16, w // 16))
        cache[table[b].long()] = tiles.reshape(Hkv, pages, page // 16, -1).transpose(0, 1)
    state["cache"] = cache
    if case["op"] == "attn":
        dt = DTYPES[case["dtype"]]
        state["q"] = torch.randn((B, case["H"], case["n_q"], dk), generator=gen, device="cuda").to(dt)
        state["mask"] = None
        if case["mask"]:
            shape = (B, 1, case["n_q"], pages * page)
            m = torch.randn(shape, generator=gen, device="cuda") * 0.5
            m[torch.rand(shape, generator=gen, device="cuda") < 0.1] = -math.inf
            state["mask"] = m.to(dt)
    elif case["op"] == "write":
        # the projections' own order: tokens before heads
        for name, w, spread in (("k", dk, True), ("v", dv, False)):
            x = _rows((B, Hkv, case["new"], w), case["dtype"], gen, spread)
            state[name] = x.transpose(1, 2).contiguous().transpose(1, 2)
        state["new"] = torch.tensor(_new(case), dtype=torch.int32, device="cuda")
    return state


# ---------------------------------------------------------------- the operators

def run(state):
    return {"attn": _attn, "write": _write, "read": _read}[state["case"]["op"]](state)


def _attn(state):
    case = state["case"]
    dk, dv, dt = case["dk"], case["dv"], DTYPES[case["out"]]
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        return gdn.flash_attn_kv4(state["q"], state["cache"], state["table"], state["lens"], dv,
                                  state["mask"], causal=case["causal"], out_dtype=dt)
    q, lens = state["q"], state["lens"]
    B, H, n_q, _ = q.shape
    Hkv = case["Hkv"]
    t = state["cache"][state["table"].long()].transpose(1, 2)                 # (B, Hkv, pages, tiles, bytes)
    t = t.reshape(B, Hkv, -1, t.shape[-1])
    k = _dense(*_unpack_keys(t[..., :9 * dk], dk)).reshape(B, Hkv, -1, dk)
    v = _dense(*_unpack_values(t[..., 9 * dk:], dv)).reshape(B, Hkv, -1, dv)
    m = k.shape[2]
    s = q.float().reshape(B, Hkv, H // Hkv * n_q, dk) @ k.transpose(2, 3)
    s = s.reshape(B, Hkv, H // Hkv, n_q, m) * (1.0 / math.sqrt(dk))
    if state["mask"] is not None:
        s = s + state["mask"].float().reshape(B, 1, 1, n_q, m)
    sees = lens.reshape(B, 1, 1)
    if case["causal"]:
        sees = sees - (n_q - 1) + torch.arange(n_q, device=q.device).reshape(1, n_q, 1)
    hidden = torch.arange(m, device=q.device).reshape(1, 1, m) >= sees
    s = s.masked_fill(hidden.reshape(B, 1, 1, -1, m), -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, m) @ v).reshape(B, H, n_q, dv)
    o = torch.where(total.reshape(B, H, n_q, 1) > 0, o / total.reshape(B, H, n_q, 1), torch.zeros_like(o))
    return o.transpose(1, 2).contiguous().to(dt)


def _write(state):
    """Writes the new rows and reads the same positions back: what later steps will see of them."""
    case, k, v = state["case"], state["k"], state["v"]
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        gdn.kv4_write(k, v, state["cache"], state["table"], state["lens"], state["new"])
        return gdn.kv4_read(state["cache"], state["table"], state["lens"], k.shape[2], case["dk"],
                            case["dv"], lens=state["new"], dtype=k.dtype)
    B, Hkv, T, _ = k.shape
    dk, dv = case["dk"], case["dv"]
    new = state["new"].long()
    first = state["lens"].long() - new
    tile, where = _where(state, first, T)
    n_t = tile.shape[1]
    place = tile.unsqueeze(-1) * 16 + torch.arange(16, device=k.device)       # (B, n_t, 16)
    i = place - first.reshape(B, 1, 1)                       # the new token at each place
    fresh = (i >= 0) & (i < new.reshape(B, 1, 1))
    i = i.clamp(0, T - 1).reshape(B, 1, n_t * 16, 1)
    touched = fresh.any(-1)
    old = state["cache"][where[0], :, where[1]].transpose(1, 2)               # (B, Hkv, n_t, bytes)
    parts = []
    for x, w, lo, pack, unpack in ((k, dk, 0, _pack_keys, _unpack_keys),
                                   (v, dv, 9 * dk, _pack_values, _unpack_values)):
        code, byte, _ = _split(x)
        code = torch.gather(code, 2, i.expand(-1, Hkv, -1, w)).reshape(B, Hkv, n_t, 16, w)
        byte = torch.gather(byte, 2, i.expand(-1, Hkv, -1, w // 16)).reshape(B, Hkv, n_t, 16, w // 16)
        was = unpack(old[..., lo:lo + 9 * w], w)
        f = fresh.reshape(B, 1, n_t, 16, 1)
        parts.append(pack(torch.where(f, code, was[0]), torch.where(f, byte, was[1])))
    tiles = torch.cat(parts, -1).transpose(1, 2)             # (B, n_t, Hkv, bytes)
    state["cache"][where[0][touched], :, where[1][touched]] = tiles[touched]
    return _back(state, T, new, k.dtype)


def _read(state):
    case = state["case"]
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        return gdn.kv4_read(state["cache"], state["table"], state["lens"], case["n"], case["dk"],
                            case["dv"], lens=state["lens"], dtype=DTYPES[case["dtype"]])
    return _back(state, case["n"], state["lens"].long(), DTYPES[case["dtype"]])


def _where(state, first, T):
    """The tiles that T tokens from first[b] on can touch, and their pages and places in them: (B, tiles) each."""
    page, table = state["case"]["page"], state["table"]
    tile = (first // 16).reshape(-1, 1) + torch.arange((T + 30) // 16, device=first.device)
    at = torch.clamp(tile * 16 // page, max=table.shape[1] - 1)
    return tile, (torch.gather(table.long(), 1, at), tile % (page // 16))


def _back(state, T, count, dtype):
    """The last count[b] tokens of each sequence, dense in (B, Hkv, T, d), zeros behind them."""
    case, B = state["case"], state["lens"].shape[0]
    first = state["lens"].long() - count
    _, where = _where(state, first, T)
    t = state["cache"][where[0], :, where[1]].transpose(1, 2)
    i = torch.arange(T, device=t.device).reshape(1, T)
    held = (i < count.reshape(B, 1)).reshape(B, 1, T, 1)
    at = ((first % 16).reshape(B, 1) + i).reshape(B, 1, T, 1)
    out = []
    for w, lo, unpack in ((case["dk"], 0, _unpack_keys), (case["dv"], 9 * case["dk"], _unpack_values)):
        code, byte = unpack(t[..., lo:lo + 9 * w], w)
        code = torch.gather(code.reshape(B, case["Hkv"], -1, w), 2, at.expand(-1, case["Hkv"], -1, w))
        byte = torch.gather(byte.reshape(B, case["Hkv"], -1, w // 16), 2,
                            at.expand(-1, case["Hkv"], -1, w // 16))
        x = _dense(code, byte)
        out.append(torch.where(held, x, torch.zeros_like(x)).to(dtype))
    return tuple(out)


def work(case):
    B, Hkv, dk, dv = case["B"], case["Hkv"], case["dk"], case["dv"]
    width = {"f32": 4, "bf16": 2, "f16": 2}
    e = width[case["dtype"]]
    tokens = sum(_lens(case))
    if case["op"] == "attn":
        rows = B * case["H"] * case["n_q"]
        size = Hkv * tokens * (dk + dv) * 9 / 16 + rows * (dk * e + dv * width[case["out"]])
        if case["mask"]:
            size += case["n_q"] * tokens * e
        return {"bytes": size, "flops": 2 * tokens * case["H"] * case["n_q"] * (dk + dv)}
    if case["op"] == "write":  # rows in, cache out, and back again: cache in, every output row written
        new, rows = sum(_new(case)), B * case["new"]
        return {"bytes": Hkv * (dk + dv) * (new * (e + 9 / 8) + rows * e), "flops": new * Hkv * (dk + dv) * 4}
    return {"bytes": Hkv * (dk + dv) * (tokens * 9 / 16 + B * case["n"] * e),
            "flops": tokens * Hkv * (dk + dv)}


# ---------------------------------------------------------------- from the definition, in 64 bits

def _table(device):
    """Every scale there is, in order, and the nearest-value borders."""
    s = np.array([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 18) for e in range(31) for m in range(8)])
    return torch.tensor(s[s <= 10240], dtype=torch.float64, device=device)


def _nearest(x, values):
    """Index of the nearest of the sorted `values`, the even one of two as near."""
    mid = (values[1:] + values[:-1]) / 2
    lo, hi = torch.searchsorted(mid, x, right=False), torch.searchsorted(mid, x, right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def _kept(x):
    """What the format keeps of the rows x (..., d), in 64 bits."""
    g = x.double().reshape(-1, 16)
    scales = _table(x.device)
    s = scales[_nearest(g.abs().amax(1) / 6, scales)].unsqueeze(1)
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    r = torch.where(s > 0, g.abs() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    return (torch.sign(g) * level[_nearest(r, level)] * s).reshape(x.shape)


def _tile_rows(tiles, dk, dv):
    """Keys (16 m, dk) and values (16 m, dv) of tiles (m, bytes), element by element from the layout's description."""
    dev = tiles.device
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                         device=dev)
    power = torch.tensor([2.0 ** (i - 18) for i in range(32)], dtype=torch.float64, device=dev)
    tok = torch.arange(16, device=dev).unsqueeze(1)
    x = torch.arange(dk, device=dev).unsqueeze(0)
    part = min(dk, 128)
    byte = (x // part) * 8 * part + tok * (part // 2) + x % part // 2
    scale = 8 * dk + (x // part) * part + tok * (part // 16) + x % part // 16
    nib = (x % 2).expand(16, -1)
    rows = []
    for w, base in ((dk, 0), (dv, 9 * dk)):
        if base:
            x = torch.arange(w, device=dev).unsqueeze(0)
            L = min(16, w // 8)
            y = x % 128
            g, z = y // L, y % L
            first = 2 * (x // 128) + z // 8
            byte = (((first * 8 + g) * 4 + tok // 4) * 4 + z % 8 // 2) * 4 + 2 * (tok % 4 // 2) + z % 2
            scale = 8 * w + (x // 16) * 16 + tok
            nib = (tok % 2).expand(-1, w)
        code = (tiles[:, base + byte.reshape(-1)].int() >> (4 * nib.reshape(-1))) & 15
        s = tiles[:, base + scale.reshape(-1)].int()
        ex, man = s >> 3, s & 7
        sv = torch.where(ex == 0, man, man + 8).double() * power[ex.clamp(min=1).long()]
        rows.append((level[code.long()] * sv).reshape(-1, w))
    return rows


def exact(case, seed):
    state = prepare(case, seed)
    B, Hkv, dk, dv, page = (case[k] for k in ("B", "Hkv", "dk", "dv", "page"))
    lens = _lens(case)
    if case["op"] == "write":
        out = []
        for x in (state["k"], state["v"]):
            y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
            for b, m in enumerate(_new(case)):
                y[b, :, :m] = _kept(x[b, :, :m])
            out.append(y)
        return tuple(out)
    if case["op"] == "read":
        k = torch.zeros((B, Hkv, case["n"], dk), dtype=torch.float64, device="cuda")
        v = torch.zeros((B, Hkv, case["n"], dv), dtype=torch.float64, device="cuda")
    else:
        H, n_q = case["H"], case["n_q"]
        out = torch.zeros((B, n_q, H, dv), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b]
        used = state["cache"][state["table"][b, :-(-n // page)].long()]
        for h in range(Hkv):
            kr, vr = _tile_rows(used[:, h].reshape(-1, used.shape[-1])[:-(-n // 16)], dk, dv)
            kr, vr = kr[:n], vr[:n]
            if case["op"] == "read":
                k[b, h, :n], v[b, h, :n] = kr, vr
                continue
            rep = H // Hkv
            for i in range(n_q):
                seen = n - (n_q - 1) + i if case["causal"] else n
                if seen <= 0:
                    continue
                s = state["q"][b, h * rep:(h + 1) * rep, i].double() @ kr[:seen].T / math.sqrt(dk)
                if state["mask"] is not None:
                    s = s + state["mask"][b, 0, i, :seen].double()
                p = torch.softmax(s, 1)
                out[b, i, h * rep:(h + 1) * rep] = torch.nan_to_num(p) @ vr[:seen]
    return (k, v) if case["op"] == "read" else out
