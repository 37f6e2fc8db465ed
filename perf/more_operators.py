"""Workloads of a decode step's way through a paged key / value cache of 16- or 32-bit rows: page tables and slot maps
made from the sequences' lengths, rotary positions with several axes, rows written into pages, and decode attention
over the pages.

``run`` computes each operator with elementary torch operations where ``own``
is false and through this package's entry points where it is true.

Keys lie in k_cache (n_pages, n_heads_kv, page, dk), values in v_cache (n_pages,
n_heads_kv, page, dv).  Position p of sequence b stands in page table[b][p // page] at p % page;
its slot is table[b][p // page] * page + p % page.  Pages that nobody holds lie on a stack: the
first `count` entries of `free`, the next one to be given away last.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WIDTH = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- the cases

def listed():
    attn = dict(op="attn", n_q=1, dk=128, dv=128, page=64, dtype="bf16", out="f32", ragged=False,
                causal=False, mask=False, token_major=False)
    rot = dict(op="rotary", H=32, Hkv=8, d=128, r=128, base=1e4, sections="64", dealt=False, pairs="halves",
               inverse=False, dtype="bf16", far=0)
    tables = dict(op="tables", page=16, new=1, ragged=True)
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
             page=16, dtype="f16", ragged=True, causal=True, token_major=True),
        # 32-bit rows, unequal widths and an additive mask
        dict(attn, name="attn_b3_h8_kv2_q3_n1000_d64_256_f32", B=3, H=8, Hkv=2, n=1000, n_q=3, dk=64,
             dv=256, page=32, dtype="f32", mask=True),
        # a serving batch's decode step: a new page for some sequences, a slot for every new token
        dict(tables, name="tables_b64_t1", B=64, n=4096),
        # a batch of prompts of unequal length, admitted together
        dict(tables, name="tables_b256_t4096", B=256, n=8192, new=4096),
        # queries and keys of a decode step's new tokens
        dict(rot, name="rotary_t64_h32_kv8_d128", T=64, far=4096),
        # a prompt of text and images: time, height and width share the frequencies
        dict(rot, name="rotary_t16384_h32_kv8_d128_3axes", T=16384, sections="16 24 24", dealt=True),
        # training: the gradient of a layer that turns the first quarter of wide heads
        dict(rot, name="rotary_back_t5001_h16_kv4_d256_r64_f32", T=5001, H=16, Hkv=4, d=256, r=64, sections="32",
             base=1e7, pairs="neighbours", inverse=True, dtype="f32"),
        # a decode step's new tokens: queries and keys turned, keys and values into their pages
        dict(rot, name="step_t64_h32_kv8_d128", op="step", T=64, page=64, pages=256, far=4096),
        # a long prompt's keys and values into their pages
        dict(op="write", name="write_t131072_kv8_d128", T=131072, Hkv=8, dk=128, dv=128, page=64, pages=2050,
             dtype="bf16", holes=0.0),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["attn", "attn", "attn", "tables", "rotary", "step", "write"])
    c = dict(op=op, page=rng.choice([16, 32, 48, 64, 128, 256]))
    if op == "tables":
        c["page"] = rng.choice([1, 5, 16, 16, 64, 256])
        c["B"], c["n"], c["ragged"] = log(1, 1024), log(1, 8192), rng.random() < 0.7
        c["new"] = 1 if rng.random() < 0.4 else log(1, c["n"])
        # at most the largest listed case's tokens, new and held
        c["n"] = max(1, min(c["n"], 256 * 8192 // c["B"]))
        c["new"] = max(1, min(c["new"], c["n"], 256 * 4096 // c["B"]))
        return c
    c["dtype"] = rng.choice(list(DTYPES))
    if op == "attn":
        c["B"], c["n"], c["Hkv"] = log(1, 64), log(1, 130000), rng.choice([1, 2, 3, 4, 8])
        c["dk"] = rng.choice([64, 128, 256])
        c["dv"] = c["dk"] if rng.random() < 0.7 else rng.choice([64, 128, 256])
        c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 8])
        c["n_q"] = 1 if rng.random() < 0.6 else rng.randint(2, 19)
        c["out"] = "f32" if c["dtype"] == "f32" else rng.choice(["f32", c["dtype"]])
        c["ragged"], c["causal"], c["mask"] = rng.random() < 0.6, rng.random() < 0.5, rng.random() < 0.3
        c["token_major"] = rng.random() < 0.4
        # at most what the largest listed case has
        rows = c["H"] // c["Hkv"] * c["n_q"]
        each = c["B"] * c["Hkv"] * (c["dk"] + c["dv"]) * WIDTH[c["dtype"]] * max(1.0, rows / 8)
        c["n"] = max(1, min(c["n"], int(64 * 8 * 4096 * 512 / each)))
        return c
    c["Hkv"], c["T"] = rng.choice([1, 2, 3, 4, 8]), log(1, 16384)
    if op == "write":
        c["T"] = log(1, 131072)
        c["dk"], c["dv"] = rng.choice([64, 96, 128, 256]), rng.choice([64, 128, 256])
        c["holes"] = rng.choice([0.0, 0.0, 0.3])
        c["T"] = min(c["T"], 131072 * 8 * 512 // (c["Hkv"] * (c["dk"] + c["dv"]) * WIDTH[c["dtype"]]))
        c["pages"] = -(-c["T"] // c["page"]) + 2
        return c
    c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 8])
    c["d"] = rng.choice([64, 96, 128, 256])
    c["r"] = rng.choice([c["d"], c["d"], c["d"] // 2, 32])
    c["pairs"] = rng.choice(["halves", "neighbours"])
    c["base"] = rng.choice([1e4, 5e5, 1e7])
    axes = rng.choice([1, 1, 2, 3, 4])
    cut = sorted(rng.randint(0, c["r"] // 2) for _ in range(axes - 1))
    c["sections"] = " ".join(str(b - a) for a, b in zip([0] + cut, cut + [c["r"] // 2]))
    c["dealt"] = rng.random() < 0.5
    c["inverse"] = op == "rotary" and rng.random() < 0.4
    c["far"] = rng.choice([0, 1000, 1000000])
    c["T"] = max(1, min(c["T"], 16384 * 40 * 256 // ((c["H"] + 2 * c["Hkv"]) * c["d"] * WIDTH[c["dtype"]])))
    if op == "step":
        c["pages"] = -(-c["T"] // c["page"]) + 2
    return c


def _lens(case):
    """Tokens of each sequence, by the case alone: unequal ones spread from n down to about n / B."""
    B, n = case["B"], case["n"]
    return [max(1, n * ((b * 7) % B + 1) // B) if case["ragged"] else n for b in range(B)]


def _new(case):
    """New tokens of each sequence: one, or as many as it has up to most, fewer of them in later sequences."""
    most, B = case["new"], case["B"]
    return [min(len_, most if most == 1 or not case["ragged"] else max(1, most - b * most // (2 * B)))
            for b, len_ in enumerate(_lens(case))]


def _sections(case):
    return [int(n) for n in case["sections"].split()]


def _axes(case):
    """The axis whose position turns each frequency: sections one after another, or dealt out in turn."""
    s = _sections(case)
    if not case["dealt"]:
        return [a for a, n in enumerate(s) for _ in range(n)]
    out = []
    while sum(s) > 0:
        for a in range(len(s)):
            if s[a] > 0:
                out.append(a)
                s[a] -= 1
    return out


# ---------------------------------------------------------------- inputs

def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(DTYPES[dtype])


def _cache(case, n_pages, Hkv, d, gen):
    """Pages with rows in them; token-major ones are a transposed view, as programs that append token rows keep them."""
    if case.get("token_major"):
        return _randn((n_pages, case["page"], Hkv, d), case["dtype"], gen).transpose(1, 2)
    return _randn((n_pages, Hkv, case["page"], d), case["dtype"], gen)


def prepare(case, seed):
    """What a serving program holds: pages, tables, lengths, the rotary frequencies; and this step's rows or queries."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, state = case["op"], dict(case=dict(case))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "attn":
        B, H, Hkv, n_q, n, page = (case[k] for k in ("B", "H", "Hkv", "n_q", "n", "page"))
        pages = -(-n // page)
        table = torch.randperm(B * pages + 3, generator=gen, device="cuda")[:B * pages].to(torch.int32)
        state.update(table=table.reshape(B, pages).contiguous(), lens=i32(_lens(case)))
        state["k_cache"] = _cache(case, B * pages + 3, Hkv, case["dk"], gen)
        state["v_cache"] = _cache(case, B * pages + 3, Hkv, case["dv"], gen)
        # the projections' own order: tokens before heads
        state["q"] = _randn((B, n_q, H, case["dk"]), case["dtype"], gen).transpose(1, 2)
        state["mask"] = None
        if case["mask"]:
            shape = (B, 1, n_q, pages * page)
            m = torch.randn(shape, generator=gen, device="cuda") * 0.5
            m[torch.rand(shape, generator=gen, device="cuda") < 0.1] = -math.inf
            state["mask"] = m.to(DTYPES[case["dtype"]])
    elif op == "tables":
        B, n, page = case["B"], case["n"], case["page"]
        lens, new = _lens(case), _new(case)
        held = [-(-(a - b) // page) for a, b in zip(lens, new)]
        most = -(-n // page) + 1
        n_pages = sum(-(-a // page) for a in lens) + 17
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
        has = torch.arange(most, device="cuda").reshape(1, -1) < i32(held).reshape(-1, 1)
        table[has] = order[:sum(held)]
        free = torch.cat([order[sum(held):], order[:sum(held)]])
        state.update(table=table, free=free, count=i32([n_pages - sum(held)]), lens=i32(lens), new=i32(new),
                     before=i32([a - b for a, b in zip(lens, new)]), total=sum(new))
    else:
        T, Hkv = case["T"], case["Hkv"]
        if op != "rotary":
            dk, dv = (case["d"],) * 2 if op == "step" else (case["dk"], case["dv"])
            n_pages, page = case["pages"], case["page"]
            slots = torch.randperm(n_pages * page, generator=gen, device="cuda")
            if op == "write":                 # tokens of a prompt lie one after another in their pages
                slots = torch.randperm(n_pages, generator=gen, device="cuda").reshape(-1, 1) * page
                slots = (slots + torch.arange(page, device="cuda")).reshape(-1)
            slots = slots[:T].to(torch.int32)
            if op == "write" and case["holes"]:
                slots[torch.rand((T,), generator=gen, device="cuda") < case["holes"]] = -1
            state.update(slots=slots, k_cache=_cache(case, n_pages, Hkv, dk, gen),
                         v_cache=_cache(case, n_pages, Hkv, dv, gen), v=_randn((T, Hkv, dv), case["dtype"], gen))
        if op == "write":
            state["k"] = _randn((T, Hkv, case["dk"]), case["dtype"], gen)
            return state
        A, r, far = len(_sections(case)), case["r"], case["far"]
        if far:                               # new tokens of sequences of any length
            pos = torch.randint(0, far, (A, T), generator=gen, device="cuda")
        else:                                 # a prompt's tokens; an image's rows and columns on the further axes
            pos = torch.arange(T, device="cuda").repeat(A, 1) // torch.tensor([[1], [64], [3], [7]][:A], device="cuda")
        state["pos"] = pos.to(torch.int32)
        j = torch.arange(r // 2, dtype=torch.float64, device="cuda")
        state.update(freqs=torch.tensor(float(case["base"]), dtype=torch.float64, device="cuda") ** (-2 * j / r),
                     axes=torch.tensor(_axes(case), dtype=torch.int64, device="cuda"),
                     q=_randn((T, case["H"], case["d"]), case["dtype"], gen),
                     k=_randn((T, Hkv, case["d"]), case["dtype"], gen))
        if own:
            import linear_attention_sequence_gated_gb300 as gdn
            state["plan"] = gdn.rotary_plan(r, case["base"], sections=_sections(case), dealt=case["dealt"],
                                            neighbours=case["pairs"] == "neighbours", device="cuda")
    return state


# ---------------------------------------------------------------- the operators

def run(state):
    return {"attn": _attn, "tables": _tables, "rotary": _rotary, "step": _step,
            "write": _write}[state["case"]["op"]](state)


def _attn(state):
    case = state["case"]
    dk, dv, dt = case["dk"], case["dv"], DTYPES[case["out"]]
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        return gdn.flash_attn_paged(state["q"], state["k_cache"], state["v_cache"], state["table"], state["lens"],
                                    state["mask"], causal=case["causal"], out_dtype=dt)
    q, lens = state["q"], state["lens"]
    B, H, n_q, _ = q.shape
    Hkv = case["Hkv"]
    at = state["table"].long()
    k = state["k_cache"][at].transpose(1, 2).reshape(B, Hkv, -1, dk).float()
    v = state["v_cache"][at].transpose(1, 2).reshape(B, Hkv, -1, dv).float()
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
    total = total.reshape(B, H, n_q, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.transpose(1, 2).contiguous().to(dt)


def _tables(state):
    """Pages and slots for a step's new tokens; then the step is called off and its pages go back on the stack."""
    page, n_new, total = state["case"]["page"], state["case"]["new"], state["total"]
    table, free, count, lens, new = (state[k] for k in ("table", "free", "count", "lens", "new"))
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        slots, positions, offsets = gdn.page_assign(table, lens, free, count, page, n_new, new, n_tokens=total)
        gdn.page_release(table, lens, free, count, page, state["before"])
        return slots, positions, offsets, table, free, count
    B, most = table.shape
    first = lens - new
    held, after = (first + page - 1) // page, (lens + page - 1) // page
    begin = torch.cumsum(after - held, 0) - (after - held)
    j = torch.arange(most, device="cuda").reshape(1, most)
    fresh = (j >= held.reshape(B, 1)) & (j < after.reshape(B, 1))
    which = count.reshape(1, 1) - 1 - (begin.reshape(B, 1) + j - held.reshape(B, 1))
    which = which.clamp(0, free.shape[0] - 1)
    table.copy_(torch.where(fresh, free[which.long()], table))
    offsets = torch.zeros((B + 1,), dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(new, 0)
    i = torch.arange(total, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(offsets[1:], i, right=True)
    pos = first[b] + i - offsets[b]
    slots = table[b, (pos // page).long()] * page + pos % page
    # the same pages back, in the opposite order: the stack is as it was
    back = torch.where(fresh, which.long(), torch.full_like(which, free.shape[0]).long())
    room = torch.cat([free, free[:1]])
    room[back.reshape(-1)] = table.reshape(-1)
    free.copy_(room[:-1])
    return slots.to(torch.int32), pos.to(torch.int32), offsets, table, free, count


def _turn(x, state, sign):
    case = state["case"]
    r = case["r"]
    angle = state["pos"].double()[state["axes"]].T * state["freqs"]           # (T, r / 2)
    c, s = torch.cos(angle).float().unsqueeze(1), sign * torch.sin(angle).float().unsqueeze(1)
    y = x.float()
    if case["pairs"] == "neighbours":
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        y = torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), y[..., r:]], -1)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        y = torch.cat([a * c - b * s, b * c + a * s, y[..., r:]], -1)
    return y.to(x.dtype)


def _rotary(state):
    inverse = state["case"]["inverse"]
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        return gdn.rotary(state["q"], state["k"], state["pos"], state["plan"], inverse=inverse)
    sign = -1.0 if inverse else 1.0
    return _turn(state["q"], state, sign), _turn(state["k"], state, sign)


def _put(cache, slots, x, page):
    """Rows x (T, Hkv, d) into their slots, those of negative slots nowhere."""
    keep = slots >= 0
    at = slots[keep].long()
    cache[at // page, :, at % page] = x[keep]


def _step(state):
    page = state["case"]["page"]
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        q = gdn.rotary_write(state["q"], state["k"], state["v"], state["pos"], state["plan"], state["k_cache"],
                             state["v_cache"], state["slots"])
        return q, state["k_cache"], state["v_cache"]
    _put(state["k_cache"], state["slots"], _turn(state["k"], state, 1.0), page)
    _put(state["v_cache"], state["slots"], state["v"], page)
    return _turn(state["q"], state, 1.0), state["k_cache"], state["v_cache"]


def _write(state):
    if own:
        import linear_attention_sequence_gated_gb300 as gdn
        return gdn.paged_write(state["k"], state["v"], state["k_cache"], state["v_cache"], state["slots"])
    page = state["case"]["page"]
    _put(state["k_cache"], state["slots"], state["k"], page)
    _put(state["v_cache"], state["slots"], state["v"], page)
    return state["k_cache"], state["v_cache"]


def work(case):
    op = case["op"]
    if op == "tables":
        page, lens, new = case["page"], _lens(case), _new(case)
        fresh = sum(-(-a // page) - -(-(a - b) // page) for a, b in zip(lens, new))
        # lengths and counts in, offsets out; a slot and a position a token; a page: off the stack, into its
        # table, from there and onto the stack again; pages that are begun already are looked up
        size = 4 * (3 * case["B"] + case["B"] + 1) + 8 * sum(new) + 16 * fresh + 4 * case["B"]
        return {"bytes": size, "flops": sum(new) * 4}
    e = WIDTH[case["dtype"]]
    if op == "attn":
        Hkv, dk, dv, tokens = case["Hkv"], case["dk"], case["dv"], sum(_lens(case))
        rows = case["B"] * case["H"] * case["n_q"]
        size = Hkv * tokens * (dk + dv) * e + rows * (dk * e + dv * WIDTH[case["out"]])
        if case["mask"]:
            size += case["n_q"] * tokens * e
        return {"bytes": size, "flops": 2 * tokens * case["H"] * case["n_q"] * (dk + dv)}
    T, Hkv = case["T"], case["Hkv"]
    if op == "write":
        return {"bytes": int(T * (1 - case["holes"]) * Hkv * (case["dk"] + case["dv"]) * 2 * e + 4 * T),
                "flops": T * (1 - case["holes"]) * Hkv * (case["dk"] + case["dv"])}
    heads, turned = case["H"] + (2 if op == "step" else 1) * Hkv, case["H"] + Hkv
    return {"bytes": T * (heads * case["d"] * 2 * e + 4 * len(_sections(case)) + (4 if op == "step" else 0)),
            "flops": T * turned * case["r"] * 3}


# ---------------------------------------------------------------- from the definition, in 64 bits

def _turned(x, case, state):
    """Each pair as a complex number, multiplied by e^(+-i angle)."""
    r, T = case["r"], case["T"]
    turn = torch.zeros((T, r // 2), dtype=torch.float64, device=x.device)
    for j, a in enumerate(_axes(case)):
        turn[:, j] = state["pos"][a].double() * math.pow(case["base"], -2.0 * j / r)
    z = torch.polar(torch.ones_like(turn), -turn if case["inverse"] else turn).unsqueeze(1)
    y = x.double().clone()
    if case["pairs"] == "neighbours":
        first, second = slice(0, r, 2), slice(1, r, 2)
    else:
        first, second = slice(0, r // 2), slice(r // 2, r)
    w = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _placed(cache, slots, rows, page):
    out = cache.double()
    for t in (slots >= 0).nonzero().reshape(-1).split(4096):
        at = slots[t].long()
        out.transpose(1, 2)[torch.div(at, page, rounding_mode="floor"), at % page] = rows[t].double()
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        page, lens, new = case["page"], _lens(case), _new(case)
        table, free, count = state["table"].tolist(), state["free"].tolist(), int(state["count"])
        slots, positions, offsets = [], [], [0]
        for b, (a, n) in enumerate(zip(lens, new)):
            for p in range(a - n, a):
                if p % page == 0:
                    count -= 1
                    table[b][p // page] = free[count]
                positions.append(p)
                slots.append(table[b][p // page] * page + p % page)
            offsets.append(offsets[-1] + n)
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return t(slots), t(positions), t(offsets), t(table), state["free"], state["count"]
    if op == "rotary":
        return _turned(state["q"], case, state), _turned(state["k"], case, state)
    if op == "step":
        return (_turned(state["q"], case, state),
                _placed(state["k_cache"], state["slots"], _turned(state["k"], case, state), case["page"]),
                _placed(state["v_cache"], state["slots"], state["v"], case["page"]))
    if op == "write":
        return tuple(_placed(state[x + "_cache"], state["slots"], state[x], case["page"]) for x in "kv")
    H, Hkv, n_q, dv, page = (case[k] for k in ("H", "Hkv", "n_q", "dv", "page"))
    rep = H // Hkv
    out = torch.zeros((case["B"], n_q, H, dv), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        used = state["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            k = state["k_cache"][used, h].reshape(-1, case["dk"])[:n].double()
            v = state["v_cache"][used, h].reshape(-1, dv)[:n].double()
            for i in range(n_q):
                seen = n - (n_q - 1) + i if case["causal"] else n
                if seen <= 0:
                    continue
                s = state["q"][b, h * rep:(h + 1) * rep, i].double() @ k[:seen].T / math.sqrt(case["dk"])
                if state["mask"] is not None:
                    s = s + state["mask"][b, 0, i, :seen].double()
                out[b, i, h * rep:(h + 1) * rep] = torch.nan_to_num(torch.softmax(s, 1)) @ v[:seen]
    return out
