"""Oracle for pages, rotary positions and the paged cache of 16- and 32-bit rows -- TEST
INFRASTRUCTURE ONLY.  Written from the definitions, in Python integers and float64; imports nothing
from the product.

    assign: the new tokens of sequence b stand at positions len_b - n_b + i; whichever page they are
        the first to need comes off the end of the stack, sequence by sequence.
    release: pages behind the ones that stay go back, so that an assign is undone.
    rotary: each pair of elements is a complex number, times e^(i angle).
    write: row t to page slot // page_size, place slot % page_size.
    attention: oracle.attn's, on each sequence's own rows.
"""
from __future__ import annotations

import numpy as np

from .attn import attention


def assign(table, lens, new, free, page, n_new, n_tokens=None):
    """table (B, max_pages) and free (a list, the next page last) are updated; the number of pages is len(table)
    independent.  Returns (slots, positions, offsets, ok): padded lists of lists, or packed with ``n_tokens``."""
    cap = table.shape[1] * page
    ok, slots, positions, offsets = True, [], [], [0]
    for b in range(len(lens)):
        n = n_new if new is None else min(max(int(new[b]), 0), n_new)
        size = max(int(lens[b]), 0)
        ok &= size <= cap and (new is None or int(new[b]) <= n_new)
        held = -(-max(size - n, 0) // page)
        for j in range(held, -(-min(size, cap) // page)):
            if free:
                table[b, j] = free.pop()
            else:
                table[b, j] = -1
                ok = False
        s, p = [-1] * n_new, [0] * n_new
        for i in range(n):
            at = size - n + i
            if 0 <= at < cap:
                p[i] = at
                if table[b, at // page] >= 0:
                    s[i] = int(table[b, at // page]) * page + at % page
                else:
                    ok = False           # a page that the sequence should hold already, or one that there was not
        offsets.append(offsets[-1] + n)
        slots.append(s if n_tokens is None else s[:n])
        positions.append(p if n_tokens is None else p[:n])
    if n_tokens is not None:
        slots, positions = sum(slots, []), sum(positions, [])
        ok &= len(slots) <= n_tokens
        slots = (slots + [-1] * n_tokens)[:n_tokens]
        positions = (positions + [0] * n_tokens)[:n_tokens]
    return slots, positions, offsets, ok


def release(table, before, after, free, page, n_pages):
    """The stack ``free`` (a list) after sequences shrink; (free, ok)."""
    cap = table.shape[1] * page
    back, ok = [], True
    for b in range(len(before)):
        ok &= before[b] <= cap
        hi = -(-min(max(int(before[b]), 0), cap) // page)
        lo = 0 if after is None else -(-min(max(int(after[b]), 0), cap) // page)
        for j in range(lo, hi):
            if 0 <= table[b, j] < n_pages:
                back.append(int(table[b, j]))
            else:
                ok = False
    out = free + back[::-1]
    return out[:n_pages], ok and len(out) <= n_pages


def rotary(x, positions, freqs, axes, neighbours=False, inverse=False):
    """x (T, H, d) float64; positions (axes, T); freqs, axes (r / 2)."""
    x = np.array(x, dtype=np.float64)
    r = 2 * len(freqs)
    turns = positions[np.asarray(axes, dtype=int)].astype(np.float64).T * np.asarray(freqs, dtype=np.float64)
    z = np.exp((-1j if inverse else 1j) * turns)[:, None]
    a, b = (slice(0, r, 2), slice(1, r, 2)) if neighbours else (slice(0, r // 2), slice(r // 2, r))
    w = (x[..., a] + 1j * x[..., b]) * z
    x[..., a], x[..., b] = w.real, w.imag
    return x


def write(cache, rows, slots):
    """cache (n_pages, H, page, d) is updated from rows (T, H, d)."""
    page = cache.shape[2]
    for t, s in enumerate(slots):
        if 0 <= s < cache.shape[0] * page:
            cache[s // page, :, s % page] = rows[t]


def attend(q, k_cache, v_cache, table, lens, mask=None, scale=None, causal=False):
    """q (B, H, n_q, dk); returns (B, n_q, H, dv).  Tokens that no row sees are left out, so they may hold anything."""
    B, H, n_q, _ = q.shape
    Hkv, page, dv = v_cache.shape[1:]
    out = np.zeros((B, n_q, H, dv))
    cap = table.shape[1] * page
    for b in range(B):
        raw = max(int(lens[b]), 0)
        n = min(raw, cap)
        used = table[b, :-(-n // page)].astype(int)
        there = np.repeat((used >= 0) & (used < k_cache.shape[0]), page)[:n]
        if not there.any():
            continue
        k, v = (c[np.where((used >= 0) & (used < len(c)), used, 0)].transpose(1, 0, 2, 3).reshape(Hkv, -1, c.shape[3])[:, :n]
                for c in (k_cache, v_cache))
        for i in range(n_q):
            sees = there.copy()
            if causal:
                sees &= np.arange(n) <= raw - n_q + i
            m = np.zeros(n) if mask is None else np.asarray(mask[b, 0, i, :n], dtype=np.float64)
            sees &= m != -np.inf
            if sees.any():
                out[b:b + 1, i:i + 1] = attention(q[b:b + 1, :, i:i + 1], k[None][:, :, sees], v[None][:, :, sees],
                                                 m[sees][None, None, None], scale)
    return out
