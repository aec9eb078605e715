"""Plain fp64 numpy oracle of the paged 8-bit key/value cache (test infrastructure only).

The cache is a dict of numpy arrays: k, v (layers, pages, kv_heads, page, head_dim) uint8 e4m3 codes;
k_scale, v_scale (layers, pages, kv_heads); table (seqs, max_pages), lengths, refcount.  Each function
changes it in place by the definition in include/tp_mlp.h, one entry and one page at a time, and
returns the status flags it would raise.
"""
from __future__ import annotations

import math

import numpy as np

BAD_SEQUENCE, BAD_LENGTH, BAD_PAGE, NO_PAGES, SHARED_PAGE = 1, 2, 4, 8, 16


def _table():
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = float("nan") if (b & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = -x if b >> 7 else x
    return out


VALUES = _table()                                  # the number of each code
_POS = VALUES[:127]                                # ascending, 0 .. 448


def encode(x):
    """The code of the nearest e4m3 number (ties to the even code; beyond 448: 448; NaN: 0x7f)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(_POS[hi] == a, hi, code).astype(np.uint8)
    code = np.where(np.isnan(x), 127, code).astype(np.uint8)
    return np.where(np.signbit(x), code | 128, code).astype(np.uint8)


def step_of(x):
    """The scale of rows x: 2^ceil(log2(largest finite magnitude / 448)), at least 2^-100."""
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)]
    m = a.max() if a.size else 0.0
    if m == 0.0:
        return 2.0 ** -100
    f, e = math.frexp(m)                           # m = f * 2^e, 0.5 <= f < 1; 448 = 0.875 * 2^9
    return 2.0 ** max(-100, e - 9 if f <= 0.875 else e - 8)


def new_cache(layers, pages, kv_heads, page, head_dim, seqs, max_pages):
    pool = (layers, pages, kv_heads, page, head_dim)
    return dict(k=np.zeros(pool, np.uint8), v=np.zeros(pool, np.uint8), k_scale=np.ones(pool[:3]), v_scale=np.ones(pool[:3]),
                table=np.full((seqs, max_pages), -1, np.int32), lengths=np.zeros(seqs, np.int32),
                refcount=np.zeros(pages, np.int32))


def _pages(c, tokens):
    return -(-tokens // c["k"].shape[3])


def _entries(c, seqs):
    """(index, sequence) of the list's usable entries, and flags: -1 is passed over, a repeat or an outsider flagged."""
    out, flags, seen = [], 0, set()
    for i, s in enumerate(seqs):
        if s == -1:
            continue
        if s < 0 or s >= len(c["lengths"]) or s in seen:
            flags |= BAD_SEQUENCE
            continue
        seen.add(s)
        out.append((i, int(s)))
    return out, flags


def reserve(c, seqs, counts):
    page, room = c["k"].shape[3], c["table"].shape[1] * c["k"].shape[3]
    entries, flags = _entries(c, seqs)
    todo, shared = [], {}
    for i, s in entries:
        n, add = int(c["lengths"][s]), int(counts[i])
        if n < 0 or add < 0 or n + add > room:
            flags |= BAD_LENGTH
            continue
        last = -1
        if add and n % page:
            last = int(c["table"][s, n // page])
            if not 0 <= last < len(c["refcount"]):
                flags |= BAD_PAGE
                continue
            if c["refcount"][last] <= 1:
                last = -1
        if last >= 0:
            shared.setdefault(last, []).append(s)
        todo.append((s, n, add, last))
    free = [p for p in range(len(c["refcount"])) if c["refcount"][p] == 0]
    plan, used = [], 0
    for s, n, add, last in todo:
        copies = last >= 0 and not (len(shared[last]) == c["refcount"][last] and shared[last][0] == s)
        fresh = _pages(c, n + add) - _pages(c, n)
        plan.append((s, n, add, last if copies else -1, used))
        used += copies + fresh
    if used > len(free):
        return flags | NO_PAGES
    for s, n, add, last, at in plan:
        if last >= 0:
            new = free[at]
            at += 1
            for name in ("k", "v", "k_scale", "v_scale"):
                c[name][:, new] = c[name][:, last]
            c["table"][s, n // page] = new
            c["refcount"][new] = 1
            c["refcount"][last] -= 1
        for x in range(_pages(c, n), _pages(c, n + add)):
            c["table"][s, x] = free[at]
            c["refcount"][free[at]] = 1
            at += 1
        c["lengths"][s] = n + add
    return flags


def fork(c, parents, children):
    flags, seen, pairs = 0, set(), []
    seqs = len(c["lengths"])
    used = {int(p) for p, s in zip(parents, children) if p != -1 and s != -1}
    for p, s in zip(parents, children):
        if p == -1 or s == -1:
            continue
        if not (0 <= p < seqs and 0 <= s < seqs) or s in seen or s in used:
            flags |= BAD_SEQUENCE
        else:
            pairs.append((int(p), int(s)))
        seen.add(int(s))
    for p, s in pairs:
        if c["lengths"][s] != 0:
            flags |= BAD_LENGTH
            continue
        n = _pages(c, int(c["lengths"][p]))
        c["table"][s, :n] = c["table"][p, :n]
        for x in c["table"][p, :n]:
            c["refcount"][x] += 1
        c["lengths"][s] = c["lengths"][p]
    return flags


def truncate(c, seqs, new_lengths=None):
    entries, flags = _entries(c, seqs)
    for i, s in entries:
        n, cut = int(c["lengths"][s]), 0 if new_lengths is None else int(new_lengths[i])
        if cut < 0 or cut > n:
            flags |= BAD_LENGTH
            continue
        for x in range(_pages(c, cut), _pages(c, n)):
            c["refcount"][c["table"][s, x]] -= 1
            c["table"][s, x] = -1
        c["lengths"][s] = cut
    return flags


def copy_pages(c, pairs):
    flags, pages, todo = 0, len(c["refcount"]), []
    live = [(int(a), int(b)) for a, b in pairs]
    for i, (a, b) in enumerate(live):
        if a < 0 or b < 0 or a == b:
            continue
        source = any(o[0] == b and o[1] >= 0 and o[0] != o[1] for o in live)
        again = any(o[1] == b and o[0] >= 0 and o[0] != o[1] for o in live[:i])
        if a >= pages or b >= pages or source or again:
            flags |= BAD_PAGE
        else:
            todo.append((a, b))
    for a, b in todo:
        for name in ("k", "v", "k_scale", "v_scale"):
            c[name][:, b] = c[name][:, a]
    return flags


def compact(c):
    ref = c["refcount"]
    live = int((ref != 0).sum())
    holes = [p for p in range(live) if ref[p] == 0]
    movers = [p for p in range(live, len(ref)) if ref[p] != 0]
    new = np.where(ref != 0, np.arange(len(ref)), -1).astype(np.int32)
    for a, b in zip(movers, holes):
        for name in ("k", "v", "k_scale", "v_scale"):
            c[name][:, b] = c[name][:, a]
        ref[b], ref[a], new[a] = ref[a], 0, b
    t = c["table"]
    t[t >= 0] = new[t[t >= 0]]
    return new


def append(c, layer, k, v, seqs, cu):
    page = c["k"].shape[3]
    entries, flags = _entries(c, seqs)
    before = np.maximum.accumulate(np.concatenate([[0], cu]))      # the largest bound in front of each
    for i, s in entries:
        n, end = int(cu[i + 1]) - int(cu[i]), int(c["lengths"][s])
        if n < 0 or cu[i] < before[i] or cu[i + 1] > len(k) or end - n < 0 or end > c["table"].shape[1] * page:
            flags |= BAD_LENGTH
            continue
        at, row = end - n, int(cu[i])
        while at < end:
            p, a = int(c["table"][s, at // page]), at % page
            m = min(page - a, end - at)
            if not 0 <= p < len(c["refcount"]):
                flags |= BAD_PAGE
            elif c["refcount"][p] > 1:
                flags |= SHARED_PAGE
            else:
                for name, x in (("k", k), ("v", v)):
                    for h in range(c["k"].shape[2]):
                        rows = np.asarray(x[row:row + m, h], np.float64)
                        codes, scale = c[name][layer, p, h], c[name + "_scale"]
                        step = step_of(rows)
                        if a:
                            old = scale[layer, p, h]
                            step = max(step, old)
                            if step > old:
                                codes[:a] = encode(VALUES[codes[:a]] * (old / step))
                        codes[a:a + m] = encode(rows / step)
                        scale[layer, p, h] = step
            at, row = at + m, row + m
    return flags


def dense(c, layer, s, tokens):
    """A sequence's first `tokens` keys and values, (kv_heads, tokens, head_dim); NaN where a page is not in the pool."""
    page, out = c["k"].shape[3], []
    for name in ("k", "v"):
        x = np.full((c["k"].shape[2], _pages(c, tokens) * page, c["k"].shape[4]), np.nan)
        for b in range(_pages(c, tokens)):
            p = c["table"][s, b]
            if 0 <= p < len(c["refcount"]):
                x[:, b * page:(b + 1) * page] = VALUES[c[name][layer, p]] * c[name + "_scale"][layer, p][:, None, None]
        out.append(x[:, :tokens])
    return out


def attention_partials(c, layer, q, seqs, scale, positions=None):
    """(maximum, exp_sum, weighted, largest sum |q k| scale, largest |v| seen) by rows; NaN rows for unused entries."""
    n, q_len, heads, d = q.shape
    hk = c["k"].shape[2]
    page, pages = c["k"].shape[3], len(c["refcount"])
    m, l = np.full((n, q_len, heads), np.nan), np.full((n, q_len, heads), np.nan)
    w = np.full((n, q_len, heads, d), np.nan)
    reach, vmax = 0.0, 0.0
    for i, s in enumerate(seqs):
        if s < 0 or s >= len(c["lengths"]):
            continue
        n_tok = int(c["lengths"][s])
        k, v = dense(c, layer, s, n_tok)
        kept = np.array([0 <= c["table"][s, t // page] < pages for t in range(n_tok)], bool)
        first = n_tok - q_len if positions is None else int(positions[i])
        for j in range(q_len):
            t = np.arange(n_tok)
            see = kept & (t <= first + j)
            for h in range(heads):
                g = h // (heads // hk)
                m[i, j, h], l[i, j, h], w[i, j, h] = -np.inf, 0.0, 0.0
                if not see.any():
                    continue
                x = np.asarray(q[i, j, h], np.float64)
                sc = k[g, see] @ x * scale
                m[i, j, h] = sc.max()
                p = np.exp(sc - sc.max())
                l[i, j, h] = p.sum()
                w[i, j, h] = p @ v[g, see]
                reach = max(reach, float(np.nan_to_num(np.abs(k[g, see]) @ np.abs(x)).max() * abs(scale)))
                vmax = max(vmax, float(np.nan_to_num(np.abs(v[g, see])).max()))
    return m, l, w, reach, vmax


def attention(c, layer, q, seqs, scale, positions=None):
    m, l, w, reach, vmax = attention_partials(c, layer, q, seqs, scale, positions)
    with np.errstate(invalid="ignore"):
        out = np.where(l[..., None] == 0, 0.0, w / np.where(l == 0, 1.0, l)[..., None])
    return out, reach, vmax
