"""The paged 8-bit key/value cache's operators, as measured: their cases, plain forms, work and 64-bit values.

The cache holds e4m3 codes in pages of `page` tokens, (layers, pages, kv_heads, page, head_dim), with one fp32 scale, a
power of two, for each page and head.  `table` gives each sequence's pages, `lengths` its tokens, `refcount` how many
sequences hold a page.  Four paths through it are measured:

  attention  softmax(scale * q k^T) v over each sequence's pages, queries at the sequences' ends
  partials   the same over one rank's part of the history, left as (maximum, exp_sum, weighted) for the merge over ranks
  append     new K/V rows quantised into the pages that `table` gives them
  branch     sequences forked, then one more token's place reserved in all of them (shared last pages are copied)
  retire     sequences dropped, then the remaining pages compacted to the front of the pool

With `own` false, run() computes with elementary torch operations; with `own` true it makes the framework's calls.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one chat of about four thousand tokens, a single new token: latency
        dict(name="attn_one_4k", kind="attention", n=1, q_len=1, heads=64, kv_heads=8, head_dim=128, page=64,
             len_lo=4099, len_hi=4099, dtype="bf16", mix=1),
        # a decode step of 32 chats of mixed lengths
        dict(name="attn_b32", kind="attention", n=32, q_len=1, heads=64, kv_heads=8, head_dim=128, page=64,
             len_lo=300, len_hi=6000, dtype="bf16", mix=2),
        # a decode step over long documents: the largest
        dict(name="attn_b32_long", kind="attention", n=32, q_len=1, heads=64, kv_heads=8, head_dim=128, page=128,
             len_lo=20001, len_hi=36001, dtype="bf16", mix=3),
        # four drafted tokens of 16 chats verified at once, groups of three heads, small pages, fp32 queries
        dict(name="attn_verify_f32", kind="attention", n=16, q_len=4, heads=24, kv_heads=8, head_dim=64, page=16,
             len_lo=1, len_hi=3000, dtype="f32", mix=4),
        # one rank's 512 keys for the partials that the merge takes, 32 and 256 queries of 64 heads
        dict(name="partials_bs32_f32", kind="partials", n=32, q_len=1, heads=64, kv_heads=8, head_dim=128, page=64,
             len_lo=0, len_hi=512, dtype="f32", mix=5),
        dict(name="partials_bs256", kind="partials", n=256, q_len=1, heads=64, kv_heads=8, head_dim=128, page=64,
             len_lo=512, len_hi=512, dtype="bf16", mix=6),
        # one token of each of 256 chats written
        dict(name="append_b256", kind="append", n=256, new_lo=1, new_hi=1, kv_heads=8, head_dim=128, page=64,
             len_lo=0, len_hi=700, dtype="bf16", mix=7),
        # eight prompts of mixed lengths written, some of them continuing a sequence in the middle of a page
        dict(name="append_prompts", kind="append", n=8, new_lo=500, new_hi=8001, kv_heads=8, head_dim=128, page=64,
             len_lo=0, len_hi=130, dtype="bf16", mix=8),
        # one short chat branched seven ways
        dict(name="branch_one", kind="branch", n=1, ways=7, layers=2, kv_heads=2, head_dim=64, page=16, len_lo=37,
             len_hi=37, mix=9),
        # eight chats branched four ways each, four layers
        dict(name="branch_b8", kind="branch", n=8, ways=4, layers=4, kv_heads=8, head_dim=128, page=64, len_lo=300,
             len_hi=4000, mix=10),
        # a small pool with every other sequence gone
        dict(name="retire_small", kind="retire", n=9, layers=1, kv_heads=1, head_dim=128, page=32, len_lo=10,
             len_hi=400, mix=11),
        # half of 40 sequences gone from a pool of eight layers
        dict(name="retire_b40", kind="retire", n=40, layers=8, kv_heads=8, head_dim=128, page=64, len_lo=200,
             len_hi=4000, mix=12),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["attention", "attention", "partials", "append", "branch", "retire"])
    c = dict(kind=kind, kv_heads=rng.choice([1, 2, 3, 4, 5, 8]), head_dim=rng.choice([64, 128, 128, 256]),
             page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1 << 30))
    token = c["kv_heads"] * c["head_dim"] * 2
    if kind in ("attention", "partials"):
        c["n"] = log(1, 200)
        c["q_len"] = rng.choice([1, 1, 1, 2, 3, 5, 8])
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        most = max(64, min(40000, int(6e8) // (c["n"] * token * c["q_len"])))
        c["len_hi"] = log(20, most)
        c["len_lo"] = rng.choice([0, 1, c["len_hi"] // 2, c["len_hi"]])
    elif kind == "append":
        c["n"] = log(1, 300)
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["new_hi"] = rng.choice([1, 1, rng.randrange(2, 9), log(10, max(12, min(8000, 24000 // c["n"])))])
        c["new_lo"] = rng.choice([1, c["new_hi"]])
        c["len_lo"], c["len_hi"] = 0, log(10, 600)
    elif kind == "branch":
        c["n"], c["ways"], c["layers"] = log(1, 12), rng.randrange(1, 6), rng.choice([1, 2, 4])
        c["len_lo"], c["len_hi"] = 1, log(20, 3000)
    else:
        c["n"], c["layers"] = log(2, 40), rng.choice([1, 2, 4])
        c["len_lo"], c["len_hi"] = 1, log(20, 3000)
    return c


# --- what a case stands for: lengths and page tables (the same for every seed) --------------------------------------

def _shape(c):
    """Numbers that follow from the case alone."""
    rng = random.Random(c["mix"])
    n = c["n"]
    lens = [rng.randint(c["len_lo"], c["len_hi"]) for _ in range(n)]
    new, ahead = [0] * n, [0] * n
    if c["kind"] == "append":   # the lengths count the new rows
        new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(n)]
        lens = [a + b for a, b in zip(lens, new)]
    elif c["kind"] == "partials":   # where the first query stands, from the first key of this rank's part
        ahead = [x + rng.choice([0, 700, 5000]) - c["q_len"] for x in lens]
    seqs = n * (1 + c["ways"]) if c["kind"] == "branch" else n
    pages = [-(-x // c["page"]) for x in lens]
    room = max(pages) + 2
    total = sum(pages)
    spare = 2 * seqs + 5 if c["kind"] == "branch" else 3
    order = list(range(total + spare))
    rng.shuffle(order)
    if c["kind"] == "retire":   # pages as they come out of a pool in use: mostly in order
        order.sort(key=lambda p: p + rng.uniform(0, 40))
    return dict(lens=lens, new=new, ahead=ahead, pages=pages, seqs=seqs, room=room, pool=total + spare, order=order)


def _visible(c, s):
    """Keys that any query of a sequence sees, summed, and (query, key) pairs."""
    keys = pairs = 0
    for i, x in enumerate(s["lens"]):
        first = s["ahead"][i] if c["kind"] == "partials" else x - c["q_len"]
        each = [max(0, min(x, first + j + 1)) for j in range(c["q_len"])]
        keys += max(each)
        pairs += sum(each)
    return keys, pairs


def work(case):
    c, s = case, _shape(case)
    page_bytes = c["kv_heads"] * (c["page"] * c["head_dim"] + 4) * 2
    if c["kind"] in ("attention", "partials"):
        e = 2 if c["dtype"] == "bf16" else 4
        keys, pairs = _visible(c, s)
        rows = c["n"] * c["q_len"] * c["heads"]
        scales = sum(s["pages"]) * c["kv_heads"] * 8
        stats = rows * 8 if c["kind"] == "partials" else 0
        return {"bytes": keys * c["kv_heads"] * c["head_dim"] * 2 + scales + 2 * rows * c["head_dim"] * e + stats,
                "flops": 4 * pairs * c["heads"] * c["head_dim"]}
    if c["kind"] == "append":
        e = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": sum(s["new"]) * c["kv_heads"] * c["head_dim"] * 2 * (e + 1) + c["n"] * c["kv_heads"] * 8,
                "flops": 0}
    if c["kind"] == "branch":   # of the holders of a partly filled last page, one keeps it and the others get copies
        moved = sum((x % c["page"] != 0) * c["ways"] for x in s["lens"])
        return {"bytes": 2 * moved * c["layers"] * page_bytes + s["pool"] * 4 + s["seqs"] * s["room"] * 4, "flops": 0}
    left = {p for i, k in enumerate(s["pages"]) if i % 2 for p in _row(s, i)[:k]}
    moved = sum(p >= len(left) for p in left)
    return {"bytes": 2 * moved * c["layers"] * page_bytes + s["pool"] * 8 + 2 * s["seqs"] * s["room"] * 4, "flops": 0}


def _row(s, i):
    at = sum(s["pages"][:i])
    return s["order"][at:at + s["pages"][i]]


# --- inputs -----------------------------------------------------------------------------------------------------------

def _step_of(amax):
    """The power of two that brings amax to at most 448, not below 2^-100: exact, from the parts of the number."""
    m, e = torch.frexp(amax)                     # amax = m * 2^e with 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp_min(-100)
    e = torch.where(amax == 0, torch.full_like(e, -100), e)
    return ((e + 127) << 23).int().view(torch.float32)


def prepare(case, seed):
    c, s = case, _shape(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    layers, hk, d, page = c.get("layers", 1), c["kv_heads"], c["head_dim"], c["page"]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def values(*shape):   # a few channels stand out, as in trained keys and values
        x = torch.randn(*shape, generator=g, device=dev)
        return x * (1 + 3 * (torch.rand(shape[-1], generator=g, device=dev) > 0.97))

    st = {"case": dict(c)}
    for name in ("k", "v"):
        x = values(layers, s["pool"], hk, page, d)
        scale = _step_of(x.abs().amax(dim=(3, 4)))
        st[name] = (x / scale[..., None, None]).to(E4M3).view(torch.uint8)
        st[name + "_scale"] = scale
        del x
    table = torch.full((s["seqs"], s["room"]), -1, dtype=torch.int32)
    refcount = torch.zeros(s["pool"], dtype=torch.int32)
    for i, k in enumerate(s["pages"]):
        row = torch.tensor(_row(s, i), dtype=torch.int32)
        table[i, :k] = row
        refcount[row.long()] = 1
    st["table"], st["refcount"] = table.to(dev), refcount.to(dev)
    st["lengths"] = ints(s["lens"] + [0] * (s["seqs"] - c["n"]))
    st["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if c["kind"] in ("attention", "partials"):
        st["seqs"] = ints(random.Random(c["mix"] + 1).sample(range(c["n"]), c["n"]))
        st["q"] = (1.5 * torch.randn(c["n"], c["q_len"], c["heads"], d, generator=g, device=dev)).to(DTYPES[c["dtype"]])
        st["positions"] = ints(s["ahead"])[st["seqs"].long()].contiguous()
        st["scale"] = d ** -0.5
        # stale bytes behind each sequence's end, NaN codes among them
        tail = torch.arange(page, device=dev)[None, :] >= (st["lengths"] - 1).clamp_min(0)[:, None] % page + 1
        held = st["lengths"] > 0
        last = st["table"].gather(1, ((st["lengths"] - 1).clamp_min(0) // page).long()[:, None])[held, 0].long()
        for name in ("k", "v"):
            rows = st[name][0, last]
            st[name][0, last] = torch.where(tail[held][:, None, :, None], torch.full_like(rows, 0x7F), rows)
    elif c["kind"] == "append":
        total = sum(s["new"])
        cu = [0]
        for x in s["new"]:
            cu.append(cu[-1] + x)
        # K and V as columns of one projection's output, behind the queries
        both = torch.cat([values(total, hk * d), values(total, hk * d)], dim=1).to(DTYPES[c["dtype"]])
        st["k_new"] = both[:, :hk * d].unflatten(1, (hk, d))
        st["v_new"] = both[:, hk * d:].unflatten(1, (hk, d))
        st["cu"], st["seqs"] = ints(cu), ints(list(range(c["n"])))
        st["of"] = torch.repeat_interleave(torch.arange(c["n"], device=dev), st["cu"].diff().long(), output_size=total)
    else:
        st["saved"] = {k: st[k].clone() for k in ("table", "lengths", "refcount")}
        if c["kind"] == "branch":
            n, w = c["n"], c["ways"]
            st["parents"] = ints([i for i in range(n) for _ in range(w)])
            st["children"] = ints([n + i for i in range(n * w)])
            st["all"] = ints(list(range(s["seqs"])))
            st["ones"] = ints([1] * s["seqs"])
        else:
            st["gone"] = ints(list(range(0, c["n"], 2)))
    return st


# --- plain forms ------------------------------------------------------------------------------------------------------

def _plain_attention(st):
    c = st["case"]
    seqs, page, d, hk = st["seqs"].long(), c["page"], c["head_dim"], c["kv_heads"]
    rows, lens = st["table"][seqs].clamp_min(0).long(), st["lengths"][seqs]
    n, width = rows.shape

    def dense(name):   # (n, kv_heads, tokens, head_dim) in fp32
        x = st[name][0][rows].view(E4M3).float() * st[name + "_scale"][0][rows][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(n, hk, width * page, d)

    first = st["positions"] if c["kind"] == "partials" else lens - c["q_len"]
    t = torch.arange(width * page, device=rows.device)
    q_at = first[:, None] + torch.arange(c["q_len"], device=rows.device)
    seen = (t < lens[:, None])[:, None, :] & (t <= q_at[:, :, None])              # (n, q_len, tokens)
    q = st["q"].float().unflatten(2, (hk, c["heads"] // hk)).permute(0, 2, 1, 3, 4)     # (n, hk, q_len, group, d)
    s = (q.flatten(2, 3) @ dense("k").transpose(2, 3)).unflatten(2, q.shape[2:4]) * st["scale"]
    s = s.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    top = s.amax(dim=4)
    p = torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top)[..., None])
    v = dense("v").masked_fill(~seen.any(dim=1)[:, None, :, None], 0)
    total, o = p.sum(dim=4), (p.flatten(2, 3) @ v).unflatten(2, q.shape[2:4])

    def whole(x):   # back to (n, q_len, heads, ...)
        return x.transpose(1, 2).flatten(2, 3)

    if c["kind"] == "partials":
        return {"maximum": whole(top), "exp_sum": whole(total), "weighted": whole(o).to(st["q"].dtype)}
    return whole(o / torch.where(total > 0, total, torch.ones_like(total))[..., None]).to(st["q"].dtype)


def _cache(st):
    out = {name: st[name] for name in ("k_scale", "v_scale")}
    return out | {"k": st["k"].view(E4M3), "v": st["v"].view(E4M3)}


def _plain_append(st):
    page = st["case"]["page"]
    seqs, of, new = st["seqs"].long(), st["of"], st["cu"].diff()
    start = st["lengths"][seqs] - new
    at = start[of] + torch.arange(of.numel(), device=of.device) - st["cu"][of]
    pages, slot = st["table"][seqs[of], at // page].long(), (at % page).long()
    kept = start % page                                   # slots of the first page that hold earlier tokens
    first = st["table"][seqs, start // page].long()
    for name in ("k", "v"):
        x, scale, pool = st[name + "_new"].float(), st[name + "_scale"][0], st[name][0]
        amax = torch.zeros_like(scale).index_reduce_(0, pages, x.abs().amax(dim=2), "amax")
        step = _step_of(amax[pages])                      # (tokens, kv_heads)
        goes_on = (kept[of] > 0) & (pages == first[of])
        old = scale[first]
        step = torch.where(goes_on[:, None], torch.maximum(step, scale[pages]), step)
        scale.index_copy_(0, pages, step)                 # rows of one page agree
        held = pool[first].view(E4M3).float() * (old / scale[first])[..., None, None]
        stays = (torch.arange(page, device=of.device) < kept[:, None])[:, None, :, None]
        pool[first] = torch.where(stays, held.to(E4M3).view(torch.uint8), pool[first])
        pool[pages, :, slot] = (x / step[..., None]).to(E4M3).view(torch.uint8)
    return _cache(st)


def _restore(st):
    """Both kinds of page work start from the page map that was saved."""
    for name, x in st["saved"].items():
        st[name].copy_(x)


def _pages_out(st):
    return _cache(st) | {name: st[name] for name in ("table", "lengths", "refcount")}


def _plain_branch(st):
    page, ref, table, lengths = st["case"]["page"], st["refcount"], st["table"], st["lengths"]
    parents, children, seqs = st["parents"].long(), st["children"].long(), st["all"].long()
    pool = ref.numel()
    # fork: the children hold their parents' pages
    rows = table[parents]
    table[children], lengths[children] = rows, lengths[parents]
    counts = torch.zeros(pool + 1, dtype=torch.int32, device=ref.device)
    idx = torch.where(rows >= 0, rows, pool).long().flatten()
    ref += counts.index_add_(0, idx, torch.ones_like(idx, dtype=torch.int32))[:pool]
    # reserve: the lowest free pages, in the sequences' order; a shared, partly filled last page is copied, except for
    # the first of its holders in the list where all of them are in it
    free = torch.argsort((ref != 0).int(), stable=True).int()
    rows, lens = table[seqs], lengths[seqs]
    held, after = (lens + page - 1) // page, (lens + st["ones"] + page - 1) // page
    at = torch.arange(rows.shape[1], device=ref.device)
    last = rows.gather(1, (lens // page).long()[:, None])[:, 0]
    shared = (lens % page > 0) & (ref[last.clamp_min(0).long()] > 1)
    same = shared & (last[:, None] == last)
    keeps = (same.sum(1) == ref[last.clamp_min(0).long()]) & (same.int().argmax(1) == torch.arange(len(last), device=ref.device))
    own_copy = shared & ~keeps
    takes = after - held + own_copy
    base = takes.cumsum(0) - takes
    new_at = base[:, None] + own_copy[:, None] + (at - held[:, None])
    fresh = (at >= held[:, None]) & (at < after[:, None])
    moved = own_copy[:, None] & (at == (lens // page)[:, None])
    pick = torch.where(moved, base[:, None], torch.where(fresh, new_at, torch.zeros_like(new_at))).clamp(0, pool - 1)
    rows = torch.where(fresh | moved, free[pick.long()], rows)
    table[seqs], lengths[seqs] = rows, lens + st["ones"]
    change = torch.zeros(pool + 1, dtype=torch.int32, device=ref.device)
    idx = torch.where(fresh | moved, rows, pool).long().flatten()
    change.index_add_(0, idx, torch.ones_like(idx, dtype=torch.int32))
    change.index_add_(0, torch.where(own_copy, last, pool).long(), torch.full_like(last, -1))
    ref += change[:pool]
    source = torch.arange(pool + 1, device=ref.device)
    target = torch.where(own_copy, free[base.clamp(0, pool - 1).long()], pool).long()
    source = source.index_copy(0, target, last.clamp_min(0).long())[:pool]   # where each page's contents come from
    for name in ("k", "v", "k_scale", "v_scale"):
        st[name].copy_(st[name][:, source])
    return _pages_out(st)


def _plain_retire(st):
    ref, table, lengths, gone = st["refcount"], st["table"], st["lengths"], st["gone"].long()
    pool = ref.numel()
    rows = table[gone]
    idx = torch.where(rows >= 0, rows, pool).long().flatten()
    counts = torch.zeros(pool + 1, dtype=torch.int32, device=ref.device)
    ref -= counts.index_add_(0, idx, torch.ones_like(idx, dtype=torch.int32))[:pool]
    table[gone], lengths[gone] = torch.full_like(rows, -1), torch.zeros_like(lengths[gone])
    # live pages behind the first `live` places go, in order, to the free places before them
    p = torch.arange(pool, device=ref.device)
    used = ref > 0
    live = used.sum()
    hole, mover = ~used & (p < live), used & (p >= live)
    holes, movers = torch.argsort((~hole).int(), stable=True), torch.argsort((~mover).int(), stable=True)
    goes = p < hole.sum()
    new_at = torch.cat([torch.where(used, p, -1), p.new_tensor([-1])])
    new_at = new_at.index_copy(0, torch.where(goes, movers, pool), torch.where(goes, holes, -1))
    source = torch.cat([p, p.new_tensor([0])]).index_copy(0, torch.where(goes, holes, pool), torch.where(goes, movers, 0))[:pool]
    table.copy_(torch.where(table >= 0, new_at[table.clamp_min(0).long()].int(), table))
    ref.copy_(torch.where(p < live, ref[source], torch.zeros_like(ref)))
    for name in ("k", "v", "k_scale", "v_scale"):
        st[name].copy_(st[name][:, source])
    return _pages_out(st) | {"new_index": new_at[:pool].int()}


def _handle(st):
    """The framework's cache object over the state's buffers, made once, as a program keeps it."""
    if "handle" not in st:
        from tensor_sharded_mlp_b200 import kv_cache
        st["handle"] = kv_cache.KvCache8.over(*(st[k] for k in ("k", "v", "k_scale", "v_scale", "table", "lengths",
                                                                "refcount", "status")))
    return st["handle"]


def run(state):
    st, kind = state, state["case"]["kind"]
    if kind in ("branch", "retire"):
        _restore(st)
    if not own:
        return {"attention": _plain_attention, "partials": _plain_attention, "append": _plain_append,
                "branch": _plain_branch, "retire": _plain_retire}[kind](st)
    cache = _handle(st)
    if kind == "attention":
        return cache.attention(0, st["q"], seqs=st["seqs"], scale=st["scale"])
    if kind == "partials":
        m, s, w = cache.attention_partials(0, st["q"], seqs=st["seqs"], positions=st["positions"], scale=st["scale"])
        return {"maximum": m, "exp_sum": s, "weighted": w}
    if kind == "append":
        cache.append(0, st["k_new"], st["v_new"], seqs=st["seqs"], cu_tokens=st["cu"])
        return _cache(st)
    if kind == "branch":
        cache.fork(st["parents"], st["children"])
        cache.reserve(st["all"], st["ones"])
        return _pages_out(st)
    cache.truncate(st["gone"])
    return _pages_out(st) | {"new_index": cache.compact()}


# --- 64-bit values ----------------------------------------------------------------------------------------------------

def _decode(codes):
    """The numbers that e4m3 bytes stand for, from their bit fields: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    x = np.where((b & 127) == 127, np.nan, x) * np.where(b >> 7, -1.0, 1.0)
    if isinstance(codes, torch.Tensor):
        return torch.from_numpy(x).to(codes.device)[codes.long()]
    return x[codes]


def _to_e4m3(x):
    """The nearest e4m3 number to each of x (at most 448 in size), ties to the even last bit, in 64 bits."""
    a = np.abs(x)
    _, e = np.frexp(a)
    quantum = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.copysign(np.rint(a / quantum) * quantum, x)


def _exact_attention(c, st):
    hk, d, page, q_len = c["kv_heads"], c["head_dim"], c["page"], c["q_len"]
    group = c["heads"] // hk
    outs, tops, sums = [], [], []
    lengths, table = st["lengths"].tolist(), st["table"]
    for i, s in enumerate(st["seqs"].tolist()):
        x = lengths[s]
        q = st["q"][i].double().reshape(q_len, hk, group, d)
        pages = table[s, :-(-x // page)].long()
        kd, vd = ((_decode(st[m][0][pages]) * st[m + "_scale"][0][pages].double()[..., None, None])
                  .transpose(0, 1).reshape(hk, -1, d)[:, :x] for m in ("k", "v"))
        first = int(st["positions"][i]) if c["kind"] == "partials" else x - q_len
        o = torch.zeros(q_len, hk, group, d, dtype=torch.float64, device=q.device)
        top = torch.full((q_len, hk, group), float("-inf"), dtype=torch.float64, device=q.device)
        tot = torch.zeros_like(top)
        for j in range(q_len):
            end = max(0, min(x, first + j + 1))
            if not end:
                continue
            for h in range(hk):
                s_ = q[j, h] @ kd[h, :end].T * c["head_dim"] ** -0.5
                top[j, h] = s_.amax(dim=1)
                p = torch.exp(s_ - top[j, h][:, None])
                tot[j, h] = p.sum(dim=1)
                o[j, h] = p @ vd[h, :end]
                if c["kind"] == "attention":
                    o[j, h] /= tot[j, h][:, None]
        outs.append(o.flatten(1, 2))
        tops.append(top.flatten(1))
        sums.append(tot.flatten(1))
    if c["kind"] == "attention":
        return torch.stack(outs)
    return {"maximum": torch.stack(tops), "exp_sum": torch.stack(sums), "weighted": torch.stack(outs)}


def _exact_append(c, st):
    page = c["page"]
    cu, lengths, table = st["cu"].tolist(), st["lengths"].tolist(), st["table"].cpu().numpy()
    out = {}
    for name in ("k", "v"):
        pool, scale = _decode(st[name].cpu().numpy()), st[name + "_scale"].cpu().numpy().astype(np.float64)
        rows = st[name + "_new"].double().cpu().numpy()
        for i in range(c["n"]):
            at, end, row = lengths[i] - (cu[i + 1] - cu[i]), lengths[i], cu[i]
            while at < end:
                p, a = table[i, at // page], at % page
                count = min(page - a, end - at)
                x = rows[row:row + count].transpose(1, 0, 2)                       # (kv_heads, count, head_dim)
                amax = np.abs(x).max(axis=(1, 2))
                step = np.array([2.0 ** max(-100, math.ceil(math.log2(m / 448))) if m else 2.0 ** -100 for m in amax])
                if a:
                    grown = np.maximum(step, scale[0, p])
                    pool[0, p, :, :a] = _to_e4m3(pool[0, p, :, :a] * (scale[0, p] / grown)[:, None, None])
                    step = grown
                scale[0, p] = step
                pool[0, p, :, a:a + count] = _to_e4m3(x / step[:, None, None])
                at, row = at + count, row + count
        out[name], out[name + "_scale"] = pool, scale
    return out


def exact(case, seed):
    c = case
    if c["kind"] in ("branch", "retire"):   # bytes and whole numbers that move: nothing is computed
        return None
    st = prepare(case, seed)
    return _exact_append(c, st) if c["kind"] == "append" else _exact_attention(c, st)
