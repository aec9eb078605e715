"""Attention over the paged 8-bit cache against the fp64 oracle, within bounds counted from its roundings
(kv8_helpers): head sizes, groups, lengths from nothing to thousands, pages that end inside a tile, several queries
with their causal limits, ranks' positions, NaN and garbage in unseen places, padded and invalid entries, streams,
graphs, and the whole step with append, fork and merge."""
import numpy as np
import pytest
import torch

from kv8_helpers import HALF, close, filled, flags, ints, on_gpu, score_bound, weight_bound
from oracle import kv8

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


def query(r, n, q_len, heads, d, dtype, spread=1.0):
    return torch.from_numpy((r.standard_normal((n, q_len, heads, d)) * spread).astype(np.float32)).cuda().to(TORCH[dtype])


def check(c, cache, q, seqs, scale=None, positions=None, layer=0, tokens=None, what=""):
    """Both forms against the oracle; entries without a sequence must stay as they were."""
    d, dt = q.shape[3], q.dtype
    scale = d ** -0.5 if scale is None else scale
    tokens = tokens or int(max(c["lengths"].max(), 1))
    m, l, w, reach, vmax = kv8.attention_partials(c, layer, q.double().cpu().numpy(), seqs, scale, positions)
    listed, pos = ints(seqs), None if positions is None else ints(positions)
    want = np.where(l[..., None] == 0, 0.0, w / np.where(l == 0, 1.0, l)[..., None])
    rel = weight_bound(reach, d, tokens, dt)
    sb = score_bound(reach, d)
    mark = 12345.0
    out = torch.full(q.shape, mark, dtype=dt, device="cuda")
    assert cache.attention(layer, q, listed, pos, scale, out=out) is out
    pm, pl = (torch.full(q.shape[:3], mark, device="cuda") for _ in range(2))
    pw = torch.full(q.shape, mark, dtype=dt, device="cuda")
    cache.attention_partials(layer, q, listed, pos, scale, pm, pl, pw)
    torch.cuda.synchronize()
    got, gm, gl, gw = (t.double().cpu().numpy() for t in (out, pm, pl, pw))
    keep = float(torch.tensor(mark, dtype=dt))
    rest = [i for i, s in enumerate(seqs) if not 0 <= s < len(c["lengths"])]
    assert all((x[rest] == y).all() for x, y in ((got, keep), (gw, keep), (gm, mark), (gl, mark)))
    rows = [i for i, s in enumerate(seqs) if 0 <= s < len(c["lengths"])]
    close(got[rows], want[rows], rel * vmax + HALF[dt] * (np.abs(want[rows]) + rel * vmax) + 1e-30, what + " out")
    close(gm[rows], m[rows], sb + 2.0 ** -22 * np.abs(np.where(np.isfinite(m[rows]), m[rows], 0)), what + " maximum")
    close(gl[rows], l[rows], l[rows] * (4 * sb + 2 * (tokens / 16 + 8) * 2.0 ** -23 + 2.0 ** -20), what + " exp_sum")
    close(gw[rows], w[rows], l[rows][..., None] * (2 * sb + rel) * vmax + HALF[dt] * (np.abs(w[rows]) +
          l[rows][..., None] * rel * vmax) + 1e-30, what + " weighted")


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 300, 511, 513]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 8), (3, 5), (1, 16), (2, 17), (1, 40)])
def test_one_query(kv_heads, group, head_dim, dtype):
    r = np.random.default_rng(head_dim + group)
    page = {64: 16, 128: 64, 256: 32}[head_dim]
    c = filled(r, LENGTHS, 1, kv_heads, page, head_dim)
    seqs = [int(x) for x in r.permutation(len(LENGTHS))]
    check(c, on_gpu(c), query(r, len(seqs), 1, kv_heads * group, head_dim, dtype), seqs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len,kv_heads,group", [(2, 2, 4), (3, 1, 1), (5, 2, 3), (16, 1, 2), (33, 1, 1), (128, 1, 1), (7, 1, 9)])
def test_several_queries_are_causal(q_len, kv_heads, group, dtype):
    r = np.random.default_rng(q_len)
    lengths = [0, 1, q_len - 1, q_len, q_len + 1, 16, 50, 131]          # the first rows of short ones see nothing
    c = filled(r, lengths, 1, kv_heads, 16, 64)
    check(c, on_gpu(c), query(r, len(lengths), q_len, kv_heads * group, 64, dtype), list(range(len(lengths))))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("head_dim", [128, 256])
@pytest.mark.parametrize("q_len,kv_heads,group", [(5, 1, 3), (2, 2, 8), (9, 1, 5)])
def test_several_queries_of_wider_heads(q_len, kv_heads, group, head_dim, dtype):
    r = np.random.default_rng(q_len + head_dim)
    lengths = [q_len - 1, q_len + 14, 100, 40]
    c = filled(r, lengths, 1, kv_heads, 32, head_dim)
    check(c, on_gpu(c), query(r, 4, q_len, kv_heads * group, head_dim, dtype), [3, 2, 1, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_segments_beside_a_long_one(dtype):
    """Sequences of one step each, and one of hundreds: every way a segment's start and end can meet a cut."""
    r = np.random.default_rng(30)
    lengths = [int(x) for x in r.integers(0, 20, 120)] + [5000] + [int(x) for x in r.integers(0, 70, 60)]
    c = filled(r, lengths, 1, 2, 16, 64)
    check(c, on_gpu(c), query(r, len(lengths), 1, 6, 64, dtype), list(range(len(lengths))))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes_and_layers(page):
    r = np.random.default_rng(page)
    c = filled(r, [3, page - 1, page, page + 1, 2 * page + 9, 700], 3, 2, page, 128)
    cache = on_gpu(c)
    for layer in range(3):
        check(c, cache, query(r, 6, 2, 8, 128, "bf16"), [5, 4, 3, 2, 1, 0], layer=layer)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ranks_positions(dtype):
    r = np.random.default_rng(11)
    lengths = [64, 64, 64, 64, 30, 30, 0, 64]
    c = filled(r, lengths, 1, 2, 16, 64)
    positions = [1000, 62, -1, -4, 29, 2 ** 31 - 1, 5, -2 ** 31]
    check(c, on_gpu(c), query(r, 8, 4, 6, 64, dtype), list(range(8)), positions=positions)


def test_long_sequences():
    """Split over every SM and joined; one long sequence beside short ones."""
    r = np.random.default_rng(12)
    c = filled(r, [9001, 5, 4096, 1], 1, 1, 64, 64)
    check(c, on_gpu(c), query(r, 4, 1, 8, 64, "bf16"), [0, 1, 2, 3])
    check(c, on_gpu(c), query(r, 5, 2, 3, 64, "f32"), [3, 0, 0, 1, 2])


def test_large_scores_and_peaked_rows():
    """Scores of some hundreds: the maximum moves many times, most weights vanish."""
    r = np.random.default_rng(13)
    c = filled(r, [777, 33, 260], 1, 2, 32, 128, spread=3.0)
    q = query(r, 3, 2, 8, 128, "f32", 20.0)
    check(c, on_gpu(c), q, [0, 1, 2], scale=0.02)
    # keys in rising order of score: every tile raises the maximum
    order = np.argsort(kv8.dense(c, 0, 0, 777)[0][0] @ q[0, 1, 0].double().cpu().numpy())
    assert len(order) == 777
    k = torch.from_numpy(kv8.dense(c, 0, 0, 777)[0].transpose(1, 0, 2)[order].astype(np.float32)).cuda()
    up = kv8.new_cache(1, 30, 2, 32, 128, 1, 30)
    kv8.reserve(up, [0], [777])
    kv8.append(up, 0, k.double().cpu().numpy(), k.double().cpu().numpy(), [0], [0, 777])
    check(up, on_gpu(up), q[:1], [0], scale=0.05)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_of_very_different_scales(dtype):
    """Value scales from 2^-40 to 2^20 between pages: small pages count where the weights are."""
    r = np.random.default_rng(14)
    c = filled(r, [200, 90], 1, 1, 16, 64)
    c["v_scale"] *= 2.0 ** r.integers(-40, 20, c["v_scale"].shape)
    cache = on_gpu(c)
    q = query(r, 2, 2, 4, 64, dtype)
    check(c, cache, q, [0, 1])
    # the weight sits on a page of small values, a page of large values gets next to none
    c["v_scale"][:] = 2.0 ** -30
    c["v_scale"][0, c["table"][0, 3]] = 2.0 ** 10
    cache = on_gpu(c)
    m, l, w, reach, vmax = kv8.attention_partials(c, 0, q.double().cpu().numpy(), [0, 1], 2.0)
    out = cache.attention(0, q, ints([0, 1]), scale=2.0)
    want = w / l[..., None]
    k, v = kv8.dense(c, 0, 0, 200)
    sc = np.einsum("qhd,td->qht", q[0].double().cpu().numpy(), k[0]) * 2.0
    p = np.exp(sc - sc.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    see = np.arange(200) <= 198 + np.arange(2)[:, None, None]
    p = np.where(see, np.exp(sc - np.where(see, sc, -np.inf).max(-1, keepdims=True)), 0)
    p /= p.sum(-1, keepdims=True)
    term = p @ np.abs(v[0])                                            # sum of the terms' magnitudes, per output
    dt = q.dtype
    close(out[0], want[0], (weight_bound(reach, 64, 200, dt) * 2 + HALF[dt]) * term * 1.01, "by terms")


def test_zero_and_arbitrary_scales():
    """Scales of a caller's own: not powers of two, and zero."""
    r = np.random.default_rng(15)
    c = filled(r, [70, 20], 1, 2, 16, 64)
    for n in ("k_scale", "v_scale"):
        c[n] = (c[n] * r.uniform(0.5, 2.0, c[n].shape)).astype(np.float32).astype(np.float64)
    c["v_scale"][0, c["table"][0, 1], 0] = 0.0
    c["k_scale"][0, c["table"][0, 2], 1] = 0.0
    check(c, on_gpu(c), query(r, 2, 1, 4, 64, "f32"), [0, 1])


@pytest.mark.parametrize("stale", [0x7F, 0xFF, 0x00, 0x7E])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_garbage_behind_the_end(stale, dtype):
    r = np.random.default_rng(16)
    c = filled(r, [1, 17, 63, 100], 1, 2, 64, 128, stale=stale)
    check(c, on_gpu(c), query(r, 4, 3, 4, 128, dtype), [0, 1, 2, 3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_reaches_only_the_rows_that_see_it(dtype):
    r = np.random.default_rng(17)
    c = filled(r, [40, 50, 45], 1, 1, 16, 64)
    c["v"][0, c["table"][0, 2], 0, 5, 9] = 0x7F                        # token 37 of 40: queries 36..39
    c["k"][0, c["table"][1, 3], 0, 0, 3] = 0xFF                        # token 48 of 50
    c["v"][0, c["table"][2, 0], 0, 2, 63] = 0xFF                       # token 2: every query
    cache = on_gpu(c)
    q = query(r, 3, 4, 2, 64, dtype)
    check(c, cache, q, [0, 1, 2])
    out = cache.attention(0, q, ints([0, 1, 2])).float()
    assert torch.isfinite(out[0, 0]).all() and torch.isnan(out[0, 1:, :, 9]).all() and \
        torch.isfinite(out[0, :, :, :9]).all() and torch.isfinite(out[0, :, :, 10:]).all()
    assert torch.isfinite(out[1, :2]).all() and torch.isnan(out[1, 2:]).all()
    assert torch.isnan(out[2, :, :, 63]).all() and torch.isfinite(out[2, :, :, :63]).all()


def test_nan_queries_stay_in_their_rows():
    r = np.random.default_rng(18)
    c = filled(r, [40, 300], 1, 2, 16, 64)
    q = query(r, 2, 2, 8, 64, "bf16")
    q[0, 1, 3, 7] = float("nan")
    q[1, 0, 5, 0] = float("inf")
    out = on_gpu(c).attention(0, q, ints([0, 1])).float()
    bad = torch.isnan(out).all(-1)
    want = torch.zeros_like(bad)
    want[0, 1, 3], want[1, 0, 5] = True, True
    assert torch.equal(bad, want) and torch.isfinite(out[~want]).all()
    # one token: a score of minus infinity is no unseen token
    for dtype in ("bf16", "f32"):
        c = filled(r, [1, 0], 1, 1, 16, 64)
        q = query(r, 2, 1, 3, 64, dtype)
        q[:, 0, 0, 5], q[:, 0, 1, 5] = float("inf"), float("-inf")
        cache = on_gpu(c)
        out = cache.attention(0, q, ints([0, 1])).float()
        m, l, w = cache.attention_partials(0, q, ints([0, 1]))
        assert all(torch.isnan(t[0, 0, :2]).all() and torch.isfinite(t[0, 0, 2]).all() for t in (out, m, l, w.float()))
        assert not out[1].bool().any() and torch.isneginf(m[1]).all() and not l[1].bool().any()


def test_small_and_large_queries():
    """Queries far outside fp16's range: only the product with the scale matters."""
    r = np.random.default_rng(19)
    c = filled(r, [100, 37], 1, 2, 16, 64)
    cache = on_gpu(c)
    for size in (2.0 ** -100, 2.0 ** 60):
        q = query(r, 2, 1, 4, 64, "f32") * size
        check(c, cache, q, [0, 1], scale=0.125 / size)
    check(c, cache, query(r, 2, 1, 4, 64, "f32") * 0, [0, 1])


def test_padded_repeated_and_invalid_entries():
    r = np.random.default_rng(20)
    c = filled(r, [40, 7, 100], 1, 2, 16, 64)
    cache = on_gpu(c)
    check(c, cache, query(r, 7, 2, 4, 64, "bf16"), [2, -1, 0, 2, 2, 1, -1])
    assert flags(cache) == 0
    check(c, cache, query(r, 5, 2, 4, 64, "f32"), [2, 3, 0, -7, 1])
    assert flags(cache) == kv8.BAD_SEQUENCE
    c["table"][2, 1], c["table"][2, 4] = -1, len(c["refcount"])         # keys of such pages count as unseen
    cache = on_gpu(c)
    check(c, cache, query(r, 3, 2, 4, 64, "f32"), [2, 1, 0])
    assert flags(cache) == kv8.BAD_PAGE
    q = query(r, 3, 1, 4, 64, "f32")
    for length in (-1, c["table"].shape[1] * 16 + 1):
        cache.lengths[1] = length
        out = torch.full(q.shape, 7.0, device="cuda")
        cache.attention(0, q, ints([2, 1, 0]), out=out)
        assert flags(cache) == kv8.BAD_LENGTH | kv8.BAD_PAGE and (out[1] == 7).all() and (out[0] != 7).any()


def test_no_pages_at_all():
    c = filled(np.random.default_rng(21), [33], 1, 1, 16, 64)
    c["table"][0, :3] = -1
    cache = on_gpu(c)
    q = torch.ones(1, 1, 1, 64, device="cuda")
    assert not cache.attention(0, q).bool().any()
    m, l, w = cache.attention_partials(0, q)
    assert torch.isneginf(m).all() and not l.bool().any() and not w.bool().any()


def test_strided_queries():
    r = np.random.default_rng(22)
    c = filled(r, [40, 17], 1, 2, 16, 64)
    cache = on_gpu(c)
    wide = query(r, 2, 3, 12, 64, "bf16")                              # q | k | v columns
    q = wide[:, :, 4:8]
    assert not q.is_contiguous()
    assert torch.equal(cache.attention(0, q, ints([0, 1])), cache.attention(0, q.contiguous(), ints([0, 1])))
    check(c, cache, q, [0, 1])
    with pytest.raises(ValueError):
        cache.attention(0, wide.transpose(0, 1), ints([0, 1, 0]))
    with pytest.raises(ValueError):
        cache.attention(0, wide[..., :32], ints([0, 1]))
    with pytest.raises(ValueError):
        cache.attention(0, wide.half(), ints([0, 1]))


def test_many_entries():
    r = np.random.default_rng(23)
    n = 1024
    c = filled(r, [int(x) for x in r.integers(0, 40, 50)], 1, 1, 16, 64)
    seqs = [int(x) for x in r.integers(-1, 50, n)]
    check(c, on_gpu(c), query(r, n, 1, 2, 64, "bf16"), seqs)


def test_same_result_every_time_and_on_another_stream():
    r = np.random.default_rng(24)
    c = filled(r, [3000, 500, 10, 1999], 1, 2, 64, 128)
    cache = on_gpu(c)
    q, seqs = query(r, 4, 1, 16, 128, "f32"), ints([0, 1, 2, 3])
    first = cache.attention(0, q, seqs).clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(5):
        for s in streams:                                              # overlapping calls, each with scratch of its own
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                outs.append(cache.attention(0, q, seqs))
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    cache.attention(0, q, seqs, out=out, stream=streams[0])
    outs += [out, cache.attention(0, q, seqs, stream=streams[1]), cache.attention(0, q, seqs, stream=streams[2].cuda_stream)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


def test_two_caches_at_once():
    """Steps of two caches on two streams, page work and attention among each other's."""
    from tensor_sharded_mlp_b200 import kv_cache
    r = np.random.default_rng(31)
    caches, oracles, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        caches.append(kv_cache.KvCache8(1, 64, 2, 64, page_size=16, max_seqs=4, max_tokens=256))
        oracles.append(kv8.new_cache(1, 64, 2, 16, 64, 4, 16))
    seqs, counts = ints([0, 1, 2, 3]), ints([7] * 4)
    rows = [[tuple(torch.from_numpy(r.standard_normal((28, 2, 64)).astype(np.float32)).cuda() for _ in range(2)) for _ in range(2)]
            for _ in range(6)]
    q = query(r, 4, 2, 4, 64, "f32")
    torch.cuda.synchronize()
    got = [None, None]
    for step in range(6):
        for x in range(2):
            with torch.cuda.stream(streams[x]):
                caches[x].reserve(seqs, counts)
                caches[x].append(0, *rows[step][x], seqs)
                got[x] = caches[x].attention(0, q, seqs)
    torch.cuda.synchronize()
    for x in range(2):
        c = oracles[x]
        for step in range(6):
            kv8.reserve(c, range(4), [7] * 4)
            kv8.append(c, 0, *(t.double().cpu().numpy() for t in rows[step][x]), range(4), [0, 7, 14, 21, 28])
        np.testing.assert_array_equal(caches[x].table.cpu().numpy(), c["table"])
        want, reach, vmax = kv8.attention(c, 0, q.double().cpu().numpy(), range(4), 0.125)
        rel = weight_bound(reach, 64, 42, torch.float32)
        close(got[x], want, rel * vmax + HALF[torch.float32] * np.abs(want), f"cache {x}")
        caches[x].check()


def test_sizes_are_refused_when_the_cache_is_made():
    from tensor_sharded_mlp_b200 import kv_cache
    for over in (dict(page_size=24), dict(head_dim=96), dict(page_size=512), dict(kv_heads=300)):
        with pytest.raises(ValueError):
            kv_cache.KvCache8(**{**dict(layers=1, num_pages=4, kv_heads=1, head_dim=64, page_size=16, max_seqs=1,
                                        max_tokens=64), **over})
    c = kv_cache.KvCache8(1, 4, 1, 64, page_size=16, max_seqs=1, max_tokens=64)
    with pytest.raises(ValueError):
        kv_cache.KvCache8.over(c.k, c.v, c.k_scale, c.v_scale, c.table.long(), c.lengths, c.refcount, c.status)
    with pytest.raises(ValueError):
        kv_cache.KvCache8.over(c.k, c.v, c.k_scale, c.v_scale, c.table, c.lengths, c.refcount[:3], c.status)


def test_check_raises_and_clears():
    c = filled(np.random.default_rng(32), [5, 6])
    cache = on_gpu(c)
    cache.truncate(ints([0, 7]), ints([9, 0]))
    with pytest.raises(RuntimeError, match="BAD_SEQUENCE, BAD_LENGTH"):
        cache.check()
    cache.check()


def test_offsets_beyond_32_bits():
    """Pages behind 4 GiB of keys, read and written."""
    from tensor_sharded_mlp_b200 import kv_cache
    r = np.random.default_rng(25)
    cache = kv_cache.KvCache8(2, 9000, 8, 128, page_size=256, max_seqs=2, max_tokens=2048)
    assert cache.k.numel() > 2 ** 32
    small = kv8.new_cache(1, 4, 8, 256, 128, 1, 4)
    n = 700
    cache.table[1, :3] = ints([8999, 8990, 8997])
    cache.refcount[[8999, 8990, 8997]] = 1
    cache.lengths[1] = n
    kv8.reserve(small, [0], [n])
    k, v = (torch.from_numpy(r.standard_normal((n, 8, 128)).astype(np.float32)).cuda() for _ in range(2))
    cache.append(1, k, v, ints([1]))
    kv8.append(small, 0, k.double().cpu().numpy(), v.double().cpu().numpy(), [0], [0, n])
    q = query(r, 1, 1, 16, 128, "f32")
    want, reach, vmax = kv8.attention(small, 0, q.double().cpu().numpy(), [0], 128 ** -0.5)
    got = cache.attention(1, q, ints([1]))
    rel = weight_bound(reach, 128, n, q.dtype)
    close(got, want, rel * vmax + HALF[q.dtype] * np.abs(want), "far pages")
    cache.check()


def test_step_and_merge_over_ranks():
    """A history cut over three ranks' caches, written by append: the ranks' partials, merged by
    tp_mlp_merge_attention_partials, are the attention over the whole; so is one cache that holds it all."""
    from tensor_sharded_mlp_b200 import binding, kv_cache
    r = np.random.default_rng(26)
    heads, hk, d, q_len = 8, 2, 128, 3
    lens = [200, 77, 5]
    cuts = [[0, 90, 128, 200], [0, 64, 77, 77], [0, 0, 2, 5]]
    parts, oracles = [], []
    data = [[torch.from_numpy(r.standard_normal((n, hk, d)).astype(np.float32)).cuda().bfloat16() for n in lens] for _ in range(2)]
    q = query(r, 3, q_len, heads, d, "f32")
    stacks = [torch.empty(3, 3 * q_len * heads, device="cuda"), torch.empty(3, 3 * q_len * heads, device="cuda"),
              torch.empty(3, 3 * q_len * heads, d, device="cuda")]
    for rank in range(3):
        counts = [cuts[s][rank + 1] - cuts[s][rank] for s in range(3)]
        cache = kv_cache.KvCache8(1, 16, hk, d, page_size=32, max_seqs=3, max_tokens=256)
        cache.reserve(None, ints(counts))
        k, v = (torch.cat([x[s][cuts[s][rank]:cuts[s][rank + 1]] for s in range(3)]) for x in data)
        cache.append(0, k, v, cu_tokens=ints(np.concatenate([[0], np.cumsum(counts)])))
        at = [lens[s] - q_len - cuts[s][rank] for s in range(3)]
        views = [t[rank].view(3, q_len, heads, *t.shape[2:]) for t in stacks]
        cache.attention_partials(0, q, positions=ints(at), maximum=views[0], exp_sum=views[1], weighted=views[2])
        cache.check()
        c = kv8.new_cache(1, 16, hk, 32, d, 3, 8)
        kv8.reserve(c, range(3), counts)
        kv8.append(c, 0, k.double().cpu().numpy(), v.double().cpu().numpy(), range(3), np.concatenate([[0], np.cumsum(counts)]))
        oracles.append(kv8.attention_partials(c, 0, q.double().cpu().numpy(), range(3), d ** -0.5, at))
    got = binding.tp_mlp_merge_attention_partials(*stacks).view(3, q_len, heads, d)
    top = np.max([o[0] for o in oracles], axis=0)
    seen = np.isfinite(top)
    safe = np.where(seen, top, 0.0)
    turn = [np.exp(o[0] - safe) for o in oracles]
    den = sum(t * o[1] for t, o in zip(turn, oracles))
    want = sum(t[..., None] * o[2] for t, o in zip(turn, oracles)) / np.where(den == 0, 1, den)[..., None]
    reach, vmax = max(o[3] for o in oracles), max(o[4] for o in oracles)
    rel = weight_bound(reach, d, 256, q.dtype)
    close(got, want, 4 * rel * vmax + HALF[q.dtype] * np.abs(want) + 1e-30, "merged ranks")


def test_generation_with_branches_in_a_graph():
    """Prompts written, branched, and grown token by token: reserve, append and attention captured once in a CUDA graph
    and replayed (a padded entry in the batch), then cut back, freed, compacted -- against the oracle at every step."""
    from tensor_sharded_mlp_b200 import kv_cache
    r = np.random.default_rng(27)
    layers, hk, d, heads, page = 2, 2, 64, 6, 16
    cache = kv_cache.KvCache8(layers, 64, hk, d, page_size=page, max_seqs=6, max_tokens=160)
    c = kv8.new_cache(layers, 64, hk, page, d, 6, 10)
    c["k_scale"][:], c["v_scale"][:] = 1, 1
    prompts = [37, 16]
    kv8.reserve(c, [0, 1], prompts)
    cache.reserve(ints([0, 1]), ints(prompts))
    cu = [0, 37, 53]
    for layer in range(layers):
        k, v = (torch.from_numpy(r.standard_normal((53, hk, d)).astype(np.float32)).cuda() for _ in range(2))
        cache.append(layer, k, v, ints([0, 1]), ints(cu))
        kv8.append(c, layer, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 1], cu)
    kv8.fork(c, [0, 0, 1], [2, 3, 4])
    cache.fork(ints([0, 0, 1]), ints([2, 3, 4]))
    seqs = [3, 0, -1, 2, 4, 1]
    listed, counts = ints(seqs), ints([1] * 6)
    ks, vs = (torch.zeros(layers, 6, hk, d, device="cuda") for _ in range(2))
    q = torch.zeros(layers, 6, 1, heads, d, device="cuda")
    outs = torch.zeros_like(q)

    def step():
        cache.reserve(listed, counts)
        for layer in range(layers):
            cache.append(layer, ks[layer], vs[layer], listed)
            cache.attention(layer, q[layer], listed, out=outs[layer])

    saved = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, cache.lengths, cache.refcount)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                         # warm-up; undone below
    torch.cuda.current_stream().wait_stream(side)
    for t, x in zip((cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, cache.lengths, cache.refcount), saved):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for it in range(20):
        for t in (ks, vs, q):
            t.copy_(torch.from_numpy(r.standard_normal(tuple(t.shape)).astype(np.float32) * 1.3 ** it))
        graph.replay()
        assert kv8.reserve(c, seqs, [1] * 6) == 0
        for layer in range(layers):
            kv8.append(c, layer, ks[layer].double().cpu().numpy(), vs[layer].double().cpu().numpy(), seqs, list(range(7)))
            qd = q[layer].double().cpu().numpy()
            want, reach, vmax = kv8.attention(c, layer, qd, seqs, d ** -0.5)
            rel = weight_bound(reach, d, 64, torch.float32)
            rows = [0, 1, 3, 4, 5]
            close(outs[layer][rows], want[rows], rel * vmax + HALF[torch.float32] * np.abs(want[rows]), f"step {it}")
            assert not outs[layer][2].bool().any()
        np.testing.assert_array_equal(cache.table.cpu().numpy(), c["table"])
        np.testing.assert_array_equal(cache.lengths.cpu().numpy(), c["lengths"])
    kv8.truncate(c, [3, 1], [40, 0])
    cache.truncate(ints([3, 1]), ints([40, 0]))
    np.testing.assert_array_equal(cache.compact().cpu().numpy(), kv8.compact(c))
    check(c, cache, query(r, 5, 2, heads, d, "bf16"), [0, 1, 2, 3, 4], layer=1)
    cache.check()


def test_workspace_and_buffers_are_checked():
    from tensor_sharded_mlp_b200 import binding as b
    cache = on_gpu(filled(np.random.default_rng(28), [5]))
    q = torch.zeros(1, 1, 2, 64, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    L, p = b._lib, b._ptr
    need = L.tp_mlp_kv8_attention_workspace_bytes(cache.c, 1, 1, 2)

    def call(c, ws_bytes, out=q):
        return L.tp_mlp_kv8_attention(c, 0, p(q), 128, None, None, 1, 1, 2, 1.0, 0, p(out), p(ws), ws_bytes, None)
    assert call(cache.c, need) == 0 and call(cache.c, need - 1) == 7
    big = b.Kv8Cache.from_buffer_copy(cache.c)
    big.layers = 1 << 24
    assert call(big, need) == 2
    host = torch.zeros(64, 64)
    bad = b.Kv8Cache.from_buffer_copy(cache.c)
    bad.k = host.data_ptr() & ~15
    assert call(bad, need) == 1
    torch.cuda.synchronize()
