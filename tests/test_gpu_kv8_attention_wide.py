"""Attention over the paged 8-bit cache with many query rows for each KV head (a prompt's chunk on its history), which a
kernel of its own takes, against the fp64 oracle and within the bounds of kv8_helpers."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, flags, ints, on_gpu
from oracle import kv8
from test_gpu_kv8_attention import check, query

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


@pytest.mark.parametrize("head_dim", [64, 128, 256])
@pytest.mark.parametrize("q_len,kv_heads,group", [(66, 1, 1), (9, 2, 8), (16, 1, 8), (43, 1, 3), (128, 2, 2), (3, 1, 25), (1, 1, 100)])
def test_rows_and_lengths(q_len, kv_heads, group, head_dim):
    """One row tile and several, whole and ragged; sequences shorter than the queries, and tiles that end anywhere."""
    r = np.random.default_rng(q_len + head_dim)
    lengths = [0, 1, q_len - 1, q_len, 63, 64, 65, 127, 128, 129, 300, 700]
    c = filled(r, lengths, 1, kv_heads, {64: 16, 128: 64, 256: 32}[head_dim], head_dim)
    seqs = [int(x) for x in r.permutation(len(lengths))]
    check(c, on_gpu(c), query(r, len(seqs), q_len, kv_heads * group, head_dim, "bf16"), seqs)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes_and_layers(page):
    r = np.random.default_rng(page + 1)
    c = filled(r, [3, page - 1, page, page + 1, 2 * page + 9, 700], 2, 2, page, 128)
    cache = on_gpu(c)
    for layer in range(2):
        check(c, cache, query(r, 6, 17, 8, 128, "bf16"), [5, 4, 3, 2, 1, 0], layer=layer)


@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_long_sequences_over_every_sm(head_dim):
    r = np.random.default_rng(40)
    c = filled(r, [21000, 5, 4096, 1], 1, 1, 64, head_dim)
    check(c, on_gpu(c), query(r, 5, 33, 4, head_dim, "bf16"), [3, 0, 2, 1, 2])


def test_many_short_segments_beside_a_long_one():
    r = np.random.default_rng(41)
    lengths = [int(x) for x in r.integers(0, 40, 120)] + [5000] + [int(x) for x in r.integers(0, 300, 60)]
    c = filled(r, lengths, 1, 2, 16, 64)
    check(c, on_gpu(c), query(r, len(lengths), 12, 12, 64, "bf16"), list(range(len(lengths))))


def test_the_longest_list():
    r = np.random.default_rng(42)
    c = filled(r, [int(x) for x in r.integers(0, 40, 16)], 1, 1, 16, 256)
    seqs = [int(x) for x in r.integers(0, 16, 1024)]
    check(c, on_gpu(c), query(r, 1024, 9, 8, 256, "bf16"), seqs)


def test_ranks_positions():
    r = np.random.default_rng(43)
    lengths = [64, 64, 64, 64, 130, 130, 0, 64]
    c = filled(r, lengths, 1, 2, 16, 64)
    positions = [1000, 62, -1, -14, 29, 2 ** 31 - 1, 5, -2 ** 31]
    check(c, on_gpu(c), query(r, 8, 24, 6, 64, "bf16"), list(range(8)), positions=positions)


def test_rising_scores_and_peaked_rows():
    """Keys in rising order of score: the reference moves in most tiles, and the outputs so far are rescaled."""
    r = np.random.default_rng(44)
    c = filled(r, [777], 1, 1, 32, 128, spread=3.0)
    q = query(r, 1, 17, 4, 128, "bf16", 20.0)
    check(c, on_gpu(c), q, [0], scale=0.02)
    order = np.argsort(kv8.dense(c, 0, 0, 777)[0][0] @ q[0, 16, 0].double().cpu().numpy())
    k = kv8.dense(c, 0, 0, 777)[0].transpose(1, 0, 2)[order].astype(np.float32).astype(np.float64)
    up = kv8.new_cache(1, 30, 1, 32, 128, 1, 30)
    kv8.reserve(up, [0], [777])
    kv8.append(up, 0, k, k, [0], [0, 777])
    check(up, on_gpu(up), q, [0], scale=0.05)


@pytest.mark.parametrize("head_dim", [64, 256])
def test_nan_reaches_only_the_rows_that_see_it(head_dim):
    r = np.random.default_rng(45)
    c = filled(r, [140, 150, 145], 1, 1, 16, head_dim)
    c["v"][0, c["table"][0, 8], 0, 5, 9] = 0x7F                        # token 133 of 140
    c["v"][0, c["table"][0, 8], 0, 6, head_dim - 1] = 0xFF             # token 134
    c["k"][0, c["table"][1, 9], 0, 0, 3] = 0xFF                        # token 144 of 150
    c["v"][0, c["table"][2, 0], 0, 2, 63] = 0xFF                       # token 2: every query
    cache = on_gpu(c)
    q = query(r, 3, 40, 2, head_dim, "bf16")
    check(c, cache, q, [0, 1, 2])
    out = cache.attention(0, q, ints([0, 1, 2])).float()
    assert torch.isfinite(out[0, :33]).all() and torch.isnan(out[0, 33:, :, 9]).all()
    assert torch.isfinite(out[0, 33]).sum() == 2 * (head_dim - 1) and torch.isnan(out[0, 34:, :, head_dim - 1]).all()
    assert torch.isfinite(out[1, :34]).all() and torch.isnan(out[1, 34:]).all()
    assert torch.isnan(out[2, :, :, 63]).all() and torch.isfinite(out[2, :, :, :63]).all()


def test_nan_and_infinite_queries_stay_in_their_rows():
    r = np.random.default_rng(46)
    c = filled(r, [140, 300], 1, 2, 16, 64)
    q = query(r, 2, 20, 8, 64, "bf16")
    q[0, 1, 3, 7] = float("nan")
    q[1, 19, 5, 0] = float("inf")
    out = on_gpu(c).attention(0, q, ints([0, 1])).float()
    bad = torch.isnan(out).all(-1)
    want = torch.zeros_like(bad)
    want[0, 1, 3], want[1, 19, 5] = True, True
    assert torch.equal(bad, want) and torch.isfinite(out[~want]).all()


@pytest.mark.parametrize("stale", [0x7F, 0xFF, 0x7E])
def test_garbage_behind_the_end(stale):
    r = np.random.default_rng(47)
    c = filled(r, [1, 13, 100, 130], 1, 2, 64, 128, stale=stale)
    check(c, on_gpu(c), query(r, 4, 12, 16, 128, "bf16"), [0, 1, 2, 3])


def test_padded_repeated_and_invalid_entries():
    r = np.random.default_rng(48)
    c = filled(r, [140, 7, 100], 1, 2, 16, 64)
    cache = on_gpu(c)
    check(c, cache, query(r, 7, 20, 8, 64, "bf16"), [2, -1, 0, 2, 2, 1, -1])
    assert flags(cache) == 0
    check(c, cache, query(r, 5, 20, 8, 64, "bf16"), [2, 3, 0, -7, 1])
    assert flags(cache) == kv8.BAD_SEQUENCE
    c["table"][0, 1], c["table"][2, 4] = -1, len(c["refcount"])         # keys of such pages count as unseen
    cache = on_gpu(c)
    check(c, cache, query(r, 3, 20, 8, 64, "bf16"), [2, 1, 0])
    assert flags(cache) == kv8.BAD_PAGE


def test_pages_of_very_different_scales_and_zeros():
    r = np.random.default_rng(49)
    c = filled(r, [300, 140], 1, 2, 16, 64)
    c["v_scale"][0] *= 2.0 ** r.integers(-30, 20, c["v_scale"][0].shape)
    c["v_scale"][0, c["table"][1, 2]] = 0.0
    check(c, on_gpu(c), query(r, 2, 20, 8, 64, "bf16"), [0, 1])


def test_strided_queries():
    r = np.random.default_rng(50)
    c = filled(r, [140, 30], 1, 2, 16, 64)
    cache = on_gpu(c)
    wide = query(r, 2, 20, 24, 64, "bf16")
    out = cache.attention(0, wide[:, :, 8:16], ints([0, 1]))
    assert torch.equal(out, cache.attention(0, wide[:, :, 8:16].contiguous(), ints([0, 1])))


def test_same_result_in_graphs_and_on_another_stream():
    """Two captured calls that replay in turn, each with its own workspace, and an eager call between them."""
    r = np.random.default_rng(51)
    c = filled(r, [3000, 77, 500], 1, 2, 64, 128)
    cache = on_gpu(c)
    q = query(r, 3, 18, 16, 128, "bf16")
    want = cache.attention(0, q, ints([0, 1, 2]))
    seqs = ints([0, 1, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = cache.attention(0, q, seqs, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    outs, graphs = [torch.zeros_like(q) for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            cache.attention(0, q, seqs, out=o)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
            assert torch.equal(cache.attention(0, q, seqs), want)
            torch.cuda.synchronize()
            assert torch.equal(o, want)
    assert flags(cache) == 0


def test_workspace_of_both_kernels():
    from tensor_sharded_mlp_b200 import binding as b
    cache = on_gpu(filled(np.random.default_rng(52), [200]))
    L, p = b._lib, b._ptr
    few, many = (L.tp_mlp_kv8_attention_workspace_bytes(cache.c, 1, n, 2) for n in (1, 65))
    assert 0 < few < many < 64 << 20
    q = torch.zeros(1, 65, 2, 64, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(many, dtype=torch.uint8, device="cuda")

    def call(ws_bytes):
        return L.tp_mlp_kv8_attention(cache.c, 0, p(q), 128, None, None, 1, 65, 2, 1.0, 1, p(q), p(ws), ws_bytes, None)
    assert call(many - 1) == 7 and call(few) == 7
    torch.cuda.synchronize()
