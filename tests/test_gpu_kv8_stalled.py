"""The bounded waits of the many-rows attention kernel: one of its roles stops delivering at some tile, the others' waits
run out after 2 ms, every warp leaves, the tensor memory is given back and the status word says so; the next call's
results are right."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, flags, on_gpu

pytestmark = pytest.mark.gpu
TIMEOUT = 32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


@pytest.mark.parametrize("tile", [0, 1, 2, 5])
@pytest.mark.parametrize("role", [0, 1, 2])
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_a_role_that_stops(head_dim, role, tile):
    from tensor_sharded_mlp_b200 import binding as b
    r = np.random.default_rng(head_dim)
    cache = longer(on_gpu(filled(r, [3000, 1, 700, 2999], 1, 1, 64, head_dim)))
    q = torch.from_numpy(r.standard_normal((4, 16, 8, head_dim)).astype(np.float32)).cuda().bfloat16()
    want = cache.attention(0, q, scale=1.0)
    out = torch.full_like(q, 7.0)
    b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, q, out, role, tile, 2000)
    assert flags(cache) == TIMEOUT
    for _ in range(3):                                                  # TMEM is free again, the context healthy
        assert torch.equal(cache.attention(0, q, scale=1.0), want)
    # a tile that no CTA reaches: the call is an ordinary one
    b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, q, out, role, 100000, 100000)
    assert flags(cache) == 0 and torch.equal(out, want)


def longer(cache):
    """The same pages, listed 30 times over by every sequence."""
    from tensor_sharded_mlp_b200 import kv_cache
    rows = []
    for s in range(cache.table.shape[0]):
        held = cache.table[s][cache.table[s] >= 0]
        rows.append(held.repeat(30))
    table = torch.full((len(rows), max(map(len, rows))), -1, dtype=torch.int32, device="cuda")
    for s, row in enumerate(rows):
        table[s, :len(row)] = row
    lengths = torch.tensor([len(row) * 64 for row in rows], dtype=torch.int32, device="cuda")
    for t in (cache.k, cache.v):                                        # (the slots behind the old ends are read now)
        t[(t & 127) == 127] = 0
    return kv_cache.KvCache8.over(cache.k, cache.v, cache.k_scale, cache.v_scale, table, lengths, cache.refcount, cache.status)


def test_two_stalled_calls_and_a_graph():
    from tensor_sharded_mlp_b200 import binding as b
    r = np.random.default_rng(5)
    cache = longer(on_gpu(filled(r, [3000, 2000], 1, 2, 64, 128)))
    q = torch.from_numpy(r.standard_normal((2, 9, 16, 128)).astype(np.float32)).cuda().bfloat16()
    want, out = cache.attention(0, q, scale=1.0), torch.empty_like(q)
    for _ in range(2):
        b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, q, out, 1, 3, 2000)
        assert torch.equal(cache.attention(0, q, scale=1.0), want)
    assert flags(cache) == TIMEOUT
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, q, out, 0, 2, 2000)
        cache.attention(0, q, scale=1.0, out=out)
    for _ in range(2):
        graph.replay()
        assert flags(cache) == TIMEOUT and torch.equal(out, want)


def test_refusals():
    from tensor_sharded_mlp_b200 import binding as b
    cache = on_gpu(filled(np.random.default_rng(6), [100], kv_heads=1))
    q = torch.zeros(1, 70, 1, 64, device="cuda", dtype=torch.bfloat16)
    for role, tile, wait in ((-1, 0, 10), (3, 0, 10), (0, -1, 10), (0, 0, 0), (0, 0, 100001)):
        with pytest.raises(b.TpMlpError, match="INVALID_ARG"):
            b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, q, q.clone(), role, tile, wait)
    few = q[:, :4].contiguous()
    with pytest.raises(b.TpMlpError, match="UNSUPPORTED"):
        b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, few, few.clone(), 0, 0, 10)
    with pytest.raises(ValueError):
        b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, q.float(), q.float(), 0, 0, 10)
    assert flags(cache) == 0
