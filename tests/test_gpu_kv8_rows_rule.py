"""Attention with 33 to 64 query rows a KV head, which either kernel may take: by head_dim, rows and the tokens that the
cache lets a call see.  The same history in a small and in a large pool, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, on_gpu
from test_gpu_kv8_attention import check, query

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


def takes_many_rows(cache, q):
    """Which kernel a call takes: the self-test of the many-rows one refuses the others' calls."""
    from tensor_sharded_mlp_b200 import binding as b
    try:
        b.tp_mlp_kv8_selftest_stalled_attention(cache.c, 0, q, torch.empty_like(q), 0, 1 << 20, 100000)
    except b.TpMlpError as e:
        assert e.name == "ERR_UNSUPPORTED"
        return False
    return True


# head_dim, q_len, group, whether the large pool's call takes the kernel for many rows (the small one's never does)
CASES = [(256, 4, 8, False), (256, 11, 3, True), (256, 5, 8, True), (256, 64, 1, True), (256, 1, 64, True), (128, 6, 8, False),
         (128, 7, 7, True), (128, 8, 8, True), (64, 8, 8, False)]


@pytest.mark.parametrize("head_dim,q_len,group,many", CASES)
def test_either_kernel(head_dim, q_len, group, many):
    r = np.random.default_rng(head_dim + q_len)
    kv_heads, page = 4, 256
    lengths = [700, 1, 0, 257, 33, 300]
    large = -(-(1 << 18) // (kv_heads * page))                          # pages in all
    for spare, room in ((4, 6), (large, large // 6 + 1)):
        c = filled(np.random.default_rng(7), lengths, 1, kv_heads, page, head_dim, spare=spare, max_pages=room)
        cache = on_gpu(c)
        q = query(r, 6, q_len, kv_heads * group, head_dim, "bf16")
        assert takes_many_rows(cache, q) == (many and spare == large)
        check(c, cache, q, [3, 0, 5, 1, 2, 4])
        check(c, cache, query(r, 6, q_len, kv_heads * group, head_dim, "f32"), [5, 4, 3, 2, 1, 0])


def test_one_cache_both_ways():
    """Fewer entries of the same cache: the bound of their tokens decides, and one workspace size serves both."""
    r = np.random.default_rng(3)
    c = filled(r, [300] * 8, 1, 1, 256, 256, spare=1100, max_pages=200)
    cache = on_gpu(c)
    for n, many in ((1, False), (5, False), (6, True), (8, True), (2, False)):
        q = query(r, n, 8, 8, 256, "bf16")
        assert takes_many_rows(cache, q) == many
        check(c, cache, q, list(range(n)))
