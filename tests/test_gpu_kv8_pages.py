"""Page work of the paged 8-bit cache on the GPU: every result equal, bit for bit, to the fp64 oracle's
one-entry-at-a-time walk -- reserve (with copy on write), fork, truncate, copy and compact, alone and in long
random runs, with padded, repeated and invalid entries, exhausted pools and pools of many pages."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, flags, ints, on_gpu, same_map, same_pool
from oracle import kv8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


def both(c, cache, what, seqs, *lists):
    """One call on the oracle and on the GPU; maps, pools and flags must agree."""
    want = getattr(kv8, what)(c, list(seqs), *[list(x) for x in lists])
    getattr(cache, what)(ints(seqs), *[ints(x) for x in lists])
    assert flags(cache) == want, what
    same_map(cache, c, what)
    same_pool(cache, c, what)


@pytest.mark.parametrize("layers,kv_heads,page,head_dim", [(1, 1, 16, 64), (2, 3, 32, 64), (1, 2, 64, 128), (3, 1, 16, 256),
                                                           (1, 5, 128, 128), (1, 1, 256, 64)])
def test_reserve_and_fork_with_copy_on_write(layers, kv_heads, page, head_dim):
    r = np.random.default_rng(page + head_dim)
    lengths = [0, 1, page - 1, page, page + 1, 3 * page + 7, 0, 0, 0, 0, 0]
    c = filled(r, lengths, layers, kv_heads, page, head_dim, spare=20)
    cache = on_gpu(c)
    both(c, cache, "fork", [5, 5, 1, -1, 3], [6, 7, 8, 9, 10])
    both(c, cache, "reserve", [7, 8, 5, -1, 1], [1, page, 2, 9, 0])     # 6, a holder of 5's last page, is not here
    both(c, cache, "reserve", [10, 6, 8, 0], [1, 1, 1, 2 * page + 1])
    both(c, cache, "truncate", [5, 7, -1, 8], [2 * page + 3, 0, 5, 1])
    both(c, cache, "reserve", [5, 8], [page, page])


def test_all_holders_in_one_list_keep_one_page():
    r = np.random.default_rng(3)
    c = filled(r, [21, 0, 0, 0], spare=6)
    cache = on_gpu(c)
    both(c, cache, "fork", [0, 0, 0], [1, 2, 3])
    both(c, cache, "reserve", [2, 0, 3, 1], [1, 1, 1, 1])
    assert int((c["refcount"] == 1).sum()) == 4                         # four last pages, one of them the old one


def test_too_few_pages_change_nothing():
    r = np.random.default_rng(4)
    c = filled(r, [21, 16, 0], spare=2, max_pages=8)
    cache = on_gpu(c)
    both(c, cache, "fork", [0], [2])
    both(c, cache, "reserve", [0, 1], [1, 32])                          # a copy and two pages of two
    both(c, cache, "reserve", [0, 1], [1, 16])
    both(c, cache, "reserve", [2, 1], [1, 0])                           # the pool is full; both entries fit all the same


def test_invalid_entries_are_left_out():
    r = np.random.default_rng(5)
    c = filled(r, [5, 40, 0, 9], spare=8, max_pages=4)
    cache = on_gpu(c)
    both(c, cache, "reserve", [0, 0, 4, -2, 2, 3], [1, 5, 1, 1, 65, -1])
    both(c, cache, "truncate", [1, 1, 99, 3], [20, 0, 0, 10])
    both(c, cache, "fork", [0, 0, 1, 7, 3, 2], [2, 2, 1, 2, 0, 3])
    both(c, cache, "truncate", [2, 2])
    # a table entry outside the pool under the next token: that entry alone is left out
    c["table"][3, 0] = 1000
    cache.table[3, 0] = 1000
    both(c, cache, "reserve", [3, 1], [1, 1])


def test_a_child_may_not_be_a_parent_of_the_same_list():
    r = np.random.default_rng(6)
    c = filled(r, [20, 0, 0, 0], spare=3)
    cache = on_gpu(c)
    both(c, cache, "fork", [0, 1, 3], [1, 2, 3])


def test_copy_pages():
    r = np.random.default_rng(7)
    c = filled(r, [100, 50], layers=2, spare=10)
    cache = on_gpu(c)
    n = len(c["refcount"])
    for pairs in ([(0, 1), (2, 3)], [(0, 4), (4, 5), (1, 4), (6, 7)], [(0, 1), (2, 1), (-1, 3), (3, -1), (5, 5)],
                  [(n, 0), (0, n), (1, 2)], [(0, x) for x in range(1, n)]):
        want = kv8.copy_pages(c, pairs)
        cache.copy_pages(ints(pairs))
        assert flags(cache) == want
        same_pool(cache, c, str(pairs[:3]))
    same_map(cache, c)


@pytest.mark.parametrize("layers,kv_heads,page,head_dim", [(1, 1, 16, 64), (3, 2, 32, 128), (2, 5, 64, 64)])
def test_compact(layers, kv_heads, page, head_dim):
    r = np.random.default_rng(8)
    c = filled(r, list(r.integers(0, 6 * page, 12)), layers, kv_heads, page, head_dim, spare=9)
    cache = on_gpu(c)
    for gone in ([1, 4, 7], [], [0, 2, 3, 5, 6], [8, 9, 10, 11]):
        if gone:
            both(c, cache, "truncate", gone)
        want = kv8.compact(c)
        got = cache.compact()
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        same_map(cache, c)
        same_pool(cache, c)
        assert flags(cache) == 0


@pytest.mark.parametrize("pages", [1, 2, 127, 128, 129, 4093, 33000, 200001])
def test_pools_of_many_pages(pages):
    """Ranks of free pages over every span of the map kernels, ragged ends among them."""
    r = np.random.default_rng(pages)
    c = kv8.new_cache(1, pages, 1, 16, 64, 600, 300)
    held = r.permutation(pages)[:min(pages * 2 // 3, 100000)]
    at = 0
    for s in range(500):
        n = min(int(r.integers(0, 290)), len(held) - at)
        c["table"][s, :n] = held[at:at + n]
        c["lengths"][s] = n * 16
        at += n
    c["refcount"][held[:at]] = 1
    cache = on_gpu(c)
    gone = [s for s in range(500) if r.random() < 0.5]
    both(c, cache, "truncate", gone)
    both(c, cache, "reserve", list(range(500, 600)), [int(x) for x in r.integers(0, 40, 100)])
    want = kv8.compact(c)
    np.testing.assert_array_equal(cache.compact().cpu().numpy(), want)
    same_map(cache, c)
    both(c, cache, "reserve", [599, 500, 501], [1, 17, 0])


def test_longest_lists():
    r = np.random.default_rng(9)
    c = filled(r, [20] * 300 + [0] * 724, spare=1100)
    cache = on_gpu(c)
    both(c, cache, "fork", [i % 300 for i in range(724)], list(range(300, 1024)))
    order = [int(x) for x in r.permutation(1024)]
    both(c, cache, "reserve", order, [int(x) for x in r.integers(0, 2, 1024)])
    both(c, cache, "truncate", order[:1000])


@pytest.mark.parametrize("seed", range(6))
def test_random_runs(seed):
    r = np.random.default_rng(100 + seed)
    seqs = 12
    c = kv8.new_cache(2, 60, 2, 16, 64, seqs, 9)
    for n in ("k", "v"):
        c[n][:] = r.integers(0, 256, c[n].shape)
        c[n + "_scale"][:] = 2.0 ** r.integers(-5, 5, c[n + "_scale"].shape)
    cache = on_gpu(c)
    for _ in range(30):
        n = int(r.integers(1, 8))
        pick = [int(x) for x in r.integers(-1, seqs, n)]
        what = r.choice(["reserve", "reserve", "fork", "truncate", "compact"])
        if what == "reserve":
            both(c, cache, "reserve", pick, [int(x) for x in r.integers(0, 40, n)])
        elif what == "fork":
            both(c, cache, "fork", pick, [int(x) for x in r.integers(-1, seqs, n)])
        elif what == "truncate":
            both(c, cache, "truncate", pick, [int(x) for x in r.integers(0, 60, n)])
        else:
            np.testing.assert_array_equal(cache.compact().cpu().numpy(), kv8.compact(c))
            same_map(cache, c)
            same_pool(cache, c)
    assert (c["refcount"] >= 0).all() and (c["refcount"][c["table"][c["table"] >= 0]] > 0).all()


def test_offsets_beyond_32_bits():
    """A pool of more than 4 GiB for keys alone: pages at its far end are copied whole."""
    from tensor_sharded_mlp_b200 import kv_cache
    cache = kv_cache.KvCache8(3, 5500, 8, 128, page_size=256, max_seqs=4, max_tokens=1024)
    assert cache.k.numel() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (cache.k, cache.v):
        t[:, 5498] = torch.randint(0, 127, t[:, 5498].shape, generator=g, device="cuda", dtype=torch.uint8)
    cache.k_scale[:, 5498], cache.v_scale[:, 5498] = 4.0, 0.5
    cache.copy_pages(ints([(5498, 5499), (5498, 7)]))
    cache.check()
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        assert torch.equal(t[:, 5498], t[:, 5499]) and torch.equal(t[:, 5498], t[:, 7])
        assert torch.equal(t[:, 6], t[:, 8]) and not torch.equal(t[:, 6], t[:, 7])


def test_workspace_and_buffers_are_checked():
    from tensor_sharded_mlp_b200 import binding as b
    c = filled(np.random.default_rng(1), [5], spare=3)
    cache = on_gpu(c)
    lists, ws = ints([0]), torch.empty(16, dtype=torch.uint8, device="cuda")
    L, p = b._lib, b._ptr
    assert L.tp_mlp_kv8_reserve(cache.c, p(lists), p(lists), 1, p(ws), 16, None) == 7
    assert L.tp_mlp_kv8_compact(cache.c, None, p(ws), 16, None) == 7
    big = b.Kv8Cache.from_buffer_copy(cache.c)
    big.num_pages = 1 << 28                                             # claims more than its allocations hold
    assert L.tp_mlp_kv8_copy_pages(big, p(lists), 1, None) == 2
    torch.cuda.synchronize()
    same_map(cache, c)
