"""Appending prompts to the 8-bit cache where a CTA works through several units one after the other: more units than CTAs
are resident, runs that start in the middle of a slot, and slots without work (spare, empty, padded, shared, invalid)
between others, with odd and even numbers of KV heads.  Codes and scales bit for bit as the fp64 oracle's."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, flags, ints, on_gpu, same_pool
from oracle import kv8
from test_gpu_kv8_append import put, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


def resident(dtype):
    return torch.cuda.get_device_properties(0).multi_processor_count * (4 if dtype == "bf16" else 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv_heads,head_dim,page", [(1, 64, 16), (3, 64, 16), (5, 64, 32), (8, 128, 16)])
def test_ragged_prompts_over_many_units(kv_heads, head_dim, page, dtype):
    r = np.random.default_rng(kv_heads)
    n = -(-2 * resident(dtype) // (2 * kv_heads)) + 40                 # two spare slots an entry: units for two rounds and more
    n = min(n, 700)
    before = [int(x) if r.random() < 0.3 else 0 for x in r.integers(1, 2 * page, n)]
    new = [0 if r.random() < 0.15 else int(x) for x in r.integers(1, 4 * page + 20, n)]
    c = filled(r, before, 1, kv_heads, page, head_dim, spare=9 * n, max_pages=9)
    cache = on_gpu(c)
    assert kv8.reserve(c, range(n), new) == 0
    cache.reserve(None, ints(new))
    order = [int(x) for x in r.permutation(n)]
    cu = np.concatenate([[0], np.cumsum([new[s] for s in order])])
    slots = int(cu[-1]) // page + 2 * n
    assert slots * kv_heads > 1.5 * resident(dtype) and int(cu[-1]) // n * (head_dim // 8) > 128
    k, v = (x.clone() for x in rows(r, int(cu[-1]), kv_heads, head_dim, dtype))
    spread = torch.from_numpy(4.0 ** r.integers(-4, 5, len(k))).cuda().to(k.dtype)[:, None, None]
    k, v = k * spread, v * spread.flip(0)                               # neighbouring units' scales differ
    k[7::97, :, 3], v[5::89, -1, 5], v[40::131, 0] = float("nan"), float("inf"), float("-inf")
    listed = [-1 if r.random() < 0.1 else s for s in order]             # padded entries
    listed[3], listed[9] = listed[2], n + 5                             # one twice, one outside
    for _ in range(3):                                                  # (a call may be repeated)
        put(c, cache, 0, k.contiguous(), v.contiguous(), listed, cu)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv_heads", [1, 3, 8])
def test_shared_and_missing_pages_between_others(kv_heads, dtype):
    """Slots that a CTA finds shared or outside the pool are passed over; those around them are written."""
    r = np.random.default_rng(20 + kv_heads)
    n, page = 400 if kv_heads > 1 else 640, 16
    new = [int(x) for x in r.integers(17, 70, n)]
    c = filled(r, [0] * (n + 40), 1, kv_heads, page, 64, spare=6 * n, max_pages=6)
    cache = on_gpu(c)
    kv8.reserve(c, range(n), new)
    cache.reserve(None, ints(new + [0] * 40))
    parents = [int(x) for x in r.permutation(n)[:40]]
    assert kv8.fork(c, parents, list(range(n, n + 40))) == 0
    cache.fork(ints(parents), ints(range(n, n + 40)))
    for s in r.permutation(n)[:30]:
        b = int(r.integers(0, -(-new[s] // page)))
        if c["refcount"][c["table"][s, b]] == 1:
            c["table"][s, b] = [-1, len(c["refcount"])][int(r.integers(0, 2))]
    cache.table.copy_(ints(c["table"]))
    cu = np.concatenate([[0], np.cumsum(new)])
    k, v = rows(r, int(cu[-1]), kv_heads, 64, dtype)
    want = kv8.append(c, 0, k.double().cpu().numpy(), v.double().cpu().numpy(), list(range(n)), cu)
    assert want == kv8.SHARED_PAGE | kv8.BAD_PAGE
    cache.append(0, k, v, ints(range(n)), ints(cu))
    assert flags(cache) == want
    same_pool(cache, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_even_prompts_over_many_units(dtype):
    r = np.random.default_rng(30)
    n, each, kv_heads = 300, 50, 5                                      # pages of 16: 4 or 5 slots an entry
    before = [int(x) for x in r.integers(0, 30, n)]
    c = filled(r, before, 1, kv_heads, 16, 64, spare=5 * n, max_pages=8)
    cache = on_gpu(c)
    kv8.reserve(c, range(n), [each] * n)
    cache.reserve(None, ints([each] * n))
    k, v = rows(r, n * each, kv_heads, 64, dtype, 30.0)
    put(c, cache, 0, k, v, list(range(n)), np.arange(n + 1) * each, "all")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_runs_as_long_as_a_cta_can_hold(dtype):
    """So many slots that the number of CTAs comes from the slots that one can hold, not from what is resident."""
    r = np.random.default_rng(31)
    n = 1024
    least = 32 * resident(dtype) + 500                                  # slots
    each = (least - 2 * n) * 16 // n + 8
    new = [int(x) for x in r.integers(each - 40, each + 41, n)]
    c = filled(r, [0] * n, 1, 1, 16, 64, spare=sum(-(-x // 16) for x in new), max_pages=(each + 41) // 16 + 1)
    cache = on_gpu(c)
    kv8.reserve(c, range(n), new)
    cache.reserve(None, ints(new))
    cu = np.concatenate([[0], np.cumsum(new)])
    assert int(cu[-1]) // 16 + 2 * n > 32 * resident(dtype)
    k, v = rows(r, int(cu[-1]), 1, 64, dtype)
    put(c, cache, 0, k, v, list(range(n)), cu)


BOUNDS = [[-5, 3, 10, 30], [-40, -20, 12, 30], [0, 12, 5, 30], [0, 30, 10, 20], [4, 9, 20, 29], [0, 31, 31, 31], [-1, -1, -1, -1],
          [0, 10, 2 ** 31 - 1, 30], [-2 ** 31, 10, 20, 30], [30, 20, 10, 0], [0, 20, 19, 20], [31, 40, 50, 60]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu", BOUNDS)
def test_row_bounds_out_of_order(cu, dtype):
    """Each entry with wrong bounds is left out and flagged, wherever it stands; the others are written."""
    r = np.random.default_rng(32)
    c = filled(r, [33, 40, 37], 1, 3, 16, 64)
    cache = on_gpu(c)
    k, v = rows(r, 30, 3, 64, dtype)
    put(c, cache, 0, k, v, [2, 0, 1], cu)
    put(c, cache, 0, k, v, [-1, 1, 1], cu)                              # padded; one sequence twice
    put(c, cache, 0, k, v, [7, 0, -2], cu)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_bounds_out_of_order_in_long_lists(dtype):
    r = np.random.default_rng(33)
    n = 500
    new = [int(x) for x in r.integers(0, 60, n)]
    c = filled(r, [0] * n, 1, 1, 16, 64, spare=5 * n, max_pages=5)
    cache = on_gpu(c)
    kv8.reserve(c, range(n), new)
    cache.reserve(None, ints(new))
    cu = np.concatenate([[0], np.cumsum(new)])
    k, v = rows(r, int(cu[-1]) + 3, 1, 64, dtype)                       # (rows of no entry behind the last)
    for at, by in ((0, -70), (17, 1000), (40, -900), (333, 10 ** 7), (n, 4)):
        off = cu.copy()
        off[at] += by
        put(c, cache, 0, k, v, list(range(n)), off)


@pytest.mark.parametrize("each", [1, 40])
def test_entries_without_rows_are_checked_too(each):
    """A wrong sequence number or length is flagged though its entry has nothing to write."""
    r = np.random.default_rng(34)
    c = filled(r, [50, 60, 70, 17], 1, 3, 16, 64)
    cache = on_gpu(c)
    k, v = rows(r, 2 * each, 3, 64, "bf16")
    put(c, cache, 0, k, v, [0, 1, 0], [0, each, 2 * each, 2 * each])
    put(c, cache, 0, k, v, [4, 1, 0], [0, 0, each, 2 * each])
    put(c, cache, 0, k, v, [0, -9, 1], [0, each, each, 2 * each])
    put(c, cache, 0, k, v, [0, 3, -1, 1], [0, each, each, each, 2 * each])
    c["lengths"][3] = 10000
    cache.lengths[3] = 10000
    put(c, cache, 0, k, v, [0, 3, 1], [0, each, each, 2 * each])
    assert kv8.append(c, 0, np.zeros((0, 3, 64)), np.zeros((0, 3, 64)), [3], [0, 0]) == kv8.BAD_LENGTH
