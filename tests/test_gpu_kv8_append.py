"""Quantising new rows into the pages of the 8-bit cache: codes and scales bit for bit as the fp64 oracle's."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, flags, ints, on_gpu, same_map, same_pool
from oracle import kv8

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


def rows(r, n, heads, d, dtype, spread=1.0):
    """(n, heads, d) on the GPU: columns of a wider projection, and the same numbers for the oracle."""
    wide = torch.from_numpy((r.standard_normal((n, 3 * heads * d)) * spread).astype(np.float32)).cuda().to(TORCH[dtype])
    k, v = (wide[:, x * heads * d:(x + 1) * heads * d].unflatten(1, (heads, d)) for x in (0, 2))
    return k, v


def f64(t):
    return t.double().cpu().numpy()


def put(c, cache, layer, k, v, seqs, cu, given="cu"):
    want = kv8.append(c, layer, f64(k), f64(v), seqs, cu)
    if given == "cu":
        cache.append(layer, k, v, ints(seqs), ints(cu))
    elif given == "even":
        cache.append(layer, k, v, ints(seqs))
    else:
        cache.append(layer, k, v, n=len(seqs))
    assert flags(cache) == want
    same_pool(cache, c)
    same_map(cache, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,kv_heads,head_dim", [(16, 2, 64), (64, 8, 128), (32, 1, 256), (128, 3, 64), (256, 2, 128)])
def test_prompts_of_mixed_lengths(page, kv_heads, head_dim, dtype):
    r = np.random.default_rng(page + kv_heads)
    before = [0, 3, page - 1, page, 0, 2 * page + 5, 0]
    new = [5, page, 2, 2 * page + 1, 0, 1, page]
    c = filled(r, before, 2, kv_heads, page, head_dim, spare=20, max_pages=8)
    cache = on_gpu(c)
    seqs = [6, 1, 0, 3, 4, 2, 5]
    counts = [new[s] for s in seqs]
    assert kv8.reserve(c, seqs, counts) == 0
    cache.reserve(ints(seqs), ints(counts))
    cu = np.concatenate([[0], np.cumsum(counts)])
    for layer in (1, 0):
        k, v = rows(r, int(cu[-1]), kv_heads, head_dim, dtype, spread=10.0 ** layer)
        put(c, cache, layer, k, v, seqs, cu)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("each", [1, 2, 3, 17, 40])
def test_even_rows_step_by_step(each, dtype):
    """Generation: the same sequences grow, their last pages' scales with them."""
    r = np.random.default_rng(each)
    c = filled(r, [0, 15, 16, 30], spare=60, max_pages=16, kv_heads=3)
    cache = on_gpu(c)
    for step in range(4):
        assert kv8.reserve(c, range(4), [each] * 4) == 0
        cache.reserve(None, ints([each] * 4))
        k, v = rows(r, 4 * each, 3, 64, dtype, spread=4.0 ** (step - 1))
        put(c, cache, 0, k, v, list(range(4)), np.arange(5) * each, "even" if step % 2 else "all")


def test_extreme_values():
    r = np.random.default_rng(1)
    c = filled(r, [0, 7, 0, 0, 5], spare=10)
    cache = on_gpu(c)
    kv8.reserve(c, range(5), [3] * 5)
    cache.reserve(None, ints([3] * 5))
    k, v = (x.clone().contiguous() for x in rows(r, 15, 2, 64, "f32"))
    k[0:3] = 0                                                         # nothing: the smallest scale
    k[3:6] *= 1e30
    k[6] = float("nan")
    k[7, 0, 3], k[7, 1, 5], k[8, 0, 1] = float("inf"), float("-inf"), float("nan")
    k[9:12] = 1e-42                                                    # subnormal in fp32
    k[9, 0, 0] = -3.4e38
    v[0:3] = float("inf")                                              # no finite value in a page
    v[3:6, :, ::2] *= 1e-20
    v[12:15] = 448.0 * 2.0 ** -7                                       # on the border of a scale
    v[14, 1, 63] = float(np.nextafter(np.float32(448.0 * 2.0 ** -7), np.float32(10)))
    put(c, cache, 0, k, v, list(range(5)), np.arange(6) * 3)


def test_ties_and_every_code():
    """Values on e4m3 numbers and half-way between two: ties to even, both signs."""
    grid = np.concatenate([kv8._POS, (kv8._POS[1:] + kv8._POS[:-1]) / 2])
    x = np.zeros(512)
    x[:253], x[253:506] = grid[:253], -grid[:253]
    x[511] = 448.0                                                     # scale 1
    c = filled(np.random.default_rng(0), [0], kv_heads=1, head_dim=64, spare=2)
    cache = on_gpu(c)
    kv8.reserve(c, [0], [8])
    cache.reserve(None, ints([8]))
    for dtype in ("f32", "bf16"):
        t = torch.from_numpy(x.astype(np.float32)).cuda().to(TORCH[dtype]).view(8, 1, 64)
        assert (f64(t).ravel() == x).all()
        put(c, cache, 0, t, t.clone(), [0], [0, 8])


def test_repeated_call_changes_nothing():
    r = np.random.default_rng(2)
    c = filled(r, [9, 0, 33], spare=8)
    cache = on_gpu(c)
    kv8.reserve(c, range(3), [4] * 3)
    cache.reserve(None, ints([4] * 3))
    k, v = rows(r, 12, 2, 64, "bf16", 50.0)
    put(c, cache, 0, k, v, [0, 1, 2], [0, 4, 8, 12])
    cache.append(0, k, v, ints([0, 1, 2]), ints([0, 4, 8, 12]))
    same_pool(cache, c)


def test_padded_repeated_and_invalid_entries():
    r = np.random.default_rng(3)
    c = filled(r, [20, 5, 0, 40, 3], spare=6)
    cache = on_gpu(c)
    k, v = rows(r, 14, 2, 64, "bf16")
    # unused, repeated, outside, more rows than the sequence has tokens
    put(c, cache, 0, k, v, [0, -1, 0, 9, 1, -3, 4], [0, 2, 4, 6, 8, 10, 12, 14])
    put(c, cache, 0, k, v, [0, 2, 4], [0, 2, 4, 14])
    # shared pages and pages outside the pool
    kv8.fork(c, [3], [2])
    cache.fork(ints([3]), ints([2]))
    put(c, cache, 0, k, v, [3, 4, 0], [0, 10, 12, 14])
    c["table"][0, 1] = len(c["refcount"])
    cache.table[0, 1] = len(c["refcount"])
    put(c, cache, 0, k, v, [0, 1], [0, 12, 14])
    # row bounds outside the input
    put(c, cache, 0, k, v, [1, 4], [0, 3, 15])


def test_empty_calls():
    c = filled(np.random.default_rng(4), [5])
    cache = on_gpu(c)
    z = torch.zeros(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    cache.append(0, z, z, ints([0]), ints([0, 0]))
    cache.append(0, z, z, ints([]), ints([0]))
    same_pool(cache, c)


def test_many_sequences_in_one_call():
    r = np.random.default_rng(5)
    n = 1024
    before = [int(x) for x in r.integers(0, 40, n)]
    c = filled(r, before, kv_heads=1, spare=2100, max_pages=6)
    cache = on_gpu(c)
    new = [int(x) for x in r.integers(0, 20, n)]
    order = [int(x) for x in r.permutation(n)]
    counts = [new[s] for s in order]
    kv8.reserve(c, order, counts)
    cache.reserve(ints(order), ints(counts))
    cu = np.concatenate([[0], np.cumsum(counts)])
    k, v = rows(r, int(cu[-1]), 1, 64, "bf16")
    put(c, cache, 0, k, v, order, cu)


def test_wrapper_refuses_wrong_shapes():
    cache = on_gpu(filled(np.random.default_rng(6), [5, 6]))
    k = torch.zeros(2, 2, 64, device="cuda")
    for a, b in ((k, k.bfloat16()), (k, k[:1]), (k[..., :32], k[..., :32]), (k.half(), k.half()), (k.cpu(), k.cpu()),
                 (k.transpose(0, 1), k.transpose(0, 1))):
        with pytest.raises(ValueError):
            cache.append(0, a, b)
    with pytest.raises(ValueError):
        cache.append(0, k, k, ints([0, 1]), ints([0, 2]))
    with pytest.raises(ValueError):
        cache.append(0, k, k, torch.zeros(2, dtype=torch.int64, device="cuda"))
