"""Calls on the 8-bit cache with an explicit stream: stream objects of any kind."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, ints, on_gpu, same_map, same_pool
from oracle import kv8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


class Foreign:
    """A stream object that is not torch's."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


def test_every_call_takes_any_kind_of_stream():
    r = np.random.default_rng(2)
    c = filled(r, [21, 5, 0, 0], 2, 2, 16, 64, spare=9)
    cache = on_gpu(c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    k, v = (torch.from_numpy(r.standard_normal((3, 2, 64)).astype(np.float32)).cuda() for _ in range(2))
    one, two, zero, counts = ints([0]), ints([2]), ints([1, 2]), ints([2, 1])
    listed, pairs = ints([0, 2]), ints([(3, 4)])
    cu, cut = ints([0, 2, 3]), ints([4, 3])
    torch.cuda.synchronize()
    for given in (Foreign(side), side.cuda_stream, side):
        cache.fork(one, two, stream=given)
        cache.reserve(listed, counts, stream=given)
        cache.append(1, k, v, listed, cu, stream=given)
        cache.truncate(zero, cut, stream=given)
        cache.copy_pages(pairs, stream=given)
        cache.truncate(two, stream=given)
        index = cache.compact(stream=given)
        side.synchronize()
        kv8.fork(c, [0], [2])
        kv8.reserve(c, [0, 2], [2, 1])
        kv8.append(c, 1, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 2], [0, 2, 3])
        kv8.truncate(c, [1, 2], [4, 3])
        kv8.copy_pages(c, [(3, 4)])
        kv8.truncate(c, [2])
        np.testing.assert_array_equal(index.cpu().numpy(), kv8.compact(c))
        same_map(cache, c)
        same_pool(cache, c)
        cache.check()
