"""Calls on the 8-bit cache with an explicit stream: their scratch and results are allocated on that stream, not in memory
that the current stream's queued work may still be using; stream objects of any kind; results that outlive their names."""
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


def freed(nbytes):
    """Addresses of a block of the current stream's pool that is free for the next request of its size there."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return t.data_ptr(), t.data_ptr() + nbytes


def outside(block, *tensors):
    return all(t.data_ptr() + t.numel() * t.element_size() <= block[0] or t.data_ptr() >= block[1] for t in tensors)


def setup(n=512):
    r = np.random.default_rng(1)
    cache = on_gpu(filled(r, [300, 20], 1, 2, 16, 128))
    q = torch.from_numpy(r.standard_normal((n, 1, 16, 128)).astype(np.float32)).cuda()     # 4 MiB
    return cache, q, ints([i % 2 for i in range(n)])


def test_memory_of_the_current_stream_is_not_taken(monkeypatch):
    from tensor_sharded_mlp_b200 import binding as b
    cache, q, seqs = setup()
    want = cache.attention(0, q, seqs)
    side = torch.cuda.Stream()
    taken = []
    scratch = b._scratch
    monkeypatch.setattr(b, "_scratch", lambda nbytes, stream: taken.append(scratch(nbytes, stream)) or taken[-1])
    for size in (q.numel() * 4, int(b._lib.tp_mlp_kv8_attention_workspace_bytes(cache.c, 1, 1, 16)), 512 * 16 * 4):
        for given in (side, side.cuda_stream, Foreign(side)):
            block = freed(size)
            out = cache.attention(0, q, seqs, stream=given)
            parts = cache.attention_partials(0, q, seqs, stream=given)
            index = cache.compact(stream=given)
            side.synchronize()
            assert len(taken) == 3 and outside(block, out, *parts, index, *taken)
            assert torch.equal(out, want)
            taken.clear()
            del out, parts, index


def test_results_are_kept_for_the_current_stream():
    """Dropped while the current stream still has work queued, a result's memory is not given to the next call."""
    cache, q, seqs = setup()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = cache.attention(0, q, seqs, stream=side)
    side.synchronize()
    want, copy, at, other = out.clone(), torch.empty_like(out), out.data_ptr(), -q
    torch.cuda._sleep(1000)                                             # (kernels are loaded before they are queued in earnest)
    copy.copy_(out)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                                      # about 0.1 s
    copy.copy_(out)
    copied = torch.cuda.Event()
    copied.record()
    del out
    later = [cache.attention(0, other, seqs, stream=side) for _ in range(3)]
    assert not copied.query()                                           # (else the test has shown nothing)
    assert all(t.data_ptr() != at for t in later)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


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
