"""Forking with padded lists: a pair with a -1 is unused, whatever its other number."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, on_gpu
from test_gpu_kv8_pages import both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


@pytest.mark.parametrize("parents,children", [
    ([-1, 0], [2, 2]),                                                  # an unused pair in front names the child
    ([3, 0], [-1, 3]),                                                  # ... or has it as its parent
    ([0, -1, -1, 1], [2, 2, 3, 3]),
    ([-1, -1, 0, 0, 0], [2, 2, 2, 2, 3]),                               # the used ones' own repeat is still refused
    ([0, 2, 2], [2, -1, 3]),                                            # and so is a used parent
    ([-1, 9, 0], [4, -1, 4]), ([0, -9, 1], [2, 3, 3])])
def test_unused_pairs_count_for_nothing(parents, children):
    c = filled(np.random.default_rng(1), [20, 33, 0, 0, 0], spare=3)
    both(c, on_gpu(c), "fork", parents, children)


def test_padded_pairs_in_a_long_list():
    r = np.random.default_rng(2)
    n = 1024
    c = filled(r, [20] * 30 + [0] * 600, spare=3)
    parents = [int(x) if r.random() < 0.5 else -1 for x in r.integers(0, 30, n)]
    children = [int(x) for x in r.integers(28, 630, n)]
    both(c, on_gpu(c), "fork", parents, children)
