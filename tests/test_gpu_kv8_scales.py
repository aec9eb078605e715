"""Attention over pages whose value scales lie anywhere in what append writes, 2^-100 (pages of zeros) to 2^120 (values near
fp32's largest), mixed in one history: against the fp64 oracle and within the bounds of kv8_helpers."""
import numpy as np
import pytest
import torch

from kv8_helpers import filled, on_gpu
from oracle import kv8
from test_gpu_kv8_attention import check, query

pytestmark = pytest.mark.gpu
SHAPES = [("bf16", 64, 1, 4), ("bf16", 128, 2, 8), ("bf16", 256, 1, 4), ("f32", 64, 1, 4), ("f32", 128, 2, 8), ("f32", 256, 1, 4),
          ("f32", 64, 5, 6), ("bf16", 64, 9, 8), ("bf16", 128, 9, 8), ("bf16", 256, 9, 8)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


@pytest.mark.parametrize("dtype,head_dim,q_len,heads", SHAPES)
@pytest.mark.parametrize("log", [60, 92, 108])
def test_zero_pages_beside_pages_of_large_values(log, dtype, head_dim, q_len, heads):
    """The two kinds' references are up to 210 binades apart; the zeros' weights count in every sum all the same."""
    r = np.random.default_rng(log + head_dim)
    for first in (0, 1, 2):                                             # zeros in every second page, or first, or last
        c = filled(r, [700, 90], 1, 1, 16, head_dim)
        for s in range(2):
            pages = c["table"][s][:-(-int(c["lengths"][s]) // 16)]
            zero = pages[::2] if first == 0 else pages[:len(pages) // 2] if first == 1 else pages[len(pages) // 2:]
            c["v_scale"][0, pages] = 2.0 ** log
            c["v_scale"][0, zero] = 2.0 ** -100
            live = c["v"][0, zero]
            c["v"][0, zero] = np.where((live & 127) == 127, live, 0)    # (bytes behind the end stay)
        check(c, on_gpu(c), query(r, 2, q_len, heads, head_dim, dtype), [0, 1])


@pytest.mark.parametrize("dtype,head_dim,q_len,heads", SHAPES)
def test_weights_far_below_the_largest_on_pages_of_the_largest_values(dtype, head_dim, q_len, heads):
    """Half the tokens' weights are 2^-13 of the peak's, and all of the result."""
    n, log = 600, 112
    c = filled(np.random.default_rng(3), [n], 1, 1, 16, head_dim)
    pages = c["table"][0][:-(-n // 16)]
    c["k"][0, pages] = 0
    c["v"][0, pages] = kv8.encode(1.0)
    c["v_scale"][0], c["k_scale"][0] = 2.0 ** log, 1.0
    c["k"][0, pages[0], 0, 3, 0], c["v"][0, pages[0], 0, 3] = kv8.encode(9.0), 0
    q = torch.zeros(1, q_len, heads, head_dim, device="cuda", dtype={"f32": torch.float32, "bf16": torch.bfloat16}[dtype])
    q[..., 0] = 1.0
    cache = on_gpu(c)
    check(c, cache, q, [0], scale=1.0)
    # the bound above is against the largest value; this one against the result: the tail's weights have 11 bits at least
    p, tail = np.exp(-9.0), n - q_len + np.arange(q_len)                # tokens of the tail that each query sees
    want = tail * p / (1 + tail * p) * 2.0 ** log
    got = cache.attention(0, q, scale=1.0).double().cpu().numpy()[0]
    err = np.abs(got / want[:, None, None] - 1).max()
    assert err <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22) + \
        2 * (9 * (head_dim / 16 + 6) * 2.0 ** -23 + 2.0 ** -22) + 2 * (n / 16 + 4) * 2.0 ** -23
