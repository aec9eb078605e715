"""Attention over the 8-bit cache where one token's score stands far above tens of thousands of others (a sink), and
other rows whose terms differ by many binades.

Bounds are against the sum of the terms' own magnitudes, sum_t p_t |v_t|, not against the largest value: a term may be
small, but its weight still has 11 bits (bf16 results: fp16) or 22 (fp32: two parts of fp16).  A weight is at least 2^6
at a row's largest score (it lies in [2^6, 2^15)) and fp16 is full down to 2^-14, so that holds down to 2^-20 of the
largest weight; below it an absolute 2^-25 takes over (fp32: 2^-37, the lower part is held 2^12 times as large), that is
2^-31 (2^-43) of the largest for each token."""
import itertools

import numpy as np
import pytest
import torch

from kv8_helpers import HALF, close, filled, flags, ints, on_gpu, score_bound, weight_bound
from oracle import kv8
from test_gpu_kv8_attention import check, query

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
FLOOR = {torch.bfloat16: 2.0 ** -31, torch.float32: 2.0 ** -43}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tensor_sharded_mlp_b200 import build
    build.build()


class History:
    """One sequence for each row of key (column 0; the others are zero) and value (the same in every column)."""

    def __init__(self, key, value, head_dim, page=64, v_scale=1.0):
        self.key, self.value = key, [x * v_scale for x in value]
        need = [-(-len(x) // page) for x in key]
        self.c = c = kv8.new_cache(1, sum(need), 1, page, head_dim, len(key), max(need))
        c["refcount"][:] = 1
        c["v_scale"][:] = v_scale
        at = 0
        for s, n in enumerate(need):
            c["table"][s, :n] = np.arange(at, at + n)
            c["lengths"][s] = len(key[s])
            for t in range(0, len(key[s]), page):
                k, v = key[s][t:t + page], value[s][t:t + page]
                c["k"][0, at, 0, :len(k), 0] = kv8.encode(k)
                c["v"][0, at, 0, :len(v)] = kv8.encode(v)[:, None]
                at += 1

    def check(self, q0, q_len, heads, dtype, scale, what, times=1):
        """All queries are q0 in column 0 and stand at the sequences' ends: every head of a query has the same result.
        `times`: the sequences are listed so often, so that a warp or a CTA has a whole one for itself."""
        dt, d, n = TORCH[dtype], self.c["k"].shape[4], len(self.key)
        q = torch.zeros(n * times, q_len, heads, d, device="cuda", dtype=dt)
        q[..., 0] = q0
        m, l, w, terms = (np.zeros((n, q_len)) for _ in range(4))
        for s in range(n):
            for j in range(q_len):
                see = len(self.key[s]) - q_len + j + 1
                sc, v = self.key[s][:see] * q0 * scale, self.value[s][:see]
                p = np.exp(sc - sc.max())
                m[s, j], l[s, j], w[s, j], terms[s, j] = sc.max(), p.sum(), p @ v, p @ np.abs(v)
        tokens, reach = max(map(len, self.key)), max(np.abs(x).max() for x in self.key) * abs(q0 * scale)
        bound = weight_bound(reach, d, tokens, dt) * terms + FLOOR[dt] * tokens * max(np.abs(x).max() for x in self.value)
        sb = score_bound(reach, d)
        cache = on_gpu(self.c)
        seqs = ints(list(range(n)) * times)
        out = cache.attention(0, q, seqs, scale=scale)
        gm, gl, gw = cache.attention_partials(0, q, seqs, scale=scale)

        def near(got, want, by, name):
            shape = (n * times, q_len) + (1,) * (got.dim() - 2)
            want, by = (np.broadcast_to(x, (times, n, q_len)).reshape(shape) for x in (want, by))
            close(got, np.broadcast_to(want, got.shape), by, f"{what} {name}")
        near(out, w / l, (bound + HALF[dt] * (terms + bound)) / l, "out")
        near(gm, m, sb + 2.0 ** -22 * np.abs(m), "maximum")
        near(gl, l, l * (4 * sb + 2 * (tokens / 16 + 8) * 2.0 ** -23 + 2.0 ** -20), "exp_sum")
        near(gw, w, 2 * sb * terms + bound + HALF[dt] * (terms + bound), "weighted")
        assert flags(cache) == 0


SHAPES = [("bf16", 64, 1, 8), ("bf16", 128, 1, 8), ("bf16", 256, 1, 3), ("bf16", 128, 3, 8), ("f32", 64, 1, 8), ("f32", 128, 1, 8),
          ("f32", 256, 1, 2), ("f32", 64, 1, 20), ("f32", 128, 2, 8),
          ("bf16", 64, 9, 8), ("bf16", 128, 9, 8), ("bf16", 256, 9, 8)]     # (the last three: the kernel for many rows)


@pytest.mark.parametrize("nats", [4, 9, 13, 14, 16, 17])
@pytest.mark.parametrize("dtype,head_dim,q_len,heads", SHAPES)
def test_one_token_far_above_a_long_flat_tail(dtype, head_dim, q_len, heads, nats):
    """The peak's value is zero, so the result is the tail's: tens of thousands of weights down to 4e-8 of the peak's."""
    key, value = [], []
    for n, t in ((40000, 0), (40000, 39980), (700, 300)):               # the peak first, nearly last, and in the middle
        k, v = np.zeros(n), np.ones(n)
        k[t], v[t] = 16.0, 0.0
        key.append(k)
        value.append(v)
    History(key, value, head_dim).check(nats / 16, q_len, heads, dtype, 1.0, f"{nats} nats")   # (exact in bf16)


@pytest.mark.parametrize("nats", [9, 14, 17])
@pytest.mark.parametrize("dtype,head_dim,q_len,heads", SHAPES)
def test_a_peak_in_the_same_share_as_its_whole_tail(dtype, head_dim, q_len, heads, nats):
    key, value = np.zeros(20000), np.ones(20000)
    key[7], value[7] = 16.0, 0.0
    h = History([key], [value], head_dim)
    h.check(nats / 16, q_len, heads, dtype, 1.0, f"{nats} nats", 400 if head_dim == 256 else 700)


@pytest.mark.parametrize("dtype,head_dim,q_len,heads", SHAPES)
def test_scores_within_the_slack_of_the_reference(dtype, head_dim, q_len, heads):
    """Scores just below what moves the reference, with the largest codes and scales between powers of two: weights reach
    their largest, nothing overflows."""
    t = np.arange(900)
    key = np.where(t < 64, 0.0, np.where(t % 3, 15.0, 14.0))
    value = np.where(t < 64, 1.0, np.where(t % 2, 448.0, -416.0))
    h = History([key], [value], head_dim, page=32, v_scale=float(np.float32(1.99)))
    for top in (4.5, 5.5, 6.5, 7.5, 7.9, 8.5, 14.5, 15.5):              # base-2 logs above the first tokens
        h.check(1.0, q_len, heads, dtype, float(np.float32(top / 15.0 * np.log(2.0))), f"2^{top}")


@pytest.mark.parametrize("dtype,head_dim,q_len,heads,size", [(*x, 2.0 ** (13 if x[0] == "f32" else 20)) for x in SHAPES] +
                         [("f32", 128, 1, 8, 2.0 ** 16), ("bf16", 128, 1, 8, 2.0 ** 22), ("bf16", 128, 9, 8, 2.0 ** 22)])
def test_a_query_element_far_above_the_others(dtype, head_dim, q_len, heads, size):
    """It meets keys of zero, so the scores are the other elements' alone, within the bound of their own products."""
    r = np.random.default_rng(head_dim + heads)
    c = filled(r, [300, 45], 1, 1, 32, head_dim)
    for s in range(2):
        for t in range(int(c["lengths"][s])):
            c["k"][0, c["table"][s, t // 32], 0, t % 32, 3] = 0
    q = query(r, 2, q_len, heads, head_dim, dtype)
    q[..., 3] = size
    check(c, on_gpu(c), q, [0, 1])


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,head_dim,q_len,heads", SHAPES)
def test_values_of_one_under_scores_of_millions(dtype, head_dim, q_len, heads, sign):
    """fp32 scores of that size lie up to 8 apart, but whatever the weights, their mean of ones is one: no weight may leave
    fp16's range, and each must count the same in both sums (11 or 22 bits, and a sum's own 2^-23 a step)."""
    r = np.random.default_rng(head_dim)
    n = 700
    c = kv8.new_cache(1, 11, 1, 64, head_dim, 1, 11)
    c["refcount"][:], c["table"][0], c["lengths"][0] = 1, np.arange(11), n
    c["v"][:] = kv8.encode(1.0)
    c["k"][0, :, 0, :, 0] = kv8.encode(15.0)
    c["k"][0, :, 0, :, 1] = kv8.encode(np.sort(r.choice(kv8._POS[kv8._POS <= 30], 704)).reshape(11, 64))     # rising
    cache = on_gpu(c)
    times = 300 if head_dim == 256 else 600                             # (a warp or a CTA has the sequence for itself)
    seqs = ints([0] * times)
    q = torch.zeros(times, q_len, heads, head_dim, device="cuda", dtype=TORCH[dtype])
    for log, binade in itertools.product((10, 16, 19, 20, 21, 22), (-9, -6, -4, -1, 0, 1, 2, 3, 4, 5, 6, 8, 11, 12, 13, 14)):
        scale = float(np.float32(1.99)) * 2.0 ** binade                 # up to 15 * 2^22 nats, 2^26.5 base-2 logs
        cache.v_scale.fill_(scale)
        q[..., 0], q[..., 1] = sign * 2.0 ** log, 1.0
        out = cache.attention(0, q, seqs, scale=1.0).double() / scale
        err = float((out - 1).abs().nan_to_num(1e9).max())
        bound = (2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 2.0 ** -24 + 2.0 ** -22) + 2 * (n / 16 + 8) * 2.0 ** -23 + 2.0 ** -21
        assert err <= bound, (log, binade, err, bound)
