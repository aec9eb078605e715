"""The paged 8-bit cache without a GPU: the oracle's pins, and the calls' refusals."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import kv8


@pytest.fixture(scope="module")
def b():
    from tensor_sharded_mlp_b200 import build
    build.build()
    from tensor_sharded_mlp_b200 import binding
    return binding


# --- the oracle ------------------------------------------------------------------------------------------------------

def test_codes_are_torchs_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kv8.VALUES, want)
    r = np.random.default_rng(0)
    x = np.concatenate([r.standard_normal(20000) * 2.0 ** r.integers(-12, 8, 20000), kv8.VALUES[np.isfinite(kv8.VALUES)],
                        (kv8._POS[1:] + kv8._POS[:-1]) / 2, -(kv8._POS[1:] + kv8._POS[:-1]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(kv8.encode(x), want)
    np.testing.assert_array_equal(kv8.encode([np.inf, -np.inf, 1e30]), [0x7E, 0xFE, 0x7E])
    assert kv8.encode([np.nan])[0] & 127 == 127


@pytest.mark.parametrize("amax,want", [(448.0, 1.0), (448.0001, 2.0), (447.0, 1.0), (224.0, 0.5), (0.0, 2.0 ** -100),
                                       (1e-38, 2.0 ** -100), (1.0, 2.0 ** -8), (3.4e38, 2.0 ** 120)])
def test_scale_is_the_smallest_power_of_two_that_fits(amax, want):
    assert kv8.step_of([amax, -amax / 3, np.inf, np.nan]) == want


def test_attention_is_the_pages_attention():
    """Merged over two ranks' caches it equals the oracle's attention over the whole history."""
    r = np.random.default_rng(1)
    d, n = 64, 50
    k, v, q = (r.standard_normal(s).astype(np.float32) for s in ((n, 1, d), (n, 1, d), (1, 1, 1, d)))
    parts, ks, vs = [], [], []
    for lo, hi in ((0, 23), (23, 50)):
        c = kv8.new_cache(1, 8, 1, 16, d, 1, 4)
        assert kv8.reserve(c, [0], [hi - lo]) == 0
        assert kv8.append(c, 0, k[lo:hi], v[lo:hi], [0], [0, hi - lo]) == 0
        parts.append(kv8.attention_partials(c, 0, q, [0], d ** -0.5, [n - 1 - lo])[:3])
        a, b_ = kv8.dense(c, 0, 0, hi - lo)
        ks.append(a[0])
        vs.append(b_[0])
    m, l, w = (np.stack([p[x].reshape(-1) if x < 2 else p[x].reshape(1, d) for p in parts]).astype(np.float32)
               for x in range(3))
    got = oracle.merge_attention_partials(m, l, w)
    want = oracle.attention_full(q.reshape(1, d), np.concatenate(ks).astype(np.float32),
                                 np.concatenate(vs).astype(np.float32), d ** -0.5)
    np.testing.assert_allclose(got, want, rtol=0, atol=2e-6)


def test_growing_scale_keeps_values():
    """Codes of a page whose scale grows keep their values but for e4m3's subnormals."""
    r = np.random.default_rng(2)
    c = kv8.new_cache(1, 2, 1, 16, 64, 1, 1)
    x = r.standard_normal((5, 1, 64))
    kv8.reserve(c, [0], [5])
    kv8.append(c, 0, x, x, [0], [0, 5])
    before = kv8.dense(c, 0, 0, 5)[0]
    kv8.reserve(c, [0], [1])
    kv8.append(c, 0, np.full((1, 1, 64), 100.0), x[:1], [0], [0, 1])
    after = kv8.dense(c, 0, 0, 5)[0]
    step = c["k_scale"][0, c["table"][0, 0], 0]
    normal = np.abs(before) >= 2.0 ** -6 * step
    np.testing.assert_array_equal(before[normal], after[normal])
    assert np.abs(before - after).max() <= 2.0 ** -10 * step     # half of a subnormal's step


def test_page_map_of_the_oracle():
    """fork, reserve, truncate and compact on a pool small enough to follow by hand."""
    c = kv8.new_cache(1, 8, 1, 16, 64, 4, 3)
    assert kv8.reserve(c, [1, 0], [20, 16]) == 0
    assert c["table"][1].tolist() == [0, 1, -1] and c["table"][0].tolist() == [2, -1, -1]
    assert kv8.fork(c, [1, 1], [2, 3]) == 0
    assert c["refcount"].tolist() == [3, 3, 1, 0, 0, 0, 0, 0]
    assert kv8.reserve(c, [3, 2, 1], [1, 1, 1]) == 0             # all three holders: sequence 3 keeps page 1
    assert c["table"][3].tolist() == [0, 1, -1] and c["table"][2].tolist() == [0, 3, -1] and c["table"][1].tolist() == [0, 4, -1]
    assert kv8.reserve(c, [0], [60]) == kv8.BAD_LENGTH
    assert kv8.reserve(c, [0, 1, 2, 3], [32, 16, 16, 16]) == kv8.NO_PAGES and c["lengths"].tolist() == [16, 21, 21, 21]
    assert kv8.truncate(c, [3, 0]) == 0
    assert c["refcount"].tolist() == [2, 0, 0, 1, 1, 0, 0, 0]
    assert kv8.compact(c).tolist() == [0, -1, -1, 1, 2, -1, -1, -1]
    assert c["table"][2].tolist() == [0, 1, -1] and c["table"][1].tolist() == [0, 2, -1]


# --- refusals of the C calls (nothing is launched, no device is present) ----------------------------------------------

def _cache(b, **over):
    p = ctypes.c_void_p(0x100000)
    c = b.Kv8Cache(p, p, p, p, p, p, p, p, 2, 8, 2, 16, 64, 4, 3)
    for name, value in over.items():
        setattr(c, name, value)
    return c


SIZES = [dict(layers=0), dict(num_pages=0), dict(num_pages=(1 << 30) + 1), dict(kv_heads=0), dict(kv_heads=257),
         dict(page_size=24), dict(page_size=8), dict(page_size=512), dict(head_dim=96), dict(head_dim=32),
         dict(head_dim=512), dict(max_seqs=0), dict(max_pages=0), dict(max_pages=1 << 27, page_size=16)]


@pytest.mark.parametrize("over", SIZES)
def test_cache_sizes_are_refused(b, over):
    L, p, c = b._lib, ctypes.c_void_p(0x100000), _cache(b, **over)
    assert L.tp_mlp_kv8_pages_workspace_bytes(c) == 0
    assert L.tp_mlp_kv8_attention_workspace_bytes(c, 1, 1, 2) == 0
    assert L.tp_mlp_kv8_reserve(c, p, p, 1, p, 1 << 20, None) == 2
    assert L.tp_mlp_kv8_fork(c, p, p, 1, None) == 2
    assert L.tp_mlp_kv8_truncate(c, p, p, 1, None) == 2
    assert L.tp_mlp_kv8_copy_pages(c, p, 1, None) == 2
    assert L.tp_mlp_kv8_compact(c, p, p, 1 << 20, None) == 2
    assert L.tp_mlp_kv8_append(c, 0, p, p, 128, 1, p, None, 1, 1, None) == 2
    assert L.tp_mlp_kv8_attention(c, 0, p, 128, p, None, 1, 1, 2, 1.0, 1, p, p, 1 << 20, None) == 2
    assert L.tp_mlp_kv8_get_status(c, ctypes.byref(ctypes.c_int())) == 2


def test_call_arguments_are_refused(b):
    L, p, c = b._lib, ctypes.c_void_p(0x100000), _cache(b)
    assert L.tp_mlp_kv8_get_status(None, ctypes.byref(ctypes.c_int())) == 1
    assert L.tp_mlp_kv8_get_status(c, None) == 1
    for n in (-1, 1025):
        assert L.tp_mlp_kv8_reserve(c, p, p, n, p, 1 << 20, None) == 2
        assert L.tp_mlp_kv8_fork(c, p, p, n, None) == 2
        assert L.tp_mlp_kv8_truncate(c, p, p, n, None) == 2
        assert L.tp_mlp_kv8_copy_pages(c, p, n, None) == 2
        assert L.tp_mlp_kv8_append(c, 0, p, p, 128, 0, p, None, n, 1, None) == 2
        assert L.tp_mlp_kv8_attention(c, 0, p, 128, p, None, n, 1, 2, 1.0, 1, p, p, 1 << 20, None) == 2
        assert L.tp_mlp_kv8_attention_workspace_bytes(c, n, 1, 2) == 0
    # empty lists are no-ops, whatever the pointers
    assert L.tp_mlp_kv8_reserve(c, None, None, 0, None, 0, None) == 0
    assert L.tp_mlp_kv8_fork(c, None, None, 0, None) == 0
    assert L.tp_mlp_kv8_truncate(c, None, None, 0, None) == 0
    assert L.tp_mlp_kv8_copy_pages(c, None, 0, None) == 0
    assert L.tp_mlp_kv8_append(c, 0, None, None, 128, 0, None, None, 0, 1, None) == 0
    assert L.tp_mlp_kv8_append(c, 0, None, None, 128, 0, None, None, 3, 1, None) == 0
    assert L.tp_mlp_kv8_attention(c, 0, None, 128, None, None, 0, 1, 2, 1.0, 1, None, None, 0, None) == 0
    # sizes and enums of the data calls
    A = L.tp_mlp_kv8_append
    assert A(c, -1, p, p, 128, 1, p, None, 1, 1, None) == 2 and A(c, 2, p, p, 128, 1, p, None, 1, 1, None) == 2
    assert A(c, 0, p, p, 120, 1, p, None, 1, 1, None) == 2          # rows shorter than kv_heads * head_dim
    assert A(c, 0, p, p, 130, 1, p, None, 1, 1, None) == 3          # rows off the 16-byte boundary
    assert A(c, 0, p, p, 128, 3, p, None, 2, 1, None) == 2          # rows do not divide
    assert A(c, 0, p, p, 128, (1 << 22) + 2, p, None, 2, 1, None) == 2
    assert A(c, 0, p, p, 128, 1, p, None, 1, 2, None) == 1          # dtype
    assert A(c, 0, p, p, 128, 5, None, None, 5, 1, None) == 2       # more entries than sequences
    Q = L.tp_mlp_kv8_attention
    ws = 1 << 30
    assert Q(c, 2, p, 128, p, None, 1, 1, 2, 1.0, 1, p, p, ws, None) == 2      # layer
    assert Q(c, 0, p, 128, p, None, 1, 0, 2, 1.0, 1, p, p, ws, None) == 2      # q_len
    assert Q(c, 0, p, 128, p, None, 1, 129, 2, 1.0, 1, p, p, ws, None) == 2
    assert Q(c, 0, p, 192, p, None, 1, 1, 3, 1.0, 1, p, p, ws, None) == 2      # heads % kv_heads
    assert Q(c, 0, p, 1 << 20, p, None, 1, 1, 258, 1.0, 1, p, p, ws, None) == 2   # group of 129
    assert Q(c, 0, p, 64, p, None, 1, 1, 2, 1.0, 1, p, p, ws, None) == 2       # row stride
    assert Q(c, 0, p, 129, p, None, 1, 1, 2, 1.0, 1, p, p, ws, None) == 3
    assert Q(c, 0, p, 128, p, None, 1, 1, 2, float("nan"), 1, p, p, ws, None) == 1
    assert Q(c, 0, p, 128, p, None, 1, 1, 2, float("inf"), 1, p, p, ws, None) == 1
    assert Q(c, 0, p, 128, p, None, 1, 1, 2, 1.0, 9, p, p, ws, None) == 1
    assert Q(c, 0, None, 128, p, None, 1, 1, 2, 1.0, 1, p, p, ws, None) == 1
    assert Q(c, 0, p, 128, None, None, 5, 1, 2, 1.0, 1, p, p, ws, None) == 2   # more entries than sequences
    P = L.tp_mlp_kv8_attention_partials
    assert P(c, 0, p, 128, p, None, 1, 1, 2, 1.0, 1, None, p, p, p, ws, None) == 1
    assert P(c, 0, p, 128, p, None, 1, 1, 2, 1.0, 1, p, None, p, p, ws, None) == 1
    # buffers: null and misaligned ones are found before any driver query
    assert L.tp_mlp_kv8_truncate(_cache(b, table=None), p, None, 1, None) == 1
    assert L.tp_mlp_kv8_truncate(_cache(b, table=0x100004), p, None, 1, None) == 3
    assert L.tp_mlp_kv8_get_status(_cache(b, status=0x100004), ctypes.byref(ctypes.c_int())) == 3


def test_attention_workspace_is_bounded(b):
    """It holds the split pieces of every SM, not the history: the same for a cache of any length."""
    for d in (64, 128, 256):
        small = b._lib.tp_mlp_kv8_attention_workspace_bytes(_cache(b, head_dim=d), 4, 1, 2)
        large = b._lib.tp_mlp_kv8_attention_workspace_bytes(_cache(b, head_dim=d, num_pages=1 << 20, max_pages=1 << 16), 4, 1, 2)
        assert 0 < small == large < 64 << 20


def test_wrappers_refuse_host_tensors(b):
    c = _cache(b)
    t = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: b.tp_mlp_kv8_fork(c, t, t), lambda: b.tp_mlp_kv8_truncate(c, t),
                 lambda: b.tp_mlp_kv8_copy_pages(c, t.view(1, 2)), lambda: b.tp_mlp_kv8_reserve(c, None, t),
                 lambda: b.tp_mlp_kv8_append(c, 0, torch.zeros(2, 2, 64), torch.zeros(2, 2, 64)),
                 lambda: b.tp_mlp_kv8_attention(c, 0, torch.zeros(1, 1, 2, 64), 1.0)):
        with pytest.raises(ValueError):
            call()


# --- the order of a CTA's units in the prompt append --------------------------------------------------------------------

RUN_PROGRAM = r"""
#include <cstdio>
#include "kv8_run.h"
int main() {   // heads head0 run bits: the slots with something to write -> "slot head turn" of each unit that runs
    int heads, head0, run;
    unsigned long long bits;
    while (std::scanf("%d %d %d %llu", &heads, &head0, &run, &bits) == 4) {
        tpmlp::for_units(run, head0, heads, [&](int s) { return (bits >> s & 1) != 0; },
                         [&](int s, int h, int t) { std::printf("%d %d %d ", s, h, t); });
        std::printf("\n");
    }
}
"""


def test_units_that_follow_each_other_use_two_buffers(tmp_path):
    """Every unit with something to write runs once, in order, and no two in a row take the same exchange buffer: empty
    slots (which odd kv_heads make an odd number of skipped units) must not bring two of the same turn together."""
    import itertools
    import os
    import shutil
    import subprocess
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no host compiler")
    src = tmp_path / "run.cpp"
    src.write_text(RUN_PROGRAM)
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tensor_sharded_mlp_b200", "csrc")
    subprocess.run([cc, "-std=c++17", "-I", csrc, str(src), "-o", str(tmp_path / "run")], check=True)
    cases = []
    for heads, bits in itertools.product((1, 2, 3, 5, 8), range(64)):
        for head0 in {0, heads // 2, heads - 1}:
            for run in (1, heads, 6 * heads - head0):
                cases.append((heads, head0, run, bits))
    out = subprocess.run([str(tmp_path / "run")], input="\n".join(" ".join(map(str, x)) for x in cases), text=True,
                         capture_output=True, check=True).stdout.split("\n")
    for (heads, head0, run, bits), line in zip(cases, out):
        got = np.array(line.split(), int).reshape(-1, 3)
        units = [divmod(head0 + u, heads) for u in range(run)]
        assert [tuple(x) for x in got[:, :2]] == [x for x in units if bits >> x[0] & 1], (heads, head0, run, bits)
        assert (got[1:, 2] != got[:-1, 2]).all(), (heads, head0, run, bits)
        assert set(got[:, 2]) <= {0, 1}


@pytest.mark.parametrize("cu,written", [([0, 4, 9, 12], [0, 1, 2]), ([-5, 3, 10, 12], [1, 2]), ([0, 8, 5, 12], [0]),
                                        ([2, 4, 9, 10], [0, 1, 2]), ([0, 4, 13, 12], [0]), ([0, 12, 5, 9], [0])])
def test_row_bounds_of_the_oracle(cu, written):
    c = kv8.new_cache(1, 8, 1, 16, 64, 3, 2)
    kv8.reserve(c, [0, 1, 2], [12, 12, 12])
    c["k_scale"][:] = 7.0
    x = np.ones((12, 1, 64))
    want = kv8.BAD_LENGTH if len(written) < 3 else 0
    assert kv8.append(c, 0, x, x, [0, 1, 2], cu) == want
    assert [s for s in range(3) if c["k"][0, c["table"][s, 0], 0].any()] == written


def test_stalled_attention_is_refused(b):
    L, p, ws = b._lib.tp_mlp_kv8_selftest_stalled_attention, ctypes.c_void_p(0x100000), 1 << 30
    c = _cache(b)
    assert L(None, 0, p, 1, 100, 2, p, p, ws, 0, 0, 10, None) == 1
    assert L(_cache(b, page_size=24), 0, p, 1, 100, 2, p, p, ws, 0, 0, 10, None) == 2
    assert L(c, 0, p, 1, 129, 2, p, p, ws, 0, 0, 10, None) == 2
    for role, tile, wait in ((-1, 0, 10), (3, 0, 10), (0, -1, 10), (0, 0, 0), (0, 0, 100001)):
        assert L(c, 0, p, 1, 100, 2, p, p, ws, role, tile, wait, None) == 1
    assert L(c, 0, p, 1, 16, 2, p, p, ws, 0, 0, 10, None) == 4            # few rows
    assert L(c, 2, p, 1, 100, 2, p, p, ws, 0, 0, 10, None) == 2           # layer
    assert L(c, 0, None, 1, 100, 2, p, p, ws, 0, 0, 10, None) == 1


def test_calls_of_two_threads_get_their_own_workspace(b, monkeypatch):
    """Another thread's call between two looks at the size kept on the cache must not change this call's scratch."""
    class Shared(b.Kv8Cache):
        looks = 0

        @property
        def attention_workspace(self):
            Shared.looks += 1
            return (128, 2, 1 << 20) if Shared.looks == 1 else (1, 2, 16)   # from the second look on the other thread's

        @attention_workspace.setter
        def attention_workspace(self, value):
            pass

    monkeypatch.setattr(b, "_scratch", lambda nbytes, stream: nbytes)
    c = Shared.from_buffer_copy(_cache(b))
    assert b._kv8_workspace(c, 128, 2, None) == 1 << 20
    Shared.looks = 1                                                      # not kept: asked for, and not looked up again
    assert b._kv8_workspace(c, 128, 2, None) == b._lib.tp_mlp_kv8_attention_workspace_bytes(c, 1, 128, 2)


def test_a_torch_without_the_private_functions(b, monkeypatch):
    """The current device and stream come from torch's public calls then, for every wrapper."""
    class Stream:
        cuda_stream = 0x1234

    for name in ("_get_device", "_get_stream"):
        monkeypatch.setattr(b, name, None)
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    assert b._current_device() == 3
    assert b._stream(None).value == 0x1234 and b._stream(Stream()).value == 0x1234 and b._stream(0x99).value == 0x99


@pytest.mark.parametrize("parents,children,made,flags", [([-1, 0], [2, 2], [2], 0), ([3, 0], [-1, 3], [3], 0),
                                                         ([-1, 0, 0], [2, 2, 2], [2], kv8.BAD_SEQUENCE),
                                                         ([0, 2], [2, 3], [], kv8.BAD_SEQUENCE)])
def test_unused_pairs_of_the_oracles_fork(parents, children, made, flags):
    c = kv8.new_cache(1, 4, 1, 16, 64, 4, 2)
    kv8.reserve(c, [0], [20])
    assert kv8.fork(c, parents, children) == flags
    assert [s for s in (2, 3) if c["lengths"][s]] == made
