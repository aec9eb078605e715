"""Shared by the tests of the paged 8-bit cache: an oracle cache, its copy on the GPU, and error bounds.

The bounds count roundings, worst case, for reach = the largest sum_d |q_d k_d| * scale of a row:
  score      each of head_dim / 16 accumulations and a final one may lose 2^-23 of the sum's reach; q and the
             factors in front of it a few more 2^-23                        -> (head_dim / 16 + 6) 2^-23 reach
  weight     exp's argument is off by that and by 2^-23 of its size, exp itself by 2^-22; a weight that
             multiplies the values is rounded to fp16 (2^-11) for bf16 results, and to two fp16 parts (2^-22) for fp32
  sum        tokens / 16 accumulations of 2^-23 each, and as many again where parts are joined and rescaled
  result     half a step of the result's type
"""
import numpy as np
import torch

from oracle import kv8

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def score_bound(reach, head_dim):
    return (head_dim / 16 + 6) * 2.0 ** -23 * reach


def weight_bound(reach, head_dim, tokens, dtype):
    """Relative error of a weighted sum, against the sum of the terms' magnitudes."""
    rounding = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    return 2 * (score_bound(reach, head_dim) + 2.0 ** -22) + rounding + 2 * (tokens / 16 + 4) * 2.0 ** -23


def close(got, want, bound, what):
    """|got - want| <= bound everywhere; NaN and infinities in the same places."""
    got = np.asarray(got.detach().double().cpu() if isinstance(got, torch.Tensor) else got, np.float64)
    want = np.asarray(want, np.float64)
    bound = np.broadcast_to(bound, want.shape)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = np.isfinite(want)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=what)
    inf = np.isinf(want)
    np.testing.assert_array_equal(got[inf], want[inf], err_msg=what)
    off = np.abs(got[fin] - want[fin]) - bound[fin]
    assert not off.size or off.max() <= 0, f"{what}: {off.max():.3e} over a bound of {bound[fin][off.argmax()]:.3e}"


def filled(r, lengths, layers=1, kv_heads=2, page=16, head_dim=64, spare=4, max_pages=None, spread=1.0, stale=0x7F):
    """An oracle cache whose sequences hold random rows in scattered pages; all other slots hold `stale` bytes."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    c = kv8.new_cache(layers, pages, kv_heads, page, head_dim, len(lengths), max_pages or max(need + [1]) + 2)
    c["k"][:], c["v"][:] = stale, stale
    order = list(r.permutation(pages))
    for s, n in enumerate(lengths):
        for b in range(need[s]):
            p = order.pop()
            c["table"][s, b], c["refcount"][p] = p, 1
            m = min(page, n - b * page)
            for layer in range(layers):
                for h in range(kv_heads):
                    for name in ("k", "v"):
                        x = r.standard_normal((m, head_dim)) * spread * 2.0 ** r.integers(-2, 3)
                        step = kv8.step_of(x)
                        c[name + "_scale"][layer, p, h] = step
                        c[name][layer, p, h, :m] = kv8.encode(x / step)
        c["lengths"][s] = n
    return c


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda").contiguous()


def on_gpu(c):
    from tensor_sharded_mlp_b200 import kv_cache
    dev = {n: torch.from_numpy(np.array(c[n])).cuda() for n in ("k", "v")}
    for n in ("k_scale", "v_scale"):
        dev[n] = torch.from_numpy(c[n].astype(np.float32)).cuda()
    return kv_cache.KvCache8.over(dev["k"], dev["v"], dev["k_scale"], dev["v_scale"], ints(c["table"]), ints(c["lengths"]),
                                  ints(c["refcount"]), torch.zeros(1, dtype=torch.int32, device="cuda"))


def flags(cache):
    from tensor_sharded_mlp_b200 import binding
    return binding.tp_mlp_kv8_get_status(cache.c)


def same_map(cache, c, what=""):
    for n in ("lengths", "refcount", "table"):
        np.testing.assert_array_equal(getattr(cache, n).cpu().numpy(), c[n], err_msg=f"{what} {n}")


def same_pool(cache, c, what=""):
    """Codes and scales bit for bit (NaN codes of either sign count as one)."""
    for n in ("k", "v"):
        got, want = getattr(cache, n).cpu().numpy(), c[n]
        nan = ((got & 127) == 127) & ((want & 127) == 127)
        np.testing.assert_array_equal(np.where(nan, 127, got), np.where(nan, 127, want), err_msg=f"{what} {n}")
        np.testing.assert_array_equal(getattr(cache, n + "_scale").cpu().numpy(), c[n + "_scale"].astype(np.float32),
                                      err_msg=f"{what} {n}_scale")
