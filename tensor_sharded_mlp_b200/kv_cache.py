"""A paged key/value cache in 8 bits: its buffers, and the calls that work on them.

``KvCache8`` owns the tensors that the C calls ``tp_mlp_kv8_*`` (``include/tp_mlp.h``)
take: e4m3 codes in pages, one scale for each page and KV head, and the page map
shared by all layers.  One decode step of a batch:

    cache.reserve(seqs, counts)                # places for the new tokens, shared last pages copied
    for layer in range(layers):
        cache.append(layer, k, v, seqs)        # quantise the new rows into them
        out = cache.attention(layer, q, seqs)  # q: (n, q_len, heads, head_dim)

Under decode context parallelism ("LLM 推理并行化：先找瓶颈，再决定怎么切", §三 4)) each
rank holds a part of the history; ``attention_partials`` gives the rank's
(maximum, exp_sum, weighted), which ``binding.tp_mlp_merge_attention_partials``
merges.

Lists of sequences, counts and lengths are int32 CUDA tensors, so a step can be
captured in a CUDA graph; what does not fit is left out on the device and
reported by ``check()``.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import binding


class KvCache8:
    """The cache of one GPU: `layers` layers of `num_pages` pages of `page_size`
    tokens, for up to `max_seqs` sequences of up to `max_tokens` tokens."""

    def __init__(self, layers: int, num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64,
                 max_seqs: int = 256, max_tokens: int = 8192, device=None):
        device = torch.device("cuda" if device is None else device)
        pool = (layers, num_pages, kv_heads, page_size, head_dim)

        def ints(*shape, value=0):
            return torch.full(shape, value, dtype=torch.int32, device=device)

        self._take(torch.zeros(pool, dtype=torch.uint8, device=device), torch.zeros(pool, dtype=torch.uint8, device=device),
                   torch.ones(pool[:3], device=device), torch.ones(pool[:3], device=device),
                   ints(max_seqs, -(-max_tokens // page_size), value=-1), ints(max_seqs), ints(num_pages), ints(1))

    @classmethod
    def over(cls, k, v, k_scale, v_scale, table, lengths, refcount, status) -> "KvCache8":
        """A cache over buffers that exist already (layouts as in include/tp_mlp.h)."""
        cache = cls.__new__(cls)
        cache._take(k, v, k_scale, v_scale, table, lengths, refcount, status)
        return cache

    def _take(self, k, v, k_scale, v_scale, table, lengths, refcount, status):
        if k.dim() != 5 or v.shape != k.shape or any(t.dtype not in (torch.uint8, torch.float8_e4m3fn) for t in (k, v)):
            raise ValueError("k and v must be uint8 or float8_e4m3fn (layers, num_pages, kv_heads, page_size, head_dim)")
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype != torch.float32 or t.shape != k.shape[:3]:
                raise ValueError(f"{what} must be float32 (layers, num_pages, kv_heads)")
        if table.dim() != 2 or lengths.shape != table.shape[:1] or refcount.shape != k.shape[1:2] or status.numel() != 1:
            raise ValueError("table must be (max_seqs, max_pages), lengths (max_seqs,), refcount (num_pages,), status one word")
        if any(t.dtype != torch.int32 for t in (table, lengths, refcount, status)):
            raise ValueError("table, lengths, refcount and status must be int32")
        tensors = (k, v, k_scale, v_scale, table, lengths, refcount, status)
        if any(not t.is_cuda or t.device != k.device or not t.is_contiguous() for t in tensors):
            raise ValueError("the cache's tensors must be contiguous and on one CUDA device")
        (self.k, self.v, self.k_scale, self.v_scale, self.table, self.lengths, self.refcount, self.status) = tensors
        self.layers, self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.device = k.device
        self.c = binding.Kv8Cache(*(ctypes.c_void_p(t.data_ptr()) for t in tensors), *k.shape, *table.shape)
        if binding._lib.tp_mlp_kv8_pages_workspace_bytes(self.c) == 0:
            raise ValueError("page_size must be 16, 32, 64, 128 or 256, head_dim 64, 128 or 256, kv_heads at most 256, "
                             "and every size at least 1")

    def _on(self):
        if binding._current_device() != self.device.index:
            raise ValueError(f"the cache is on {self.device}, which is not the current CUDA device")
        return self.c

    def reserve(self, seqs: Optional[torch.Tensor], counts: torch.Tensor, stream=None) -> None:
        binding.tp_mlp_kv8_reserve(self._on(), seqs, counts, stream)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, seqs: Optional[torch.Tensor] = None,
               cu_tokens: Optional[torch.Tensor] = None, n: Optional[int] = None, stream=None) -> None:
        binding.tp_mlp_kv8_append(self._on(), layer, k, v, seqs, cu_tokens, n, stream)

    def attention(self, layer: int, q: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                  positions: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """scale defaults to head_dim ** -0.5."""
        return binding.tp_mlp_kv8_attention(self._on(), layer, q, self.head_dim ** -0.5 if scale is None else scale,
                                            seqs, positions, out, stream)

    def attention_partials(self, layer: int, q: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                           positions: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                           maximum: Optional[torch.Tensor] = None, exp_sum: Optional[torch.Tensor] = None,
                           weighted: Optional[torch.Tensor] = None,
                           stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        return binding.tp_mlp_kv8_attention_partials(self._on(), layer, q,
                                                     self.head_dim ** -0.5 if scale is None else scale, seqs, positions,
                                                     maximum, exp_sum, weighted, stream)

    def fork(self, parents: torch.Tensor, children: torch.Tensor, stream=None) -> None:
        binding.tp_mlp_kv8_fork(self._on(), parents, children, stream)

    def truncate(self, seqs: torch.Tensor, new_lengths: Optional[torch.Tensor] = None, stream=None) -> None:
        binding.tp_mlp_kv8_truncate(self._on(), seqs, new_lengths, stream)

    def copy_pages(self, pairs: torch.Tensor, stream=None) -> None:
        binding.tp_mlp_kv8_copy_pages(self._on(), pairs, stream)

    def compact(self, new_index: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Returns the new number of every page (-1 for pages that were free)."""
        if new_index is None:
            new_index = binding._new(stream, self.num_pages, dtype=torch.int32, device=self.device)
        binding.tp_mlp_kv8_compact(self._on(), new_index, stream)
        return new_index

    def check(self) -> None:
        """Raise if a call so far met something that did not fit (see KV8_FLAGS); synchronises and clears."""
        flags = binding.tp_mlp_kv8_get_status(self._on())
        if flags:
            raise RuntimeError("the cache's calls met " +
                               ", ".join(name for bit, name in binding.KV8_FLAGS.items() if flags & bit))
