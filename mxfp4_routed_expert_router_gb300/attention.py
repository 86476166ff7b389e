"""Attention of a decoder layer: a paged key-value cache with its writer and its reader, and attention within prompts.

torch is used only for device memory and streams; everything runs in
libmoe_gb300.so through ``binding``.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B
from .linear import stream_workspace


def rope_table(n_positions: int, rot_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines for ``KvCache.append``: float32 [n_positions, rot_dim], angle = position * theta^(-2 i / rot_dim)
    for plane i, taken in 64 bits (a far position's angle loses its fraction in 32)."""
    i = torch.arange(rot_dim // 2, device=device, dtype=torch.float64)
    angle = torch.arange(n_positions, device=device, dtype=torch.float64).unsqueeze(1) * theta ** (-2 * i / rot_dim)
    return torch.cat((angle.cos(), angle.sin()), 1).float()


class KvCache:
    """One layer's keys and values in pages: k, v [n_pages, n_kv_heads, page_size, head_dim], bfloat16, or
    float8_e4m3fn with k_scales, v_scales uint8 [n_pages, n_kv_heads, page_size, head_dim / 32] (MXFP8).

    The tensors are the caller's (``empty`` makes them) and stay with the cache.  The slot of a token is
    page * page_size + offset.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in (torch.bfloat16,
                                                                                     torch.float8_e4m3fn):
            raise B.MoeError(B.MOE_EINVAL, "k, v: bfloat16 or float8_e4m3fn [n_pages, n_kv_heads, page_size, head_dim] "
                                           f"tensors are needed, not {k.dtype} {tuple(k.shape)} and {v.dtype} "
                                           f"{tuple(v.shape)}")
        mx = k.dtype == torch.float8_e4m3fn
        if mx != (k_scales is not None) or mx != (v_scales is not None):
            raise B.MoeError(B.MOE_EINVAL, "k_scales, v_scales: MXFP8 needs both, bfloat16 none")
        n_pages, n_kv, page, dim = k.shape
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None and (t.dtype != torch.uint8 or t.shape != (n_pages, n_kv, page, dim // 32)):
                raise B.MoeError(B.MOE_EINVAL, f"{name}: uint8 {(n_pages, n_kv, page, dim // 32)} is needed, not "
                                               f"{t.dtype} {tuple(t.shape)}")
        tensors = [t for t in (k, v, k_scales, v_scales) if t is not None]
        if any(not t.is_contiguous() or not t.is_cuda or t.device != k.device for t in tensors):
            raise B.MoeError(B.MOE_EINVAL, "a cache's tensors must be dense and on one CUDA device")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.device = k.device
        self._workspace = {}  # n_heads -> bytes that ``decode`` needs
        self.page_size, self.n_kv_heads, self.head_dim = page, n_kv, dim
        self.c = B.MoeKvCache(k.data_ptr(), v.data_ptr(), B._ptr(k_scales), B._ptr(v_scales),
                              B.MOE_ROWS_MXFP8 if mx else B.MOE_ROWS_BF16, n_pages, page, n_kv, dim)
        self.c.device = k.get_device()

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int = 64, head_dim: int = 128, fmt: str = "bf16",
              device="cuda") -> "KvCache":
        """A cache of zeros; fmt: "bf16" or "mxfp8"."""
        if fmt not in ("bf16", "mxfp8"):
            raise B.MoeError(B.MOE_EINVAL, f"unknown cache format {fmt!r}")
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        ty = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
        parts = [torch.zeros(shape, dtype=ty, device=device) for _ in range(2)]
        if fmt == "mxfp8":
            parts += [torch.zeros(shape[:3] + (head_dim // 32,), dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(*parts)

    def append(self, qkv: torch.Tensor, n_heads: int, slots: torch.Tensor, positions: Optional[torch.Tensor] = None,
               rope: Optional[torch.Tensor] = None, pairs: bool = False, q_out: Optional[torch.Tensor] = None,
               k_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Turns queries and keys of qkv (bfloat16 [T, (n_heads + 2 n_kv_heads) * head_dim]) by their positions, writes
        keys and values to their slots (-1: nowhere) and returns the queries, [T, n_heads, head_dim].  rope: a table
        as ``rope_table`` makes (None: nothing is turned), planes of a head's halves or, with pairs, of neighbours.
        k_out: also receives the turned keys, [T, n_kv_heads, head_dim]."""
        if q_out is None:
            with _on(stream):
                q_out = torch.empty((qkv.shape[0], n_heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
        B.moe_kv_append(self.c, qkv, n_heads, slots, positions, rope, B.MOE_ROPE_PAIRS if pairs else B.MOE_ROPE_HALVES,
                        q_out, k_out, stream)
        return q_out

    def decode(self, q: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of one token for each of B sequences (q bfloat16 [B, n_heads, head_dim]) over their lens[b] tokens
        in the pages page_table[b] (int32 [B, max_pages]).  scale: 1 / sqrt(head_dim) by default."""
        if q.dim() != 3:
            raise B.MoeError(B.MOE_EINVAL, f"q: shape {tuple(q.shape)} where [B, n_heads, head_dim] is needed")
        n = self._workspace.get(q.shape[1])
        if n is None:  # (the same for every number of sequences)
            n = self._workspace[q.shape[1]] = B.moe_attention_decode_workspace_bytes(1, q.shape[1], self.n_kv_heads,
                                                                                     self.head_dim)
        if stream is None:
            ws = stream_workspace(n, self.device) if n else None
            out = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
        else:
            with _on(stream):
                ws = stream_workspace(n, self.device) if n else None
                out = torch.empty_like(q, memory_format=torch.contiguous_format) if out is None else out
        B.moe_attention_decode(self.c, q, page_table, lens, self.head_dim ** -0.5 if scale is None else scale, out, ws,
                               n, stream)
        return out


def prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor, scale: Optional[float] = None,
           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention within packed prompts: q bfloat16 [T, n_heads, head_dim], k, v [T, n_kv_heads, head_dim] (views
    of wider rows will do), offsets int32 [n_seqs + 1].  Rows that no sequence holds are left as they are in out (of
    an out made here they hold anything)."""
    if out is None:
        with _on(stream):
            out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    B.moe_attention_prompt(q, k, v, offsets, q.shape[-1] ** -0.5 if scale is None else scale, out, stream)
    return out


class Attention:
    """A decoder layer's attention on the rows of its input projection (bfloat16 [T, (n_heads + 2 n_kv_heads) *
    head_dim]: queries, keys and values side by side), over a cache of its own.

    rope: a table as ``rope_table`` makes, or None (nothing is turned); scale: 1 / sqrt(head_dim) by default.  Both
    calls turn the queries and keys of the rows in place, write keys and values to their slots (int32 [T]; -1: padding)
    and return bfloat16 [T, n_heads * head_dim]; positions (int32 [T]) are needed with rope.  A call that is refused has
    touched neither the rows nor the cache.
    """

    def __init__(self, n_heads: int, cache: KvCache, rope: Optional[torch.Tensor] = None, pairs: bool = False,
                 scale: Optional[float] = None):
        if n_heads < 1 or n_heads % cache.n_kv_heads:
            raise B.MoeError(B.MOE_EINVAL, f"n_heads: {n_heads} is no multiple of the cache's {cache.n_kv_heads} heads")
        if rope is not None and (rope.dim() != 2 or rope.dtype != torch.float32 or not rope.is_contiguous() or
                                 rope.device != cache.device):
            raise B.MoeError(B.MOE_EINVAL, "rope: a dense float32 [n_positions, rot_dim] tensor beside the cache is "
                                           "needed")
        self.n_heads, self.cache, self.rope, self.pairs = n_heads, cache, rope, pairs
        self.scale = cache.head_dim ** -0.5 if scale is None else scale
        B.check_attention(cache.c, n_heads, self.scale)
        self.row = (n_heads + 2 * cache.n_kv_heads) * cache.head_dim  # values of a row of the projection

    def _heads_of(self, qkv: torch.Tensor):
        """Views of the rows' queries, keys and values."""
        n, kv, dim = self.n_heads, self.cache.n_kv_heads, self.cache.head_dim
        if qkv.dim() != 2 or qkv.shape[1] != self.row or qkv.stride(1) != 1:
            raise B.MoeError(B.MOE_EINVAL, f"qkv: shape {tuple(qkv.shape)} where [T, {self.row}] is needed")
        rows = qkv.unflatten(1, (n + 2 * kv, dim))
        return rows[:, :n], rows[:, n:n + kv], rows[:, n + kv:]

    def decode(self, qkv: torch.Tensor, slots: torch.Tensor, positions: Optional[torch.Tensor],
               page_table: torch.Tensor, lens: torch.Tensor) -> torch.Tensor:
        """One new token for each sequence; lens (int32 [T]) counts it.  A row without a sequence has slot -1 and
        length 0, and gives zeros."""
        q, _, _ = self._heads_of(qkv)
        B.check_decode(self.cache.c, qkv, page_table, lens)
        self.cache.append(qkv, self.n_heads, slots, positions, self.rope, self.pairs, q)
        return self.cache.decode(q, page_table, lens, self.scale).flatten(1)

    def prompt(self, qkv: torch.Tensor, slots: torch.Tensor, positions: Optional[torch.Tensor],
               offsets: torch.Tensor) -> torch.Tensor:
        """Whole prompts, packed: sequence s has the rows offsets[s] .. offsets[s + 1] - 1 (int32 [n_seqs + 1]).  Rows
        of no sequence give zeros."""
        q, k, v = self._heads_of(qkv)
        B.check_prompt(self.cache.c, qkv, self.n_heads, offsets)
        self.cache.append(qkv, self.n_heads, slots, positions, self.rope, self.pairs, q, k)
        out = torch.zeros((q.shape[0], self.n_heads, self.cache.head_dim), dtype=torch.bfloat16, device=qkv.device)
        return prompt(q, k, v, offsets, self.scale, out).flatten(1)


def sync(stream=None) -> None:
    """Waits for the stream and raises if an attention kernel on the current device, on whatever stream, recorded an error
    since the last time on this stream."""
    B.moe_attention_status(stream)


class _on:
    """torch.cuda.stream for a stream, its address, or None (the current one)."""

    def __init__(self, stream):
        self.guard = None if stream is None else torch.cuda.stream(
            torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
