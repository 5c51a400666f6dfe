"""The 4-bit key/value cache of a served model: append, attend, read back.

Layout, grid and masks: include/kronq.h (kronq_kv4_*).  A batch is three int32
device tensors, the same in every call of a step:

  block_table (batch x pages)  the pages of each sequence, in order
  q_start     (batch + 1)      rows of each sequence's new tokens
  kv_len      (batch)          cached tokens of each, the new ones included

A layer's step is

  q = kv4.append(q, k, v, cache, block_table, q_start, kv_len, rope=table, signs=signs)
  o = kv4.attend(q, cache, block_table, q_start, kv_len)

on the current stream; both can be captured into a graph and replayed with other
lengths and pages in the same tensors.  Outputs and workspaces that are not
given are allocated on the current stream.
"""

from __future__ import annotations

import torch

from . import abi


def make_cache(pages: int, page_size: int, heads: int, head_dim: int, device=None) -> torch.Tensor:
    """An empty cache (its contents need no set-up: only appended tokens are read)."""
    nbytes = abi.kronq_kv4_block_bytes(page_size, head_dim)
    if nbytes == 0:
        raise ValueError(f"page_size {page_size} / head_dim {head_dim} is not supported "
                         "(16, 32, 64, 128, 256 / 64, 128, 256)")
    return torch.empty((pages, heads, nbytes), dtype=torch.uint8, device=device or "cuda")


def rope_table(rows: int, rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """Row p: the rot/2 cosines and then the sines of p base^(-2i/rot) (angles in fp64)."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device or "cuda") / rot)
    ang = torch.arange(rows, dtype=torch.float64, device=f.device)[:, None] * f
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def append(q, k, v, cache, block_table, q_start, kv_len, rope=None, interleaved: bool = False,
           positions=None, signs=None, q_out=None, info=None, stream=None):
    """Puts the batch's new keys and values into the cache; returns the rotated
    queries (None when q is None)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return append(q, k, v, cache, block_table, q_start, kv_len, rope, interleaved, positions, signs,
                          q_out, info)
    return abi.kronq_kv4_append(q, k, v, cache, block_table, q_start, kv_len, q_out, rope, interleaved, positions,
                                signs, info)


def gather(cache, block_table, q_start, kv_len, tokens: int, head_dim: int, dtype=torch.bfloat16,
           info=None, stream=None):
    """(keys, values) of the batch's new tokens as the cache holds them, tokens x
    heads x head_dim; rows that are no sequence's are left unset."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gather(cache, block_table, q_start, kv_len, tokens, head_dim, dtype, info)
    return abi._kv4_calls().gather_new(cache, block_table, q_start, kv_len, tokens, head_dim, dtype, info)


def attend(q, cache, block_table, q_start, kv_len, scale: float | None = None, causal: bool = True,
           window: int = 0, sinks: int = 0, out=None, lse=None, ws=None, info=None, stream=None):
    """Attention of q (tokens x q_heads x head_dim) over the cache; scale defaults
    to head_dim^-1/2.  Rows that are no sequence's are left as they were (unset in a
    fresh output)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return attend(q, cache, block_table, q_start, kv_len, scale, causal, window, sinks, out, lse, ws, info)
    return abi.kronq_kv4_attention(q, cache, block_table, q_start, kv_len, out, ws, scale, causal, window, sinks,
                                   lse, info)
