"""CPU oracle for writing tokens into the paged caches and reading sequences
back: TEST INFRASTRUCTURE.

Slot by slot, with the 8-bit formats taken from their definition
(``oracle.fp8``): a code is found as the nearest of the format's finite values,
by comparing distances, not by bit arithmetic.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import fp8
from .attention import gather_kv, sequence_block_ids

__all__ = ["encode", "kv_write", "kv_read"]


def encode(y: torch.Tensor, fmt: str) -> torch.Tensor:
    """uint8 codes of the float32 numbers ``y``: nearest finite value (of two
    equally near ones the even code), the largest one for anything beyond it,
    the sign kept (-0 too), a NaN code for NaN."""
    table = [(fp8.code_value(c, fmt), c) for c in range(128)]
    table = [(v, c) for v, c in table if math.isfinite(v)]
    values = torch.tensor([v for v, _ in table], dtype=torch.float64)  # ascending, from 0
    a = y.to(torch.float64).abs().clamp(max=float(values[-1])).flatten()
    hi = torch.searchsorted(values, a.nan_to_num(0.0)).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = values[hi] - a, a - values[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = torch.where(up == 0, hi, pick)
    nan = next(c for c in range(128) if math.isnan(fp8.code_value(c, fmt)))
    code = torch.tensor([c for _, c in table])[pick]
    code = torch.where(torch.isnan(a), torch.tensor(nan), code)
    sign = torch.signbit(y).flatten() & ~torch.isnan(a)
    return (code + 128 * sign).to(torch.uint8).reshape(y.shape)


def kv_write(key_cache: torch.Tensor, value_cache: torch.Tensor, key: torch.Tensor,
             value: torch.Tensor, slot_mapping: torch.Tensor, kv_cache_dtype: str = "auto",
             k_scale: float = 1.0, v_scale: float = 1.0):
    """The caches after the write, as new tensors.  ``slot = block * block_size
    + offset``; negative slots and slots past the caches are skipped."""
    fmt = fp8.format_of(kv_cache_dtype)
    key_cache, value_cache = key_cache.clone(), value_cache.clone()
    nb, hk, _, bs, x = key_cache.shape
    D = value_cache.shape[2]
    for i, slot in enumerate(slot_mapping.tolist()):
        if slot < 0 or slot >= nb * bs:
            continue
        k, v = key[i], value[i]
        if fmt is not None:
            k = encode(k.float() / torch.tensor(k_scale, dtype=torch.float32), fmt)
            v = encode(v.float() / torch.tensor(v_scale, dtype=torch.float32), fmt)
        key_cache[slot // bs, :, :, slot % bs, :] = k.reshape(hk, D // x, x)
        value_cache[slot // bs, :, :, slot % bs] = v
    return key_cache, value_cache


def kv_read(key_out: torch.Tensor, value_out: torch.Tensor, key_cache, value_cache, block_tables,
            cu_seq_lens, seq_starts=None, kv_indptr: Optional[torch.Tensor] = None,
            kv_cache_dtype: str = "auto", k_scale: float = 1.0, v_scale: float = 1.0):
    """``key_out`` / ``value_out`` after the read, as new tensors: the products
    ``code value * scale`` rounded to float32 and then to the output's dtype."""
    fmt = fp8.format_of(kv_cache_dtype)
    key_out, value_out = key_out.clone(), value_out.clone()
    bs = key_cache.shape[3]
    cu = [int(c) for c in cu_seq_lens]
    ks, vs = (float(torch.tensor(s, dtype=torch.float32)) for s in (k_scale, v_scale))
    for s in range(len(cu) - 1):
        n = cu[s + 1] - cu[s]
        first = 0 if seq_starts is None else int(seq_starts[s])
        if n == 0:
            continue
        ids = sequence_block_ids(block_tables, s, -(-(first + n) // bs), kv_indptr)
        for h in range(key_cache.shape[1]):
            K, V = gather_kv(key_cache, value_cache, ids, first + n, h,
                             **({} if fmt is None else dict(kv_format=fmt, k_scale=ks, v_scale=vs)))
            key_out[cu[s]:cu[s + 1], h] = K[first:].float().to(key_out.dtype)
            value_out[cu[s]:cu[s + 1], h] = V[first:].float().to(value_out.dtype)
    return key_out, value_out
