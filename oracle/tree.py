"""CPU oracle for the attention of drafted token trees over a paged cache,
float64: TEST INFRASTRUCTURE.

A sequence's drafted tokens are the last ones of its cached tokens.  Row i
sees every token before them and the drafted tokens its mask row names; the
tokens a row does not see are left out before any arithmetic, so nothing
stored there can reach the result.
"""
from __future__ import annotations

from typing import Optional

import torch

from .attention import _kv_options, gather_kv, kv_head_of, sequence_block_ids

__all__ = ["tree_attention"]


def tree_attention(query, key_cache, value_cache, block_tables, seq_lens, cu_query_lens,
                   scale: float, tree_mask: Optional[torch.Tensor] = None,
                   positions: Optional[torch.Tensor] = None, logits_soft_cap: float = 0.0,
                   kv_indptr: Optional[torch.Tensor] = None, kv_cache_dtype: str = "auto",
                   k_scale: float = 1.0, v_scale: float = 1.0, alibi_slopes=None) -> torch.Tensor:
    """``[num_tokens, num_heads, head_size]`` float64; rows past the last
    sequence are NaN.  ``tree_mask`` ``None``: a chain (drafted token j <= i)."""
    N, H, D = query.shape
    Hk, bs = key_cache.shape[1], key_cache.shape[3]
    key_cache, value_cache, kvq = _kv_options(key_cache, value_cache, kv_cache_dtype, k_scale,
                                              v_scale)
    out = torch.full((N, H, D), float("nan"), dtype=torch.float64)
    cu = [int(c) for c in cu_query_lens]
    for s in range(len(cu) - 1):
        T, L = cu[s + 1] - cu[s], int(seq_lens[s])
        ctx = L - T
        ids = sequence_block_ids(block_tables, s, (L + bs - 1) // bs, kv_indptr)
        place = torch.arange(L)
        if positions is not None:
            place[ctx:] = positions[cu[s]:cu[s + 1]].long()
        kv = [gather_kv(key_cache, value_cache, ids, L, h, **kvq) for h in range(Hk)]
        for i in range(T):
            row = cu[s] + i
            seen = torch.ones(L, dtype=torch.bool)
            if tree_mask is None:
                seen[ctx + i + 1:] = False
            else:
                m = torch.zeros(T, dtype=torch.bool)
                cols = min(T, tree_mask.shape[1])
                m[:cols] = tree_mask[row, :cols] != 0
                seen[ctx:] = m
            for h in range(H):
                K, V = kv[kv_head_of(h, H, Hk)]
                K, V = K[seen], V[seen]
                z = (K @ query[row, h].double()) * scale
                if logits_soft_cap > 0:
                    z = logits_soft_cap * torch.tanh(z / logits_soft_cap)
                if alibi_slopes is not None:
                    z = z + float(alibi_slopes[h]) * (place[seen] - place[ctx + i]).double()
                out[row, h] = torch.softmax(z, 0) @ V if len(z) else torch.zeros(D).double()
    return out
