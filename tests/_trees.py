"""Drafted trees and 64-bit attention over what a cache holds, for the GPU tests."""
from __future__ import annotations

import numpy as np


def random_tree(n: int, rng, roots: int = 1) -> np.ndarray:
    """bool [n, n]: row i marks i and its ancestors; the first `roots` tokens have none."""
    m = np.zeros((n, n), dtype=bool)
    for i in range(n):
        if i >= roots:
            m[i] = m[rng.integers(0, i)]
        m[i, i] = True
    return m


def pack(masks, words: int = 0, stray: bool = False) -> np.ndarray:
    """int32 [sum n, words] of the rows' bool masks; `stray`: every bit past a row's n set."""
    words = words or max((m.shape[0] + 31) // 32 for m in masks)
    out = []
    for m in masks:
        b = np.full((m.shape[0], 32 * words), stray)
        b[:, :m.shape[0]] = m
        out.append((b.reshape(-1, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1))
    return np.concatenate(out).astype(np.uint32).view(np.int32)


def seen(kind: int, seq: int, off: int, mask=None, window: int = 0) -> np.ndarray:
    """bool [queries, seq]: the keys each query of a row sees (kinds: 0 decode, 1 chunk, 3 tree)."""
    key, nq = np.arange(seq), seq - off
    if kind != 3:
        pos = off + np.arange(nq)[:, None]
        return (key <= pos) & ((key > pos - window) if window else True)
    s = np.zeros((nq, seq), dtype=bool)
    s[:, off:] = mask
    pos = off + np.maximum(mask.sum(1), 1)[:, None] - 1
    s[:, :off] = (key[:off] > pos - window) if window else True
    return s


def cache_values(cache, which: int, slots):
    """fp64 [tokens, heads, head_dim] of the slots, from the cache's canonical blocks."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    fmt = (cache.k_fmt, cache.v_fmt)[which]
    b = mq.kv_export_blocks(cache, which, slots)
    if fmt == mq.F16:
        return b.view(torch.float16).double().flatten(2)
    if fmt in (mq.I8_PAGE, mq.E4M3_PAGE):
        kind = torch.int8 if fmt == mq.I8_PAGE else torch.float8_e4m3fn
        return (b[..., 4:].contiguous().view(kind).double() * b[..., :4].contiguous().view(torch.float32).double()).flatten(2)
    d = b[..., :2].contiguous().view(torch.float16).double()
    q = b[..., 2:].contiguous()
    if fmt == mq.Q8_0:
        return (q.view(torch.int8).double() * d).flatten(2)
    return ((torch.cat([q & 15, q >> 4], -1).double() - 8) * d).flatten(2)


def attention64(q, k, v, visible, scale: float):
    """fp64 [queries, heads, dv] of one row: q [queries, heads, d], k and v [keys, kv heads, .];
    a query that sees nothing gets zeros."""
    import torch
    group = q.shape[1] // k.shape[1]
    k, v = (x.repeat_interleave(group, dim=1) for x in (k, v))
    x = torch.einsum("qhd,khd->hqk", q.double(), k) * scale
    x = x.masked_fill(~torch.as_tensor(visible, device=q.device), -np.inf)
    p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
    v = torch.where(torch.as_tensor(visible, device=q.device).any(0)[:, None, None], v, torch.zeros_like(v))
    return torch.einsum("hqk,khd->qhd", p, v)
