"""64-bit latent attention and its error bound, for the GPU tests."""
from __future__ import annotations

import numpy as np

import _trees as tr


def attention64(q, k, v, visible, scale):
    """(fp64 outputs [queries, heads, dv], bound of an fp16 output's error) of one row.

    q [queries, heads, d]; k [keys, heads or 1, d], v [keys, heads or 1, dv] as they are held.
    The bound: a weight is rounded to fp16 (2^-11 of it; weights below 2^-20 of the row's largest by
    2^-31 of that), the scores' products and sums, the exponential and the sums are fp32 (together
    under 2^-13 of a weight for scores of a few tens), and the output is rounded (2^-11, or 2^-25)."""
    import torch
    vis = torch.as_tensor(visible, device=q.device)
    heads = q.shape[1]
    k, v = (x.double().expand(-1, heads, -1) for x in (k, v))
    x = torch.einsum("qhd,khd->hqk", q.double(), k) * scale
    p = torch.nan_to_num(torch.softmax(x.masked_fill(~vis, -np.inf), -1), nan=0.0)
    used = vis.any(0)[:, None, None]
    v = torch.where(used, v, torch.zeros_like(v))
    o = torch.einsum("hqk,khd->qhd", p, v)
    size = torch.einsum("hqk,khd->qhd", p, v.abs())
    tail = vis.sum(1).double()[:, None, None] * 2.0 ** -31 * float(v.abs().max())
    return o, (2.0 ** -11 + 2.0 ** -13) * size + tail + 2.0 ** -11 * o.abs() + 2.0 ** -25


def check(got, want, bound, what=""):
    err = (got.double() - want).abs()
    worst = (err - bound).max()
    assert bool((err <= bound).all()), (what, float(err.max()), float(worst))


def paged(seqs, seed, extra=3, fill=float("nan")):
    """A latent cache of N(0, 1) rows whose unwritten rows hold `fill`, its page table and each row's slots."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(seed)
    need = [-(-s // 32) for s in seqs]
    cache = mq.LatentCache.allocate(sum(need) + extra)
    cache.data.fill_(fill)
    perm = rng.permutation(cache.num_pages).astype(np.int32)
    pt = np.full((len(seqs), max(need)), -1, dtype=np.int32)
    slots, at = [], 0
    g = torch.Generator("cuda").manual_seed(seed)
    flat = cache.data.view(-1, 576)
    for r, n in enumerate(need):
        pt[r, :n] = perm[at:at + n]
        at += n
        t = np.arange(seqs[r])
        slots.append(torch.from_numpy((pt[r, t // 32] * 32 + t % 32).astype(np.int64)).cuda())
        flat[slots[r]] = torch.randn(seqs[r], 576, device="cuda", generator=g).half()
    return cache, torch.from_numpy(pt).cuda(), slots


def queries(n, heads, dim, seed, size=0.5):
    import torch
    return (torch.randn(n, heads, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)) * size).half()


def seen(kind, s, o, mask=None):
    return tr.seen(kind, s, o, mask)
