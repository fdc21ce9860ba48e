"""A query that is not a number answers NaN, whether its row is cut over the SMs or not, and no other query notices."""
import numpy as np
import pytest

import _latent as la
import _trees as tr

pytestmark = pytest.mark.gpu

DECODE, CHUNK, TREE = 0, 1, 3
NAN = float("nan")


@pytest.mark.parametrize("heads", [16, 128])
def test_absorbed(heads):
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [(DECODE, 5000, 4999), (DECODE, 40, 39), (CHUNK, 900, 896), (TREE, 705, 700)]
    cache, pt, slots = la.paged([r[1] for r in rows], 201)
    q = la.queries(11, heads, 576, 202)
    bad = [(0, 3), (1, 0), (3, 5), (9, heads - 1)]
    for t, h in bad:
        q[t, h] = NAN
    mask = tr.random_tree(5, np.random.default_rng(203))
    plan = mq.LatentPlan(cache, heads, [r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows], pt.shape[1], 0.07)
    out = torch.zeros(11, heads, 512, dtype=torch.float16, device="cuda")
    plan.run(q, pt, out, mq.alloc_workspace(plan.workspace_bytes), tree_mask=torch.from_numpy(tr.pack([mask])).cuda())
    assert mq.device_error(clear=True) == 0
    at = 0
    for t, h in bad:
        assert bool(out[t, h].isnan().all()), (t, h)
        q[t, h] = 0
        out[t, h] = 0
    for r, (kind, s, o) in enumerate(rows):
        k = cache.data.view(-1, 576)[slots[r]][:, None]
        want, bound = la.attention64(q[at:at + s - o], k, k[..., :512], la.seen(kind, s, o, mask if kind == TREE else None), 0.07)
        for t, h in bad:
            if at <= t < at + s - o:
                want[t - at, h] = 0
        la.check(out[at:at + s - o], want, bound, (r, kind, s, o))
        at += s - o
    plan.close()


def test_expanded():
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows, heads = [(6000, 5700), (200, 0)], 2
    nk, nq = 6200, 500
    q, kv, kr = la.queries(nq, heads, 192, 211, 1.0), la.queries(nk, heads, 256, 212, 1.0), la.queries(nk, 1, 64, 213, 1.0)[:, 0]
    bad = [(0, 0), (170, 1), (299, 0), (303, 1), (450, 0)]
    for t, h in bad:
        q[t, h] = NAN
    plan = mq.ExpandedPlan(heads, [r[0] for r in rows], [r[1] for r in rows], 0.07)
    out = torch.zeros(nq, heads, 128, dtype=torch.float16, device="cuda")
    plan.run(q, kv[..., :128], kr, kv[..., 128:], out, mq.alloc_workspace(plan.workspace_bytes))
    assert mq.device_error(clear=True) == 0
    for t, h in bad:
        assert bool(out[t, h].isnan().all()), (t, h)
        q[t, h] = 0
        out[t, h] = 0
    at = first = 0
    for r, (s, o) in enumerate(rows):
        key = torch.cat([kv[first:first + s, :, :128], kr[first:first + s, None].expand(-1, heads, -1)], -1)
        want, bound = la.attention64(q[at:at + s - o], key, kv[first:first + s, :, 128:], la.seen(CHUNK, s, o), 0.07)
        for t, h in bad:
            if at <= t < at + s - o:
                want[t - at, h] = 0
        la.check(out[at:at + s - o], want, bound, (r, s, o))
        at += s - o
        first += s
    plan.close()


@pytest.mark.parametrize("fmt", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("kind", [CHUNK, TREE])
@pytest.mark.parametrize("n,ctx", [(5, 300), (5, 20000), (40, 300), (40, 20000)])
def test_paged_formats(fmt, kind, n, ctx):
    """Short and long rows on decode and on chunk tiles, in one piece and in several."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    pages = -(-(ctx + n) // 32)
    cache = mq.KVCache.allocate(pages, 1, 128, fmt, fmt)
    g = torch.Generator("cuda").manual_seed(221)
    k, v = (torch.randn(ctx + n, 1, 128, device="cuda", generator=g).half() for _ in range(2))
    mq.kv_append_quant(cache, k, v, torch.arange(ctx + n, dtype=torch.int32, device="cuda"))
    pt = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q = torch.randn(n, 4, 128, device="cuda", generator=g).half()
    plan = mq.Plan(cache, 4, [kind], [ctx + n], [ctx], pages)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    mask = torch.from_numpy(tr.pack([tr.random_tree(n, np.random.default_rng(222))])).cuda() if kind == TREE else None

    def run(x):
        out = torch.zeros_like(x)
        plan.run(x, pt, out, ws, tree_mask=mask)
        assert mq.device_error(clear=True) == 0
        return out

    want, bad = run(q), q.clone()
    bad[1, 2] = bad[n - 1, 0] = NAN
    got = run(bad)
    for t, h in ((1, 2), (n - 1, 0)):
        assert bool(got[t, h].isnan().all()), (t, h)
        got[t, h] = want[t, h]
    # (a NaN row may move its neighbours to the softmax's exact step, which sums in another order: fp32)
    assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -10
    plan.close()
