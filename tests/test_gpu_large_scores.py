"""Latent attention where scaled scores are far beyond 2^24, so that no fp32 number in the exponent's units lies
within a bit of the largest of them.

Queries and keys are whole numbers whose products and their sums stay under 2^24, exact in fp32 in any order:
what 64 bits make of them is the answer, equal keys share their weight, and a key one unit below the largest
weighs exp(-softmax_scale).  The bound is `_latent.attention64`'s: the weights' fp16 rounding and the
output's; the exponent of a weight that counts is a difference of two whole numbers times the scale, off by
2^-23 of itself at most, which for differences of up to 2^5 is under the 2^-13 that the bound has for it."""
import numpy as np
import pytest

import _latent as la
import _trees as tr

pytestmark = pytest.mark.gpu

DECODE, CHUNK, TREE = 0, 1, 3
SCALES = [0.07, 1.0, 30.0, 5000.0, 9.9e5]


def _whole(shape, top, seed):
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, device="cuda", generator=g).half()


@pytest.mark.parametrize("heads", [4, 16, 32, 128])
@pytest.mark.parametrize("scale", SCALES)
def test_absorbed(heads, scale):
    """S up to 576 x 60^2 = 2^21: 2^41 in the exponent at the largest scale."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [(DECODE, 1, 0), (DECODE, 40, 39), (DECODE, 3000, 2999), (CHUNK, 390, 387), (TREE, 325, 300), (CHUNK, 70, 0)]
    cache, pt, slots = la.paged([r[1] for r in rows], 101)
    flat = cache.data.view(-1, 576)
    for r, at in enumerate(slots):
        flat[at] = _whole((len(at), 576), 60, 110 + r)
        flat[at[len(at) // 2:]] = flat[at[:len(at) - len(at) // 2]].clone()  # every key twice: weights of a half
    q = _whole((sum(s - o for _, s, o in rows), heads, 576), 60, 120)
    q[0, 0], q[3] = 0, -q[3]
    mask = tr.random_tree(25, np.random.default_rng(102))
    plan = mq.LatentPlan(cache, heads, [r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows], pt.shape[1], scale)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    ws.fill_(0xFF)
    out = torch.full((q.shape[0], heads, 512), float("nan"), dtype=torch.float16, device="cuda")
    plan.run(q, pt, out, ws, tree_mask=torch.from_numpy(tr.pack([mask])).cuda())
    assert mq.device_error(clear=True) == 0
    at = 0
    for r, (kind, s, o) in enumerate(rows):
        k = flat[slots[r]][:, None]
        want, bound = la.attention64(q[at:at + s - o], k, k[..., :512], la.seen(kind, s, o, mask if kind == TREE else None), scale)
        la.check(out[at:at + s - o], want, bound, (r, kind, s, o))
        at += s - o
    plan.close()


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("heads,rows", [(3, [(1, 0), (300, 0), (700, 650)]), (1, [(6000, 5700)]), (2, [(130, 0), (1000, 200)])])
def test_expanded(heads, rows, scale):
    """S up to 192 x 100^2 = 2^21."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    nk, nq = sum(s for s, _ in rows), sum(s - o for s, o in rows)
    q, k, kr = _whole((nq, heads, 192), 100, 131), _whole((nk, heads, 128), 100, 132), _whole((nk, 64), 100, 133)
    k[1::2], kr[1::2] = k[:nk - nk % 2:2].clone(), kr[:nk - nk % 2:2].clone()  # neighbours alike: weights of a half
    v = la.queries(nk, heads, 128, 134, 1.0)
    plan = mq.ExpandedPlan(heads, [r[0] for r in rows], [r[1] for r in rows], scale)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    ws.fill_(0xFF)
    out = torch.full((nq, heads, 128), float("nan"), dtype=torch.float16, device="cuda")
    plan.run(q, k, kr, v, out, ws)
    assert mq.device_error(clear=True) == 0
    at = first = 0
    for r, (s, o) in enumerate(rows):
        key = torch.cat([k[first:first + s], kr[first:first + s, None].expand(-1, heads, -1)], -1)
        want, bound = la.attention64(q[at:at + s - o], key, v[first:first + s], la.seen(CHUNK, s, o), scale)
        la.check(out[at:at + s - o], want, bound, (r, s, o))
        at += s - o
        first += s
    plan.close()


@pytest.mark.parametrize("rows", [[(3000, 2900)], [(2600, 2590), (3000, 0)]])
def test_expanded_scores_that_rise_slowly_past_2_to_the_22(rows):
    """Key j's score is 2906000 + j / 2, 2^22 / log2(e) at j = 2540: about 23 bits a block of 32 keys, before and
    after the reference takes a score."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    nk, nq, heads = sum(s for s, _ in rows), sum(s - o for s, o in rows), 2
    j = torch.cat([torch.arange(s) for s, _ in rows]).cuda()
    q, k = torch.zeros(nq, heads, 192, device="cuda").half(), torch.zeros(nk, heads, 128, device="cuda").half()
    q[..., 0], q[..., 130], k[..., 0] = 2000, 1, 1453
    kr = torch.zeros(nk, 64, device="cuda").half()
    kr[:, 2] = j // 2
    v = la.queries(nk, heads, 128, 141, 1.0)
    plan = mq.ExpandedPlan(heads, [r[0] for r in rows], [r[1] for r in rows], 1.0)
    out = torch.full((nq, heads, 128), float("nan"), dtype=torch.float16, device="cuda")
    plan.run(q, k, kr, v, out, mq.alloc_workspace(plan.workspace_bytes))
    assert mq.device_error(clear=True) == 0
    at = first = 0
    for s, o in rows:
        key = torch.cat([k[first:first + s], kr[first:first + s, None].expand(-1, heads, -1)], -1)
        for a in range(0, s - o, 256):
            b = min(s - o, a + 256)
            want, bound = la.attention64(q[at + a:at + b], key, v[first:first + s], la.seen(CHUNK, s, o)[a:b], 1.0)
            la.check(out[at + a:at + b], want, bound, (s, o, a))
        at += s - o
        first += s
    plan.close()


@pytest.mark.parametrize("fmt", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("kind,n", [(DECODE, 1), (CHUNK, 5), (CHUNK, 40), (TREE, 5), (TREE, 40)])
@pytest.mark.parametrize("ctx", [200, 9000])
def test_paged_formats_up_to_2_to_the_20(fmt, kind, n, ctx):
    """Every kind of row, short and cut, with scores of up to 2^20 (and beside 64 bits over what the cache holds): keys
    and queries of +-1 times one size each, so that scores are whole multiples of one step, far enough apart for a
    key, or several alike, to weigh all; the weights' and the output's rounding is what is left."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    g = torch.Generator("cuda").manual_seed(151)
    keys, pages = ctx + n, -(-(ctx + n) // 32)
    sign = lambda *s: (torch.randint(0, 2, s, device="cuda", generator=g) * 2 - 1).float()
    # 128 equal signs: a score of 128 a b / sqrt(128) = 2^20 x 0.72
    a, b = 256.0, 254.0
    cache = mq.KVCache.allocate(pages, 1, 128, fmt, fmt)
    k, v = (sign(keys, 1, 128) * b).half(), la.queries(keys, 1, 128, 152, 1.0)
    mq.kv_append_quant(cache, k, v, torch.arange(keys, dtype=torch.int32, device="cuda"))
    slots = torch.arange(keys, dtype=torch.int32, device="cuda")
    k, v = tr.cache_values(cache, 0, slots), tr.cache_values(cache, 1, slots)
    assert float((k.abs() - b).abs().max()) <= 0.13 * b  # (a code's step)
    q = torch.empty(n, 4, 128, device="cuda", dtype=torch.float16)
    q[:] = k[ctx // 2 + torch.arange(4, device="cuda"), 0].sign().half() * a  # a key of the context each
    mask = tr.random_tree(n, np.random.default_rng(153))
    pt = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    plan, out = mq.Plan(cache, 4, [kind], [keys], [ctx], pages), torch.zeros_like(q)
    plan.run(q, pt, out, mq.alloc_workspace(plan.workspace_bytes),
             tree_mask=torch.from_numpy(tr.pack([mask])).cuda() if kind == TREE else None)
    assert mq.device_error(clear=True) == 0
    want = tr.attention64(q, k, v, tr.seen(kind, keys, ctx, mask if kind == TREE else None), 128 ** -0.5)
    assert float((out.double() - want).abs().max()) <= 2e-3 + 2.0 ** -11 * float(want.abs().max())
    plan.close()
