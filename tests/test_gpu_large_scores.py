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
