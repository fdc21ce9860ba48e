"""Tree rows at other head groups, and what a tree in the batch leaves of the other rows: their bits."""
import numpy as np
import pytest

import _trees as tr
import test_gpu_tree as base

pytestmark = pytest.mark.gpu

DECODE, CHUNK, TREE = base.DECODE, base.CHUNK, base.TREE


@pytest.mark.parametrize("kf,vf", base.FORMATS)
@pytest.mark.parametrize("hq,hkv,d,window", [(8, 4, 128, 0), (4, 2, 64, 0), (8, 4, 64, 200)])
def test_two_heads_a_group(kf, vf, hq, hkv, d, window):
    rows, masks = base._rows_and_masks([(TREE, 6, 0), (TREE, 76, 64), (TREE, 45, 32), (TREE, 413, 400), (DECODE, 77, 76),
                                        (TREE, 1130, 1000), (CHUNK, 90, 80)], 111)
    base._check(kf, vf, hq, hkv, d, rows, masks, 112, window=window)


@pytest.mark.parametrize("kf,vf", base.FORMATS)
@pytest.mark.parametrize("hq,hkv,d,window", [(8, 8, 64, 0), (8, 4, 128, 0), (8, 2, 128, 300), (8, 1, 64, 40), (32, 8, 128, 0)])
def test_other_rows_keep_their_bits(kf, vf, hq, hkv, d, window):
    """Decode rows short and long, verify passes, chunks of one tile and of many: the bits of the batch without trees,
    whose places chunk rows of the same lengths take."""
    import torch
    spec = [(TREE, 45, 20), (DECODE, 1, 0), (DECODE, 33, 32), (DECODE, 3000, 2999), (TREE, 2003, 2000), (CHUNK, 403, 400),
            (CHUNK, 64, 0), (CHUNK, 700, 100), (CHUNK, 2600, 2590), (TREE, 330, 298)]
    cache, pt, _ = base._filled(kf, vf, [s for _, s, _ in spec], hkv, d, 121)
    total = sum(s - o for _, s, o in spec)
    q = torch.randn(total, hq, d, device="cuda", generator=torch.Generator("cuda").manual_seed(122)).half()
    masks = [tr.random_tree(s - o, np.random.default_rng(123)) for k, s, o in spec if k == TREE]
    got = base._run(cache, pt, spec, hq, q, masks, window)
    plain = base._run(cache, pt, [(CHUNK if k == TREE else k, s, o) for k, s, o in spec], hq, q, [], window)
    at = 0
    for k, s, o in spec:
        if k != TREE:
            assert torch.equal(got[at:at + s - o], plain[at:at + s - o]), (k, s, o)
        at += s - o
