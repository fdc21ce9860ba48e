"""Tree rows on the host: what a plan accepts, and the packed masks' reading by the kernels."""
import ctypes

import numpy as np
import pytest

import _trees as tr
import mixed_attention_quantized_gb300 as mq


def _status(kinds, seqs, offs, window_plan=False, hq=8):
    d = mq.cache_desc(512, 2, 128, mq.Q8_0, mq.Q8_0)
    arr = [(ctypes.c_int32 * len(x))(*x) for x in (kinds, seqs, offs)]
    ws = ctypes.c_size_t(0)
    return mq.load().mixattn_workspace_bytes(ctypes.byref(d), hq, len(seqs), *arr, 512, ctypes.byref(ws)), ws.value


def test_tree_rows_are_checked_like_chunk_rows():
    assert _status([mq.ROW_TREE], [110], [70])[0] == mq.OK
    assert _status([mq.ROW_TREE], [70], [70])[0] == mq.ERR_INVALID_ARG
    assert _status([mq.ROW_TREE], [70], [-1])[0] == mq.ERR_INVALID_ARG
    assert _status([2], [70], [60])[0] == mq.ERR_INVALID_ARG
    assert _status([mq.ROW_TREE], [1024], [0])[0] == mq.OK
    assert _status([mq.ROW_TREE], [1025], [0])[0] == mq.ERR_UNSUPPORTED


def test_plans_without_trees_need_no_more_workspace():
    a, b = _status([1, 0], [110, 50], [104, 49]), _status([mq.ROW_TREE, 0], [110, 50], [104, 49])
    assert a[0] == b[0] == mq.OK and a[1] <= b[1] <= a[1] + 512


def _bits(words, n, rel):
    """The kernels' 32-key reading of a mask, restated."""
    out = 0
    for e in range(32):
        j = rel + e
        if j < 0 or (j < n and j // 32 < len(words) and (words[j // 32] >> (j % 32)) & 1):
            out |= 1 << e
    return out


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 70])
def test_packed_masks_hold_the_tree(n):
    rng = np.random.default_rng(n)
    m = tr.random_tree(n, rng, 2)
    for stray in (False, True):
        p = tr.pack([m], stray=stray).view(np.uint32)
        for i in (0, n // 2, n - 1):
            vis = np.array([(_bits([int(w) for w in p[i]], n, 32 * b) >> e) & 1 for b in range(3) for e in range(32)])
            assert np.array_equal(vis[:n].astype(bool), m[i]) and not vis[n:].any()
        assert _bits([int(w) for w in p[0]], n, -40) == 0xFFFFFFFF
        assert _bits([int(w) for w in p[0]], n, -31) & 0x7FFFFFFF == 0x7FFFFFFF
