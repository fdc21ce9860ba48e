"""The bound of the page-scaled attention tests is met by correct arithmetic and exceeded by
lost keys (no GPU): a page, a warp's share, a split or a piece left out of any row."""
import numpy as np
import pytest

import _page8 as ref
import _page8_rows as bound


def _row(fmt, seq, hkv, d, seed):
    rng = np.random.default_rng(seed)
    n = -(-seq // 32)
    perm = rng.permutation(n + 1)
    slots = perm[np.arange(seq) // 32] * 32 + np.arange(seq) % 32
    planes = []
    for outliers in (True, False):
        x = rng.standard_normal((seq, hkv, d))
        if outliers:
            x[:, :, rng.integers(0, d, 3)] *= 8
        c = ref.PageCache(fmt, n + 1, hkv, d)
        c.append(x.astype(np.float16), slots)
        planes.append(c)
    return planes, slots, rng


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
@pytest.mark.parametrize("seq,off", [(40000, 39999), (9000, 8997), (4200, 4190), (300, 299)])
def test_a_lost_page_exceeds_the_bound(fmt, seq, off):
    (k, v), slots, rng = _row(fmt, seq, 1, 128, seq)
    hq = 4
    q = rng.standard_normal((seq - off, hq, 128)).astype(np.float16)
    args = (fmt, q, (k.codes, v.codes), (k.scale, v.scale), [slots], [(seq, off)])
    want, tol = bound.attention(*args)
    pages = -(-seq // 32)
    for lost in [{0}, {pages // 2}, {pages - 2}, {pages - 1}, set(range(5, 5 + min(32, pages - 6)))]:
        if lost == {pages - 1} and seq % 32:
            lost = {pages - 3}  # the last page may hold a few keys only
        got, _ = bound.attention(*args, missing=[lost])
        assert bound.off_by(got, want, tol) > 2, (lost, bound.off_by(got, want, tol))
    # and so does a page whose V scale is off by a quarter or so
    other = v.scale.copy()
    a, b = slots[0] // 32, slots[32] // 32
    other[a] = 1.25 * v.scale[b]
    got, _ = bound.attention(fmt, q, (k.codes, v.codes), (k.scale, other), [slots], [(seq, off)])
    assert bound.off_by(got, want, tol) > 1


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
@pytest.mark.parametrize("top", [-4, 0, 7, 10])
def test_rounded_weights_stay_within_the_bound(fmt, top):
    """P' as fp16 against the row's largest at 2^top, in one pass, the output as fp16."""
    seq, d = 3000, 128
    (k, v), slots, rng = _row(fmt, seq, 1, d, 5 + top)
    q = (rng.standard_normal((30, 4, d)) * 2).astype(np.float16)
    rows = [(seq, seq - 30)]
    want, tol = bound.attention(fmt, q, (k.codes, v.codes), (k.scale, v.scale), [slots], rows, tops=(top, top))
    page, place = slots // 32, slots % 32
    got = np.empty(q.shape)
    for h in range(4):
        x = (q[:, h].astype(np.float64) @ k.codes[page, 0, place].T) * k.scale[page, 0] / np.sqrt(d)
        x = np.where(np.arange(seq)[None, :] <= np.arange(seq - 30, seq)[:, None], x, -np.inf)
        x = x * np.log2(np.e) + np.log2(v.scale[page, 0].astype(np.float64))
        pp = np.exp2((x - x.max(axis=1, keepdims=True) + top).astype(np.float32))
        l = (pp / v.scale[page, 0]).sum(axis=1, keepdims=True)
        got[:, h] = (pp.astype(np.float16).astype(np.float64) @ v.codes[page, 0, place] / l).astype(np.float16)
    assert bound.off_by(got, want, tol) <= 1
