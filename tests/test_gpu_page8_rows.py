"""Attention over the page-scaled formats against the tight bound of ``_page8_rows.py``, under
which no lost page, split or piece of any row passes."""
import numpy as np
import pytest

import _page8 as ref
import _page8_rows as bound
import test_gpu_page8 as base

pytestmark = pytest.mark.gpu

FORMATS = [ref.I8, ref.E4M3]


def _planes(cache, row_slots):
    """((K, V) codes, (K, V) scales), zeros in the pages that no row uses."""
    kq, ks, vq, vs = base._planes(cache)
    used = np.isin(np.arange(cache.num_pages), np.unique(np.concatenate(row_slots) // 32))
    return tuple(np.where(used[:, None, None, None], x, 0) for x in (kq, vq)), tuple(
        np.where(used[:, None], x, 0) for x in (ks, vs))


def _kinds(rows):
    return [0 if s - o == 1 else 1 for s, o in rows]


def _queries(rows, hq, d, seed):
    return np.random.default_rng(seed).standard_normal((sum(s - o for s, o in rows), hq, d)).astype(np.float16)


def _check(fmt, cache, pt, row_slots, rows, q, window=0, **kw):
    import mixed_attention_quantized_gb300 as mq
    got = base._attend(cache, pt, rows, _kinds(rows), q.shape[1], q, window)
    assert mq.device_error(clear=True) == 0
    codes, scales = _planes(cache, row_slots)
    want, tol = bound.attention(fmt, q, codes, scales, row_slots, rows, window, **kw)
    assert bound.off_by(got, want, tol) <= 1, bound.off_by(got, want, tol)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_long_rows(fmt, d):
    """Decode splits, verify groups and cut chunk tiles: each row at its own bound."""
    rows = [(40000, 39999), (9000, 8997), (20011, 19900), (4200, 4190), (2500, 2499), (1, 0), (33, 32)]
    cache, pt, row_slots = base._filled(fmt, rows, 1, d, 177)
    _check(fmt, cache, pt, row_slots, rows, _queries(rows, 4, d, 178))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [33, 1100])
def test_windows(fmt, window):
    rows = [(6000, 5999), (3000, 2996), (5000, 4800), (700, 0)]
    cache, pt, row_slots = base._filled(fmt, rows, 2, 128, window)
    _check(fmt, cache, pt, row_slots, rows, _queries(rows, 8, 128, window + 1), window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gain", [2.0 ** -10, 2.0 ** -13])
@pytest.mark.parametrize("d", [64, 128])
def test_small_values_beside_pages_of_zeros(fmt, gain, d):
    """A page whose V is all zero counts in the softmax's sum and takes no bits from the others."""
    def gains(rng, n):
        g = np.full(-(-n // 32), gain)
        g[rng.random(len(g)) < 0.3] = 0
        g[0] = 0
        return g.repeat(32)[:n]
    rows = [(500, 499), (1500, 1499), (6000, 5999), (200, 100), (700, 694), (4000, 3960), (600, 0)]
    cache, pt, row_slots = base._filled(fmt, rows, 2, d, 203, gains)
    assert any((s == 0).any() for s in _planes(cache, row_slots)[1])
    _check(fmt, cache, pt, row_slots, rows, _queries(rows, 4, d, 204))


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_of_zeros_only(fmt):
    """No value but zeros: zeros out, in every kind of row and a batch with other rows."""
    rows = [(300, 299), (9000, 8999), (70, 66), (400, 200), (500, 499)]
    def gains(rng, n):
        return np.zeros(n) if n != 500 else np.ones(n)
    cache, pt, row_slots = base._filled(fmt, rows, 1, 128, 207, gains)
    q = _queries(rows, 4, 128, 208)
    got = base._attend(cache, pt, rows, _kinds(rows), 4, q)
    assert (got[:-1] == 0).all() and np.abs(got[-1]).max() > 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sink", [0, 1])
def test_long_tail_under_one_dominant_key(fmt, d, sink):
    """One key (the row's first, or one in the middle) 8 to 22 bits above all others, its own value
    zero: the output is the tail's, whose weights are far below the largest.  Values of one sign."""
    import mixed_attention_quantized_gb300 as mq
    rows = [(9000, 8999), (9000, 8994), (9000, 8960), (9000, 8800), (3000, 2999)]
    rng = np.random.default_rng(301)
    need = [-(-s // 32) for s, _ in rows]
    pt = np.full((len(rows), max(need)), -1, dtype=np.int32)
    perm, at, row_slots = rng.permutation(sum(need)).astype(np.int32), 0, []
    cache = base._alloc(fmt, sum(need), 1, d)
    for r, (seq, _) in enumerate(rows):
        pt[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
        t = np.arange(seq)
        slots = pt[r, t // 32] * 32 + t % 32
        k = 0.1 * rng.standard_normal((seq, 1, d))
        k[:, :, 0] = 0
        v = rng.uniform(0.5, 1.5, (seq, 1, d))
        dominant = seq // 2 * sink
        k[dominant], v[dominant] = 0, 0
        k[dominant, 0, 0] = 16
        base._append(cache, k.astype(np.float16), v.astype(np.float16), slots)
        row_slots.append(slots)
    q = _queries(rows, 4, d, 302)
    bits = rng.uniform(8, 22, q.shape[:2])
    bits[0] = [8, 14, 18, 22]
    q[:, :, 0] = bits * np.log(2) * np.sqrt(d) / 16
    got = base._attend(cache, pt, rows, _kinds(rows), 4, q)
    assert mq.device_error(clear=True) == 0
    codes, scales = _planes(cache, row_slots)
    want, tol = bound.attention(fmt, q, codes, scales, row_slots, rows, coherent=True)
    assert (tol < 0.02 * want + 2.0 ** -24).all()  # the bound means something for every element
    assert bound.off_by(got, want, tol) <= 1, bound.off_by(got, want, tol)


# (row, page numbers without a page): first, last and whole KV tiles of four pages, both pages of a
# conversion warp's pair and either one, in every kind of tile
LOST = [((1000, 999), {0, 31}), ((3000, 2995), {1, 50, 92}), ((700, 500), {0, 5, 7, 12, 13, 14, 15}), ((700, 460), {21}),
        ((2325, 2309), {8, 9, 10, 11, 40, 72}), ((4100, 4000), {1, 66, 127}), ((130, 0), {2})]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 900])
def test_rows_without_some_pages(fmt, d, window):
    """A page id outside the cache is flagged, and the row is attention over its other keys."""
    import mixed_attention_quantized_gb300 as mq
    mq.device_error(clear=True)
    rows, lost = [r for r, _ in LOST], [p for _, p in LOST]
    cache, pt, row_slots = base._filled(fmt, rows, 2, d, 501)
    bad = [cache.num_pages, -1, -5, 2 ** 31 - 1, -2 ** 31]
    for r, pages in enumerate(lost):
        for i, p in enumerate(sorted(pages)):
            pt[r, p] = bad[(r + i) % len(bad)]
    q = _queries(rows, 8, d, 502)
    got = base._attend(cache, pt, rows, _kinds(rows), 8, q, window)
    assert mq.device_error(clear=True) == mq.DEVERR_PAGE_ID
    codes, scales = _planes(cache, row_slots)
    want, tol = bound.attention(fmt, q, codes, scales, row_slots, rows, window, missing=lost)
    assert bound.off_by(got, want, tol) <= 1, bound.off_by(got, want, tol)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", ["ramp", "steps", "pairs"])
def test_scores_that_keep_moving_the_reference(fmt, d, shape):
    """Scores that rise or fall along the keys, by page or from key to key, up to 200 bits in all: the
    references move at every page or once, by a little or past all that came before."""
    import mixed_attention_quantized_gb300 as mq
    rows = [(3000, 2999), (2600, 2595), (2500, 2470), (1000, 700), (9000, 8980)]
    rng = np.random.default_rng(601)
    need = [-(-s // 32) for s, _ in rows]
    pt = np.full((len(rows), max(need)), -1, dtype=np.int32)
    perm, at, row_slots = rng.permutation(sum(need)).astype(np.int32), 0, []
    cache = base._alloc(fmt, sum(need), 1, d)
    for r, (seq, _) in enumerate(rows):
        pt[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
        t = np.arange(seq)
        slots = pt[r, t // 32] * 32 + t % 32
        k, v = rng.standard_normal((2, seq, 1, d))
        height = {"ramp": t / seq, "steps": rng.random(need[r])[t // 32], "pairs": ((t // 2) % 48) / 48}[shape]
        k[:, 0, 0] = 16 * height
        v *= np.exp2(rng.integers(-6, 7, need[r]))[t // 32, None, None]
        base._append(cache, k.astype(np.float16), v.astype(np.float16), slots)
        row_slots.append(slots)
    q = _queries(rows, 8, d, 602)
    bits = np.array([3, 12, 40, 200, -3, -12, -40, -200])
    q[:, :, 0] = bits * np.log(2) * np.sqrt(d) / 16
    got = base._attend(cache, pt, rows, _kinds(rows), 8, q)
    assert mq.device_error(clear=True) == 0
    codes, scales = _planes(cache, row_slots)
    want, tol = bound.attention(fmt, q, codes, scales, row_slots, rows)
    assert bound.off_by(got, want, tol) <= 1, bound.off_by(got, want, tol)


@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_before_the_window_are_not_read(fmt):
    """Decode and verify rows: whole pages, chunk rows: whole KV tiles of four pages before the first
    query's window may be given away (ids outside the cache here)."""
    import mixed_attention_quantized_gb300 as mq
    mq.device_error(clear=True)
    rows, window = [(6000, 5999), (3000, 2996), (5000, 4800)], 700
    cache, pt, row_slots = base._filled(fmt, rows, 2, 128, 701)
    q = _queries(rows, 8, 128, 702)
    good = base._attend(cache, pt, rows, _kinds(rows), 8, q, window)
    bad = pt.copy()
    for r, (_, off) in enumerate(rows):
        first = off + 1 - window
        bad[r, :first // 32 if r < 2 else first // 128 * 4] = cache.num_pages + 7
    np.testing.assert_array_equal(base._attend(cache, bad, rows, _kinds(rows), 8, q, window), good)
    assert mq.device_error(clear=True) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (8, 8), (8, 1)])
def test_a_query_that_sees_one_key_gets_its_value(fmt, d, hq, hkv):
    """Window 1, and the first token of a prompt: the one weight is 1 whatever it is rounded to, so the
    output is the key's value to fp16's own rounding (and 2^-21 for the fp32 steps)."""
    import mixed_attention_quantized_gb300 as mq
    rows = [(300, 299), (500, 494), (700, 500), (1100, 0), (200, 0)]
    cache, pt, row_slots = base._filled(fmt, rows, hkv, d, 801)
    q = _queries(rows, hq, d, 802)
    (_, cv), (_, dv) = _planes(cache, row_slots)
    got = base._attend(cache, pt, rows, _kinds(rows), hq, q, 1)
    at = 0
    for r, (seq, off) in enumerate(rows):
        s = np.asarray(row_slots[r])[off:seq]
        want = np.repeat(cv[s // 32, :, s % 32] * dv[s // 32].astype(np.float64)[:, :, None], hq // hkv, axis=1)
        half = np.spacing(np.abs(want).astype(np.float16)).astype(np.float64) / 2
        assert (np.abs(got[at:at + seq - off] - want) <= half + 2.0 ** -21 * np.abs(want)).all()
        at += seq - off
    # without a window, the first token of the two prompts
    first = base._attend(cache, pt, rows, _kinds(rows), hq, q)
    for at in (1 + 6 + 200, 1 + 6 + 200 + 1100):
        np.testing.assert_array_equal(first[at], got[at])
    assert mq.device_error(clear=True) == 0
