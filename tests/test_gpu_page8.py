"""The page-scaled 8-bit formats on the GPU: appends bit for bit against the documented
fp32 steps, attention against fp64 over the device's own codes."""
import numpy as np
import pytest

import _page8 as ref

pytestmark = pytest.mark.gpu

FORMATS = [ref.I8, ref.E4M3]


def _alloc(fmt, pages, hkv, d, fill=0):
    import mixed_attention_quantized_gb300 as mq
    return mq.KVCache.allocate(pages, hkv, d, fmt, fmt, fill=fill)


def _planes(cache):
    """(K codes as values, K scales, V codes, V scales) from the device."""
    import torch
    torch.cuda.synchronize()
    shape = (cache.num_pages, cache.num_kv_heads, 32, cache.head_dim)
    out = []
    for q, s in ((cache.k_quant, cache.k_scale), (cache.v_quant, cache.v_scale)):
        out.append(ref.raw_codes(cache.k_fmt, q.cpu().numpy()).reshape(shape))
        out.append(s.cpu().numpy().view(np.float32).reshape(shape[:2]))
    return out


def _append(cache, k, v, slots):
    import torch
    import mixed_attention_quantized_gb300 as mq
    mq.kv_append_quant(cache, torch.from_numpy(np.ascontiguousarray(k)).cuda(),
                       torch.from_numpy(np.ascontiguousarray(v)).cuda(),
                       torch.from_numpy(np.asarray(slots, dtype=np.int32)).cuda())


def _same(cache, k_ref, v_ref, pages):
    kq, ks, vq, vs = _planes(cache)
    for q, s, r in ((kq, ks, k_ref), (vq, vs, v_ref)):
        np.testing.assert_array_equal(s[pages], r.scale[pages])
        np.testing.assert_array_equal(q[pages], r.codes[pages])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,order", [(1, "in"), (31, "in"), (33, "in"), (257, "in"), (700, "mixed"), (1500, "mixed"),
                                     (1030, "in"), (5003, "in"), (9000, "mixed"), (20001, "in")])
def test_append_is_bit_exact(fmt, d, n, order):
    """One call of n tokens into fresh pages and into partly filled ones."""
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(n + d)
    hkv, pages = 3, n // 32 + 4
    cache = _alloc(fmt, pages, hkv, d)
    kr, vr = ref.PageCache(fmt, pages, hkv, d), ref.PageCache(fmt, pages, hkv, d)
    perm = rng.permutation(pages)
    old = 13  # tokens already there
    for first, cnt in ((0, old), (old, n)):
        t = np.arange(first, first + cnt)
        slots = perm[t // 32] * 32 + t % 32
        if order == "mixed" and first:
            slots = rng.permutation(slots)  # a page's tokens far apart in the call
            slots[::9] = -1
        x = rng.standard_normal((2, cnt, hkv, d)) * np.exp2(rng.integers(-8, 8, size=(1, cnt, hkv, 1)))
        x = x.astype(np.float16)
        x[0, ::5] = 0
        _append(cache, x[0], x[1], slots)
        kr.append(x[0], slots)
        vr.append(x[1], slots)
    assert mq.device_error(clear=True) == 0
    _same(cache, kr, vr, np.arange(pages))


@pytest.mark.parametrize("fmt", FORMATS)
def test_scale_grows_token_by_token_and_restarts(fmt):
    rng = np.random.default_rng(7)
    hkv, d = 2, 128
    cache = _alloc(fmt, 3, hkv, d, fill=0xFF)  # scales NaN, codes NaN patterns
    kr, vr = ref.PageCache(fmt, 3, hkv, d), ref.PageCache(fmt, 3, hkv, d)
    for turn in range(2):  # the second turn reuses the page
        for t in range(32):
            x = (rng.standard_normal((2, 1, hkv, d)) * 2.0 ** (t % 7 if turn else t / 3)).astype(np.float16)
            _append(cache, x[0], x[1], [32 + t])
            kr.append(x[0], [32 + t])
            vr.append(x[1], [32 + t])
        _same(cache, kr, vr, [1])
    # the neighbours keep every byte
    raw = cache.k_quant.cpu().numpy().reshape(3, -1)
    assert (raw[[0, 2]] == 0xFF).all()
    assert (cache.k_scale.cpu().numpy().reshape(3, -1)[[0, 2]] == 0xFF).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_same_slot_twice_bad_slots_and_odd_values(fmt):
    import torch
    import mixed_attention_quantized_gb300 as mq
    mq.device_error(clear=True)
    hkv, d = 1, 64
    cache = _alloc(fmt, 2, hkv, d)
    kr, vr = ref.PageCache(fmt, 2, hkv, d), ref.PageCache(fmt, 2, hkv, d)
    x = np.random.default_rng(1).standard_normal((6, hkv, d)).astype(np.float16)
    x[1, 0, :4] = [np.inf, -np.inf, np.nan, 65504]
    x[5] *= 0
    slots = [0, 1, 2, 1, 64, 33]  # slot 1 twice (the later counts), 64 outside, 33 of a page never started
    x[3, 0, :3] = [np.nan, np.inf, -3]
    _append(cache, x, -x, slots)
    kr.append(x, [0, 1, 2, 1, -1, 33])
    vr.append(-x, [0, 1, 2, 1, -1, 33])
    torch.cuda.synchronize()
    assert mq.device_error(clear=True) == mq.DEVERR_SLOT
    _same(cache, kr, vr, [0, 1])
    _append(cache, x[:0], x[:0], [])


@pytest.mark.parametrize("fmt", FORMATS)
def test_export_blocks(fmt):
    import torch
    import mixed_attention_quantized_gb300 as mq
    hkv, d = 2, 128
    cache = _alloc(fmt, 3, hkv, d)
    x = np.random.default_rng(2).standard_normal((40, hkv, d)).astype(np.float16)
    _append(cache, x, 2 * x, np.arange(40))
    s = np.array([0, 31, 32, 39], dtype=np.int32)
    kq, ks, vq, vs = _planes(cache)
    for which, q, sc in ((0, kq, ks), (1, vq, vs)):
        b = mq.kv_export_blocks(cache, which, torch.from_numpy(s).cuda()).cpu().numpy()
        assert b.shape == (4, hkv, 4, 36)
        np.testing.assert_array_equal(b[..., :4].copy().view(np.float32)[..., 0], np.repeat(sc[s // 32][..., None], 4, 2))
        np.testing.assert_array_equal(ref.raw_codes(fmt, np.ascontiguousarray(b[..., 4:])).reshape(4, hkv, d),
                                      q[s // 32, :, s % 32])


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def _filled(fmt, rows, hkv, d, seed, gains=None, spare=2, fill=0xFF):
    """A cache holding every row's keys, its page table, and each row's slots.
    gains(rng, n) -> per-token multipliers of V."""
    rng = np.random.default_rng(seed)
    need = [-(-s // 32) for s, _ in rows]
    pages = sum(need) + spare
    perm = rng.permutation(pages).astype(np.int32)
    pt = np.full((len(rows), max(need) + 1), -1, dtype=np.int32)
    cache = _alloc(fmt, pages, hkv, d, fill=fill)
    at, row_slots = 0, []
    for r, (seq, _) in enumerate(rows):
        pt[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
        t = np.arange(seq)
        slots = pt[r, t // 32] * 32 + t % 32
        k, v = rng.standard_normal((2, seq, hkv, d))
        k[:, :, rng.integers(0, d, 3)] *= 8
        if gains is not None:
            v *= gains(rng, seq)[:, None, None]
        _append(cache, k.astype(np.float16), np.clip(v, -65504, 65504).astype(np.float16), slots)
        row_slots.append(slots)
    return cache, pt, row_slots


def _attend(cache, pt, rows, kinds, hq, q, window=0):
    import torch
    import mixed_attention_quantized_gb300 as mq
    seqs, offs = [r[0] for r in rows], [r[1] for r in rows]
    plan = mq.Plan(cache, hq, kinds, seqs, offs, pt.shape[1], window=window)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    ws.fill_(0xA5)
    # rows behind the last query stay as they were
    o = torch.full((q.shape[0] + 3, hq, cache.head_dim), float("nan"), dtype=torch.float16, device="cuda")
    plan.run(torch.from_numpy(q).cuda(), torch.from_numpy(pt).cuda(), o, ws)
    torch.cuda.synchronize()
    assert torch.isnan(o[q.shape[0]:]).all()
    plan.close()
    return o[:q.shape[0]].cpu().numpy().astype(np.float64)


def _check(fmt, rows, kinds, hq, hkv, d, seed, window=0, gains=None, q_gain=1.0):
    import mixed_attention_quantized_gb300 as mq
    cache, pt, row_slots = _filled(fmt, rows, hkv, d, seed, gains)
    total = sum(s - o for s, o in rows)
    q = (np.random.default_rng(seed + 1).standard_normal((total, hq, d)) * q_gain).astype(np.float16)
    got = _attend(cache, pt, rows, kinds, hq, q, window)
    assert mq.device_error(clear=True) == 0
    kq, ks, vq, vs = _planes(cache)
    used = np.unique(np.concatenate(row_slots) // 32)
    ks0, vs0 = (np.where(np.isin(np.arange(len(s)), used)[:, None], s, 0).astype(np.float64) for s in (ks, vs))
    kv = (np.nan_to_num(kq) * ks0[:, :, None, None], np.nan_to_num(vq) * vs0[:, :, None, None])
    want, size = ref.attention(q, kv, row_slots, rows, window)
    tol = ref.attention_tolerance(fmt, q, want, size, ks0, vs0, max(s for s, _ in rows))
    bad = np.abs(got - want) > tol
    assert np.isfinite(got).all() and not bad.any(), (np.abs(got - want).max(), (np.abs(got - want) / tol).max())
    return got


DECODE = [(1, 0), (2, 1), (31, 30), (32, 31), (33, 32), (100, 99), (300, 299), (1000, 999), (2309, 2308)]
CHUNK = [(1, 0), (5, 0), (33, 30), (100, 94), (64, 0), (192, 128), (130, 0), (257, 0), (700, 500), (1100, 1099)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (4, 2), (8, 1)])
def test_decode_rows(fmt, d, hq, hkv):
    _check(fmt, DECODE, [0] * len(DECODE), hq, hkv, d, seed=hq * 10 + d)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (4, 2), (8, 1)])
def test_chunk_rows(fmt, d, hq, hkv):
    _check(fmt, CHUNK, [1] * len(CHUNK), hq, hkv, d, seed=hq * 10 + d + 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 31, 33, 300, 5000])
def test_windows(fmt, window):
    rows = DECODE + CHUNK
    _check(fmt, rows, [0] * len(DECODE) + [1] * len(CHUNK), 8, 2, 128, seed=window, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_rows_split(fmt):
    rows = [(40000, 39999), (20011, 19900), (9000, 8997)]
    _check(fmt, rows, [0, 1, 1], 4, 1, 128, seed=77)


CUT = [(7, 1030), (13, 1500), (16, 2309), (25, 1111), (32, 2000), (33, 3001), (50, 1400), (64, 1290), (65, 1025), (130, 4000)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,d,window", [(4, 1, 128, 0), (4, 1, 64, 0), (8, 1, 128, 0), (2, 2, 128, 0), (16, 2, 64, 1100)])
def test_cut_tiles_of_every_row_count(fmt, hq, hkv, d, window):
    """Key ranges of few long tiles are cut into pieces that the last to finish joins: tiles of one to
    eight 32-row blocks, the last ones partly filled, and the same bits from every run."""
    rows = [(c + n, c) for n, c in CUT]
    got = _check(fmt, rows, [1] * len(rows), hq, hkv, d, seed=13 + hq, window=window)
    cache, pt, _ = _filled(fmt, rows, hkv, d, 13 + hq)
    q = np.random.default_rng(14 + hq).standard_normal((got.shape[0], hq, d)).astype(np.float16)
    for _ in range(3):
        np.testing.assert_array_equal(_attend(cache, pt, rows, [1] * len(rows), hq, q, window), got)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64)])
def test_more_chunk_tiles_than_ctas(fmt, hq, hkv, d):
    """Enough chunk tiles that a CTA walks several, of uneven lengths and half-empty ones."""
    rows = [(1500, 0), (400, 399), (1300, 500), (200, 170)]
    if hq == hkv:
        rows = [(3000, 0), (2100, 100), (600, 599)]
    _check(fmt, rows, [0 if s - o == 1 else 1 for s, o in rows], hq, hkv, d, seed=61)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_page_scales_far_apart(fmt, d):
    """Pages of V 2^24 apart in size, and pages of zeros: each weighs in at its own scale."""
    def gains(rng, n):
        g = np.exp2(rng.integers(-12, 12, size=-(-n // 32)).astype(float))
        g[rng.random(len(g)) < 0.2] = 0
        return g.repeat(32)[:n]
    rows = [(500, 499), (1500, 1499), (200, 100), (700, 690), (33, 32)]
    _check(fmt, rows, [0, 0, 1, 1, 0], 4, 2, d, seed=3, gains=gains)
    # where every page of V is small, so are the errors
    _check(fmt, rows, [0, 0, 1, 1, 0], 4, 2, d, seed=4, gains=lambda rng, n: np.full(n, 2.0 ** -14))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_gain", [0.0, 1e-4, 6.0])
def test_flat_and_sharp_scores(fmt, q_gain):
    rows = [(700, 699), (300, 0), (40, 36)]
    _check(fmt, rows, [0, 1, 1], 8, 2, 128, seed=11, q_gain=q_gain)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_rows_bits_do_not_depend_on_its_batch(fmt):
    hq, hkv, d = 8, 2, 128
    rows, kinds = [(900, 899), (700, 500), (333, 330)], [0, 1, 1]
    cache, pt, _ = _filled(fmt, rows, hkv, d, 21)
    q = np.random.default_rng(22).standard_normal((204, hq, d)).astype(np.float16)
    whole = _attend(cache, pt, rows, kinds, hq, q)
    at = 0
    for r, (s, o) in enumerate(rows):
        alone = _attend(cache, pt[r:r + 1], rows[r:r + 1], kinds[r:r + 1], hq, q[at:at + s - o])
        np.testing.assert_array_equal(alone, whole[at:at + s - o])
        at += s - o


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_pages_are_flagged_and_skipped(fmt):
    import mixed_attention_quantized_gb300 as mq
    mq.device_error(clear=True)
    rows = [(100, 99), (200, 100)]
    cache, pt, row_slots = _filled(fmt, rows, 1, 64, 31)
    q = np.random.default_rng(1).standard_normal((101, 4, 64)).astype(np.float16)
    pt[0, 1], pt[1, 2] = cache.num_pages, -5
    got = _attend(cache, pt, rows, [0, 1], 4, q)
    assert mq.device_error(clear=True) == mq.DEVERR_PAGE_ID
    assert np.isfinite(got).all()
    # the decode row is attention without the bad page's keys
    kq, ks, vq, vs = _planes(cache)
    s = np.delete(row_slots[0], np.arange(32, 64))
    k, v = (np.nan_to_num(c) * np.nan_to_num(x)[:, :, None, None].astype(np.float64) for c, x in ((kq, ks), (vq, vs)))
    want, _ = ref.attention(q[:1], (k, v), [s], [(len(s), len(s) - 1)])
    assert np.abs(got[:1] - want).max() <= 2e-3


@pytest.mark.parametrize("fmt", FORMATS)
def test_steps_of_a_serving_loop(fmt):
    """Prefill in chunks, then decode: rotary append and attention step by step, twice through
    one captured graph, against fp64 over what the cache then holds."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    hq, hkv, d, prompt, chunk = 8, 2, 128, 150, 64
    rng = np.random.default_rng(41)
    rope = mq.Rope(64, layout=mq.ROPE_INTERLEAVED, scaling=mq.ROPE_SCALE_LINEAR, factor=4.0)
    freq, m = ref.frequencies(64, "linear", factor=4.0)
    pages = 8
    cache = _alloc(fmt, pages, hkv, d, fill=0xFF)
    perm = rng.permutation(pages).astype(np.int32)
    pt = perm[None, :]
    ptd = torch.from_numpy(pt).cuda()
    at, plan = 0, None
    for n in [64, 64, 22] + [1] * 6 + [4]:
        kind = 0 if n == 1 else 1
        pos = np.arange(at, at + n, dtype=np.int32)
        slots = (perm[pos // 32] * 32 + pos % 32).astype(np.int32)
        q, k, v = (rng.standard_normal((n, h, d)).astype(np.float16) for h in (hq, hkv, hkv))
        qd, kd, vd = (torch.from_numpy(x).cuda() for x in (q, k, v))
        qr = mq.rope_append(cache, rope, qd, kd, vd, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda())
        if plan is None:
            plan = mq.Plan(cache, hq, [kind], [at + n], [at], pages)
        else:
            plan.update([kind], [at + n], [at], pages)
        ws = mq.alloc_workspace(plan.workspace_bytes)
        o = torch.empty_like(qr)
        plan.run(qr, ptd, o, ws)
        at += n
        kq, ks, vq, vs = _planes(cache)
        used = np.isin(np.arange(pages), perm[:-(-at // 32)])[:, None]
        ks, vs = (np.where(used, s, 0).astype(np.float64) for s in (ks, vs))
        kv = (np.nan_to_num(kq) * ks[:, :, None, None], np.nan_to_num(vq) * vs[:, :, None, None])
        all_slots = perm[np.arange(at) // 32] * 32 + np.arange(at) % 32
        qn = qr.cpu().numpy()
        want, size = ref.attention(qn, kv, [all_slots], [(at, at - n)])
        tol = ref.attention_tolerance(fmt, qn, want, size, ks, vs, at)
        assert (np.abs(o.cpu().numpy() - want) <= tol).all()
        # rotated keys of this step, within the format's step of the definition
        got = kv[0][slots // 32, :, slots % 32]
        exact = ref.rotate(k, pos, freq, m, 64, True)
        step = ks[slots // 32][..., None]
        half = step * 0.501 if fmt == ref.I8 else np.maximum(2.0 ** -4 * np.abs(exact), step * 2.0 ** -10)
        assert (np.abs(got - exact) <= half * (1 + 1e-5) + 1e-5).all()
    assert mq.device_error(clear=True) == 0

    # the last step captured and replayed: the same bytes, however often
    x = [torch.from_numpy(a).cuda() for a in (q, k, v)]
    pd, sd = torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda()
    out = torch.empty_like(x[0])
    mq.rope_append(cache, rope, *x, pd, sd, out)
    torch.cuda.synchronize()
    before = [t.clone() for t in (out, cache.k_quant, cache.v_quant, cache.k_scale)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.rope_append(cache, rope, *x, pd, sd, out)
    out.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(before, (out, cache.k_quant, cache.v_quant, cache.k_scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [1, ref.I8, ref.E4M3])
def test_run_captured_and_replayed(fmt):
    """A captured run replays on new queries and keys; its plan refuses another batch, and what
    is called afterwards still works."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows, hq = [(300, 299), (400, 200), (70, 66)], 8
    cache, pt, _ = _filled(fmt, rows, 2, 128, 51)
    n = sum(s - o for s, o in rows)
    rng = np.random.default_rng(52)
    q = torch.from_numpy(rng.standard_normal((n, hq, 128)).astype(np.float16)).cuda()
    ptd = torch.from_numpy(pt).cuda()
    seqs, offs = [r[0] for r in rows], [r[1] for r in rows]
    plan = mq.Plan(cache, hq, [0, 1, 1], seqs, offs, pt.shape[1])
    ws = mq.alloc_workspace(plan.workspace_bytes)
    o = torch.empty_like(q)
    plan.run(q, ptd, o, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(q, ptd, o, ws)
    other = mq.Plan(cache, hq, [0, 1, 1], seqs, offs, pt.shape[1])
    for _ in range(2):
        q.copy_(torch.from_numpy(rng.standard_normal((n, hq, 128)).astype(np.float16)))
        want = torch.empty_like(o)
        other.run(q, ptd, want, mq.alloc_workspace(other.workspace_bytes))
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    with pytest.raises(mq.MixattnError) as e:
        plan.update([0], [100], [99], pt.shape[1])
    assert e.value.status == mq.ERR_UNSUPPORTED
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    del g
    plan.close()
    other.update([0], [300], [299], pt.shape[1])  # a plan that was not captured goes on
    other.run(q, ptd, o, mq.alloc_workspace(other.workspace_bytes))
    torch.cuda.synchronize()
    other.close()


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_call_entry_point(fmt):
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows, kinds = [(300, 299), (400, 200), (70, 66)], [0, 1, 1]
    cache, pt, _ = _filled(fmt, rows, 2, 64, 71)
    q = np.random.default_rng(72).standard_normal((205, 8, 64)).astype(np.float16)
    want = _attend(cache, pt, rows, kinds, 8, q)
    got = mq.mixed_attention(cache, torch.from_numpy(q).cuda(), torch.from_numpy(pt).cuda(), [r[0] for r in rows],
                             [r[1] for r in rows], kinds)
    np.testing.assert_array_equal(got.cpu().numpy().astype(np.float64), want)
    with pytest.raises(mq.MixattnError) as e:
        mq.mixed_attention_noalloc(cache, torch.from_numpy(q).cuda(), torch.from_numpy(pt).cuda(),
                                   [r[0] for r in rows], [r[1] for r in rows], kinds)
    assert e.value.status == mq.ERR_UNSUPPORTED


@pytest.mark.parametrize("fmt", FORMATS)
def test_planes_past_four_gigabytes(fmt):
    """Pages whose offsets need more than 32 bits, at both ends of the pool."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    hkv, d, pages = 8, 128, 140_000  # 4.6 GB of codes for each of K and V
    cache = _alloc(fmt, pages, hkv, d, fill=None)
    ids = np.array([pages - 1, 0, pages - 7, 131_072, 131_071], dtype=np.int32)
    seq, off, hq = 150, 100, 32
    rng = np.random.default_rng(81)
    k, v = rng.standard_normal((2, seq, hkv, d)).astype(np.float16)
    t = np.arange(seq)
    slots = ids[t // 32] * 32 + t % 32
    _append(cache, k, v, slots)
    q = rng.standard_normal((seq - off + 1, hq, d)).astype(np.float16)
    pt = np.stack([ids, ids])
    got = _attend(cache, pt, [(seq, off), (seq, seq - 1)], [1, 0], hq, q)
    assert mq.device_error(clear=True) == 0
    kv, scales = [], []
    for x in (k, v):
        r = ref.PageCache(fmt, 5, hkv, d)  # the same appends into a pool of five pages
        r.append(x, t)
        kv.append(r.values())
        scales.append(r.scale.astype(np.float64))
    want, size = ref.attention(q, kv, [t, t], [(seq, off), (seq, seq - 1)])
    assert (np.abs(got - want) <= ref.attention_tolerance(fmt, q, want, size, *scales, seq)).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_append_captured_and_replayed(fmt):
    """An append long enough for clusters, with rotary keys: captured, replayed on other inputs."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    n, hq, hkv, d, pages = 1500, 4, 3, 128, 60
    rng = np.random.default_rng(91)
    rope = mq.Rope(128)
    slots = torch.from_numpy(rng.permutation(pages * 32)[:n].astype(np.int32)).cuda()
    pos = torch.from_numpy(rng.integers(0, 100000, n).astype(np.int32)).cuda()
    q, k, v = (torch.randn(n, h, d, device="cuda").half() for h in (hq, hkv, hkv))
    a, b = _alloc(fmt, pages, hkv, d), _alloc(fmt, pages, hkv, d)
    oa, ob = torch.empty_like(q), torch.empty_like(q)
    mq.rope_append(a, rope, q, k, v, pos, slots, oa)
    torch.cuda.synchronize()
    for t in (a.k_quant, a.v_quant, a.k_scale, a.v_scale):
        t.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.rope_append(a, rope, q, k, v, pos, slots, oa)
    for _ in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn_like(x))
        g.replay()
        mq.rope_append(b, rope, q, k, v, pos, slots, ob)
        torch.cuda.synchronize()
        for x, y in ((oa, ob), (a.k_quant, b.k_quant), (a.v_quant, b.v_quant), (a.k_scale, b.k_scale)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_streams_at_once(fmt):
    """Two batches side by side on two streams, each with its own plan and workspace."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    jobs = []
    for seed, rows, kinds in ((1, [(3000, 2000), (5000, 4999), (900, 896)], [1, 0, 1]),
                              (2, [(2500, 0), (7000, 6999)], [1, 0])):
        cache, pt, _ = _filled(fmt, rows, 4, 128, seed)
        n = sum(s - o for s, o in rows)
        q = torch.from_numpy(np.random.default_rng(seed).standard_normal((n, 16, 128)).astype(np.float16)).cuda()
        plan = mq.Plan(cache, 16, kinds, [r[0] for r in rows], [r[1] for r in rows], pt.shape[1])
        jobs.append((plan, q, torch.from_numpy(pt).cuda(), torch.empty_like(q), mq.alloc_workspace(plan.workspace_bytes)))
    want = []
    for plan, q, pt, o, ws in jobs:
        plan.run(q, pt, o, ws)
        torch.cuda.synchronize()
        want.append(o.clone())
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        for (plan, q, pt, o, ws), s in zip(jobs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                o.zero_()
                plan.run(q, pt, o, ws)
        torch.cuda.synchronize()
        for (_, _, _, o, _), w in zip(jobs, want):
            assert torch.equal(o, w)
    assert mq.device_error(clear=True) == 0
