"""Tree rows on the GPU: drafted tokens that see their context and, of one another, what a
mask says, against 64-bit attention over the cache's own values.

Bar: 2e-3, as for the library's other rows (N(0, 1) queries and values), and the rounding of
the fp16 output, 2^-11 of the value."""
import numpy as np
import pytest

import _trees as tr

pytestmark = pytest.mark.gpu

DECODE, CHUNK, TREE = 0, 1, 3
FORMATS = [(0, 0), (1, 1), (2, 2), (1, 2), (2, 1), (3, 3), (4, 4)]


def _filled(kf, vf, seqs, hkv, d, seed):
    """A cache whose unwritten slots hold NaN patterns, the page table and each row's slots."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(seed)
    need = [-(-s // 32) for s in seqs]
    pages = sum(need) + 3
    cache = mq.KVCache.allocate(pages, hkv, d, kf, vf, fill=0xFF)
    perm = rng.permutation(pages).astype(np.int32)
    pt = np.full((len(seqs), max(need)), -1, dtype=np.int32)
    slots, at = [], 0
    for r, n in enumerate(need):
        pt[r, :n] = perm[at:at + n]
        at += n
        t = np.arange(seqs[r])
        slots.append(torch.from_numpy((pt[r, t // 32] * 32 + t % 32).astype(np.int32)).cuda())
        k, v = (torch.from_numpy(rng.standard_normal((seqs[r], hkv, d)).astype(np.float16)).cuda() for _ in range(2))
        mq.kv_append_quant(cache, k, v, slots[r])
    return cache, torch.from_numpy(pt).cuda(), slots


def _run(cache, pt, rows, hq, q, masks, window=0, stray=False, words=0):
    import torch
    import mixed_attention_quantized_gb300 as mq
    plan = mq.Plan(cache, hq, [r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows], pt.shape[1],
                   window=window)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    ws.fill_(0xFF)
    out = torch.full_like(q, float("nan"))
    mask = torch.from_numpy(tr.pack(masks, words, stray)).cuda() if masks else None
    plan.run(q, pt, out, ws, tree_mask=mask)
    torch.cuda.synchronize()
    plan.close()
    assert mq.device_error(clear=True) == 0
    return out


def _check(kf, vf, hq, hkv, d, rows, masks, seed, window=0, **kw):
    import torch
    cache, pt, slots = _filled(kf, vf, [r[1] for r in rows], hkv, d, seed)
    total = sum(s - o for _, s, o in rows)
    q = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal((total, hq, d)).astype(np.float16)).cuda()
    got = _run(cache, pt, rows, hq, q, masks, window, **kw)
    at, left = 0, list(masks)
    for r, (kind, s, o) in enumerate(rows):
        k, v = (tr.cache_values(cache, i, slots[r]) for i in (0, 1))
        vis = tr.seen(kind, s, o, left.pop(0) if kind == TREE else None, window)
        want = tr.attention64(q[at:at + s - o], k, v, vis, d ** -0.5)
        err = (got[at:at + s - o].double() - want).abs()
        assert bool((err <= 2e-3 + 2.0 ** -11 * want.abs()).all()), (r, float(err.max()))
        at += s - o
    return got


def _rows_and_masks(spec, seed, roots=2):
    rng = np.random.default_rng(seed)
    rows = [(k, s, o) for k, s, o in spec]
    return rows, [tr.random_tree(s - o, rng, roots) for k, s, o in rows if k == TREE]


# context 0, inside a page, at page and KV-tile borders; 1 to 200 drafted tokens; other kinds beside them
SPEC = [(TREE, 6, 0), (TREE, 41, 40), (TREE, 132, 127), (TREE, 134, 128), (DECODE, 77, 76), (TREE, 64, 31),
        (TREE, 164, 64), (CHUNK, 150, 30), (TREE, 1300, 1267), (TREE, 1232, 1032)]


@pytest.mark.parametrize("kf,vf", FORMATS)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 8, 64), (8, 1, 64)])
def test_trees_beside_other_rows(kf, vf, hq, hkv, d):
    rows, masks = _rows_and_masks(SPEC, 11)
    _check(kf, vf, hq, hkv, d, rows, masks, 12)


@pytest.mark.parametrize("kf,vf", FORMATS)
def test_masks_that_leave_rows_empty_and_stray_bits(kf, vf):
    rng = np.random.default_rng(21)
    rows = [(TREE, 5, 0), (TREE, 50, 0), (TREE, 305, 300), (TREE, 170, 120)]
    masks = []
    for _, s, o in rows:
        m = rng.random((s - o, s - o)) < 0.3  # any mask, tokens that do not see themselves among them
        m[::3] = False
        m[-1] = False
        masks.append(m)
    got = _check(kf, vf, 8, 2, 128, rows, masks, 22, stray=True, words=3)
    assert bool((got[0] == 0).all()) and bool((got[4] == 0).all()) and bool((got[54] == 0).all())


@pytest.mark.parametrize("kf,vf", FORMATS)
@pytest.mark.parametrize("window", [40, 300])
def test_windows_follow_the_depth(kf, vf, window):
    rows, masks = _rows_and_masks([(TREE, 506, 500), (TREE, 33, 20), (TREE, 1000, 965), (DECODE, 700, 699),
                                   (CHUNK, 640, 590), (TREE, 41, 1)], 31)
    masks[0][3] = False  # an empty mask stands at the context's end
    _check(kf, vf, 8, 2, 128, rows, masks, 32, window=window)


@pytest.mark.parametrize("kf,vf", [(0, 0), (1, 1), (4, 4)])
def test_long_contexts_cut_into_pieces(kf, vf):
    rows, masks = _rows_and_masks([(TREE, 9040, 9000), (TREE, 9505, 9500)], 41)
    masks[0][7] = False
    masks[0][7, 39] = True  # only the last key of the row
    _check(kf, vf, 4, 1, 128, rows, masks, 42)


@pytest.mark.parametrize("kf,vf", FORMATS)
def test_a_chain_is_a_verify_row_and_neighbours_keep_their_bits(kf, vf):
    """A tree that is a chain sees what a chunk row sees; and rows of other kinds have the same
    bits whether a tree is in their batch or not."""
    import torch
    spec = [(TREE, 1205, 1200), (DECODE, 400, 399), (CHUNK, 300, 100)]
    cache, pt, _ = _filled(kf, vf, [s for _, s, _ in spec], 2, 128, 51)
    q = torch.randn(206, 8, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(52)).half()
    chain = np.tril(np.ones((5, 5), dtype=bool))
    tree = _run(cache, pt, spec, 8, q, [chain])
    plain = _run(cache, pt, [(CHUNK, 1205, 1200)] + spec[1:], 8, q, [])
    assert torch.equal(tree[5:], plain[5:])
    assert float((tree[:5].float() - plain[:5].float()).abs().max()) <= 2e-3


def test_one_captured_run_serves_changing_trees():
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [(TREE, 325, 300), (TREE, 1004, 1000)]
    cache, pt, slots = _filled(4, 4, [s for _, s, _ in rows], 2, 128, 61)
    q = torch.randn(29, 8, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(62)).half()
    out = torch.empty_like(q)
    plan = mq.Plan(cache, 8, [TREE, TREE], [325, 1004], [300, 1000], pt.shape[1])
    ws = mq.alloc_workspace(plan.workspace_bytes)
    rng = np.random.default_rng(63)
    draws = [[tr.random_tree(25, rng), tr.random_tree(4, rng)] for _ in range(3)]
    mask = torch.from_numpy(tr.pack(draws[0])).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.run(q, pt, out, ws, stream=side, tree_mask=mask)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(q, pt, out, ws, tree_mask=mask)
    for masks in draws:
        mask.copy_(torch.from_numpy(tr.pack(masks)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _run(cache, pt, rows, 8, q, masks))
    graph.reset()
    plan.close()


def test_refusals():
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache, pt, _ = _filled(1, 1, [110], 2, 128, 71)
    q = torch.zeros(40, 8, 128, dtype=torch.float16, device="cuda")
    plan = mq.Plan(cache, 8, [TREE], [110], [70], pt.shape[1])
    ws = mq.alloc_workspace(plan.workspace_bytes)
    with pytest.raises(mq.MixattnError) as e:
        plan.run(q, pt, q, ws)  # a mask is missing
    assert e.value.status == mq.ERR_INVALID_ARG
    with pytest.raises(mq.MixattnError) as e:
        plan.run(q, pt, q, ws, tree_mask=torch.zeros(40, 1, dtype=torch.int32, device="cuda"))
    assert e.value.status == mq.ERR_INVALID_ARG
    for bad in (torch.zeros(39, 2, dtype=torch.int32, device="cuda"), torch.zeros(40, 2, device="cuda"),
                torch.zeros(40, 2, dtype=torch.int32), torch.zeros(80, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            plan.run(q, pt, q, ws, tree_mask=bad)
    plan.close()
    for call in (mq.mixed_attention, mq.mixed_attention_noalloc):
        with pytest.raises(mq.MixattnError) as e:
            call(cache, q, pt, [110], [70], [TREE])
        assert e.value.status in (mq.ERR_INVALID_ARG, mq.ERR_UNSUPPORTED)


@pytest.mark.parametrize("kf,vf", FORMATS)
@pytest.mark.parametrize("d,window", [(128, 0), (64, 0), (64, 300)])
def test_nodes_that_nobody_sees_need_not_be_in_the_cache(kf, vf, d, window):
    """Padded trees: the last nodes' masks are empty, no other names them, and they were never appended, so that
    their places in the cache, and the scales of whole pages, are NaN patterns."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(91)
    rows = [(TREE, 70, 30), (DECODE, 40, 39), (TREE, 36, 31), (TREE, 38, 32), (TREE, 360, 131), (TREE, 164, 0), (CHUNK, 90, 60)]
    used = [25, 1, 2, 1, 9, 1, 30]
    masks = []
    for (kind, s, o), u in zip(rows, used):
        if kind == TREE:
            m = np.zeros((s - o, s - o), dtype=bool)
            m[:u, :u] = tr.random_tree(u, rng)
            masks.append(m)
    seqs = [r[1] for r in rows]
    need = [-(-s // 32) for s in seqs]
    cache = mq.KVCache.allocate(sum(need) + 3, 2, d, kf, vf, fill=0xFF)
    perm = rng.permutation(sum(need) + 3).astype(np.int32)
    pt = np.full((len(seqs), max(need)), -1, dtype=np.int32)
    slots, at = [], 0
    for r, n in enumerate(need):
        pt[r, :n] = perm[at:at + n]
        at += n
        t = np.arange(seqs[r])
        slots.append(torch.from_numpy((pt[r, t // 32] * 32 + t % 32).astype(np.int32)).cuda())
        here = rows[r][2] + used[r]
        k, v = (torch.from_numpy(rng.standard_normal((here, 2, d)).astype(np.float16)).cuda() for _ in range(2))
        mq.kv_append_quant(cache, k, v, slots[r][:here])
    pt = torch.from_numpy(pt).cuda()
    total = sum(s - o for _, s, o in rows)
    q = torch.from_numpy(rng.standard_normal((total, 8, d)).astype(np.float16)).cuda()
    got = _run(cache, pt, rows, 8, q, masks, window)
    at, left = 0, list(masks)
    for r, (kind, s, o) in enumerate(rows):
        k, v = (tr.cache_values(cache, i, slots[r]) for i in (0, 1))
        vis = tr.seen(kind, s, o, left.pop(0) if kind == TREE else None, window)
        want = tr.attention64(q[at:at + s - o], k, v, vis, d ** -0.5)
        err = (got[at:at + s - o].double() - want).abs()
        assert bool((err <= 2e-3 + 2.0 ** -11 * want.abs()).all()), (r, float(err.max()))
        at += s - o
