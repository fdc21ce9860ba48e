"""Absorbed latent attention on the GPU against 64 bits, within the bound of `_latent.attention64`."""
import numpy as np
import pytest

import _latent as la
import _trees as tr

pytestmark = pytest.mark.gpu

DECODE, CHUNK, TREE = 0, 1, 3
SCALE = 192 ** -0.5


def _run(cache, pt, rows, heads, q, masks=(), scale=SCALE, plan=None, stray=False):
    import torch
    import mixed_attention_quantized_gb300 as mq
    own = plan is None
    if own:
        plan = mq.LatentPlan(cache, heads, [r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows],
                             pt.shape[1], scale)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    ws.fill_(0xFF)
    out = torch.full((q.shape[0], heads, 512), float("nan"), dtype=torch.float16, device="cuda")
    plan.run(q, pt, out, ws, tree_mask=torch.from_numpy(tr.pack(masks, 0, stray)).cuda() if len(masks) else None)
    torch.cuda.synchronize()
    if own:
        plan.close()
    return out


def _check(rows, heads, masks=(), seed=1, scale=SCALE, size=0.5, **kw):
    import mixed_attention_quantized_gb300 as mq
    cache, pt, slots = la.paged([r[1] for r in rows], seed)
    q = la.queries(sum(s - o for _, s, o in rows), heads, 576, seed + 1, size)
    got = _run(cache, pt, rows, heads, q, masks, scale, **kw)
    assert mq.device_error(clear=True) == 0
    at, left = 0, list(masks)
    for r, (kind, s, o) in enumerate(rows):
        k = cache.data.view(-1, 576)[slots[r]][:, None]
        vis = la.seen(kind, s, o, left.pop(0) if kind == TREE else None)
        want, bound = la.attention64(q[at:at + s - o], k, k[..., :512], vis, scale)
        la.check(got[at:at + s - o], want, bound, (r, kind, s, o))
        at += s - o
    return got


def test_one_key():
    _check([(DECODE, 1, 0)], 16)


@pytest.mark.parametrize("heads", [1, 5, 8, 16, 20, 32, 64, 100, 128])
def test_decode_rows_of_all_lengths(heads):
    _check([(DECODE, s, s - 1) for s in (1, 2, 31, 32, 33, 63, 64, 65, 96, 100, 300, 1000)], heads, seed=heads)


@pytest.mark.parametrize("heads", [8, 16, 64, 128])
def test_chunk_rows_beside_decode_rows(heads):
    _check([(CHUNK, 3, 0), (CHUNK, 40, 30), (DECODE, 500, 499), (CHUNK, 130, 128), (CHUNK, 700, 693), (CHUNK, 96, 0),
            (DECODE, 33, 32)], heads, seed=20 + heads)


@pytest.mark.parametrize("heads", [4, 16, 48, 128])
def test_trees(heads):
    rng = np.random.default_rng(31)
    rows = [(TREE, 6, 0), (TREE, 41, 40), (DECODE, 77, 76), (TREE, 134, 128), (TREE, 164, 124), (CHUNK, 60, 50)]
    masks = [tr.random_tree(s - o, rng, 2) for k, s, o in rows if k == TREE]
    masks[0][2] = False  # sees nothing: zeros
    masks[3][7] = False
    got = _check(rows, heads, masks, seed=32, stray=True)
    assert bool((got[2] == 0).all())


@pytest.mark.parametrize("heads", [1, 16, 128])
def test_nodes_that_nobody_sees_may_hold_anything(heads):
    """A padded tree: the masks of its last nodes are empty, no other names them, and their rows of the cache
    are NaN; no output of the batch notices."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(71)
    rows = [(TREE, 70, 30), (DECODE, 40, 39), (TREE, 203, 131), (TREE, 64, 0)]
    used = [25, 7, 1]
    masks = []
    for (s, o), u in zip([r[1:] for r in rows if r[0] == TREE], used):
        m = np.zeros((s - o, s - o), dtype=bool)
        m[:u, :u] = tr.random_tree(u, rng)
        masks.append(m)
    cache, pt, slots = la.paged([r[1] for r in rows], 72)
    q = la.queries(sum(s - o for _, s, o in rows), heads, 576, 73)
    want = _run(cache, pt, rows, heads, q, masks)
    flat = cache.data.view(-1, 576)
    for r, u in zip((0, 2, 3), used):
        flat[slots[r][rows[r][2] + u:]] = float("nan")
    got = _run(cache, pt, rows, heads, q, masks)
    assert mq.device_error(clear=True) == 0
    assert torch.equal(got, want) and bool(got.isfinite().all())
    assert bool((got[-63:] == 0).all())  # (no context: they see nothing)


def test_a_tree_of_1024_nodes_and_one_of_a_single_node():
    rng = np.random.default_rng(75)
    masks = [tr.random_tree(1024, rng, 3), tr.random_tree(1, rng)]
    _check([(TREE, 1124, 100), (TREE, 1, 0)], 8, masks, seed=76)


@pytest.mark.parametrize("heads", [16, 128])
def test_long_rows_are_cut_and_joined(heads):
    _check([(DECODE, 9000, 8999), (DECODE, 20, 19), (DECODE, 4001, 4000), (CHUNK, 3000, 2997)], heads, seed=41)


def test_a_long_causal_chunk():
    _check([(CHUNK, 700, 100)], 16, seed=51)


def test_scores_that_move_the_reference():
    """Queries ten times the usual size: one key weighs nearly all, and later keys pass the reference."""
    _check([(DECODE, 3000, 2999), (CHUNK, 260, 256), (DECODE, 130, 129)], 16, seed=61, size=5.0)


def test_rising_scores():
    """Keys along the query, each page's larger than the last's, so that every step moves the reference."""
    import torch
    rows = [(DECODE, 640, 639)]
    cache, pt, slots = la.paged([640], 62)
    q = la.queries(1, 16, 576, 63, 1.0)
    flat = cache.data.view(-1, 576)
    flat[slots[0]] = ((flat[slots[0]].float() * 0.1) + torch.arange(640, device="cuda")[:, None] / 32 * 0.15 *
                      q[0, 0].float()).half()
    got = _run(cache, pt, rows, 16, q)
    k = flat[slots[0]][:, None]
    want, bound = la.attention64(q, k, k[..., :512], la.seen(DECODE, 640, 639), SCALE)
    la.check(got, want, bound)


def test_the_same_bits_from_every_run_and_after_an_update():
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [(DECODE, 5000, 4999), (CHUNK, 900, 896), (DECODE, 70, 69)]
    cache, pt, _ = la.paged([r[1] for r in rows], 71)
    q = la.queries(6, 64, 576, 72)
    first = _run(cache, pt, rows, 64, q)
    for _ in range(3):
        assert torch.equal(first, _run(cache, pt, rows, 64, q))
    plan = mq.LatentPlan(cache, 64, [DECODE], [32], [31], pt.shape[1], SCALE)
    plan.update([r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows], pt.shape[1])
    assert torch.equal(first, _run(cache, pt, rows, 64, q, plan=plan))
    plan.close()


def test_captured_and_on_another_stream():
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [(DECODE, 3000, 2999), (DECODE, 70, 69)]
    cache, pt, _ = la.paged([r[1] for r in rows], 81)
    q = la.queries(2, 16, 576, 82)
    want = _run(cache, pt, rows, 16, q)
    plan = mq.LatentPlan(cache, 16, [0, 0], [3000, 70], [2999, 69], pt.shape[1], SCALE)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan.run(q, pt, out, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(q, pt, out, ws)
    with pytest.raises(mq.MixattnError) as e:
        plan.update([0], [32], [31], pt.shape[1])
    assert e.value.status == mq.ERR_UNSUPPORTED
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph.reset()
    plan.close()


def test_bad_pages_are_left_out_and_reported():
    import mixed_attention_quantized_gb300 as mq
    rows = [(DECODE, 300, 299), (DECODE, 40, 39), (DECODE, 70, 69)]
    cache, pt, slots = la.paged([r[1] for r in rows], 91)
    q = la.queries(3, 16, 576, 92)
    pt[0, 3], pt[0, 9] = 10 ** 6, -7  # (the second is the row's last, partly filled page)
    pt[1, 0] = pt[1, 1] = cache.num_pages
    got = _run(cache, pt, rows, 16, q)
    assert mq.device_error() == mq.DEVERR_PAGE_ID
    with pytest.raises(mq.MixattnError) as e:
        _run(cache, pt, rows, 16, q)
    assert e.value.status == mq.ERR_DEVICE_CHECK
    mq.device_error(clear=True)
    for r, (kind, s, o) in enumerate(rows):
        vis = la.seen(kind, s, o)
        if r == 0:
            vis[:, 96:128] = vis[:, 288:] = False
        if r == 1:
            vis[:] = False
        k = cache.data.view(-1, 576)[slots[r]][:, None]
        want, bound = la.attention64(q[r:r + 1], k, k[..., :512], vis, SCALE)
        la.check(got[r:r + 1], want, bound, r)


def test_refusals():
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache, pt, _ = la.paged([100], 95)
    q = la.queries(1, 16, 576, 96)
    o = torch.empty(1, 16, 512, dtype=torch.float16, device="cuda")

    def status(*a):
        with pytest.raises(mq.MixattnError) as e:
            mq.LatentPlan(cache, *a)
        return e.value.status

    assert status(129, [0], [100], [99], 4, SCALE) == mq.ERR_UNSUPPORTED
    assert status(16, [3], [1100], [0], 40, SCALE) == mq.ERR_INVALID_ARG  # more pages than the cache has
    for bad in ((0, [0], [100], [99], 4, SCALE), (16, [0], [100], [98], 4, SCALE), (16, [2], [100], [99], 4, SCALE),
                (16, [0], [100], [99], 3, SCALE), (16, [], [], [], 4, SCALE), (16, [1], [100], [100], 4, SCALE),
                (16, [0], [100], [99], 4, 0.0), (16, [0], [100], [99], 4, float("nan")), (16, [0], [100], [99], 4, -1.0)):
        assert status(*bad) == mq.ERR_INVALID_ARG
    plan = mq.LatentPlan(cache, 16, [0], [100], [99], pt.shape[1], SCALE)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    with pytest.raises(mq.MixattnError) as e:
        plan.run(q, pt, o, ws[:256])
    assert e.value.status == mq.ERR_WORKSPACE
    for args in ((q[..., :512], pt, o), (q.float(), pt, o), (q, pt.long(), o), (q, pt[:, :2], o), (q, pt, o[..., :500]),
                 (q.cpu(), pt, o), (q, pt, q)):
        with pytest.raises(ValueError):
            plan.run(*args, ws)
    tree = mq.LatentPlan(cache, 16, [3], [100], [99], pt.shape[1], SCALE)
    with pytest.raises(mq.MixattnError) as e:
        tree.run(q, pt, o, mq.alloc_workspace(tree.workspace_bytes))
    assert e.value.status == mq.ERR_INVALID_ARG
    plan.close()
    tree.close()
