"""Expanded latent attention on the GPU against 64 bits, within the bound of `_latent.attention64`, and a
model's path through both forms."""
import numpy as np
import pytest

import _latent as la

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _inputs(rows, heads, seed, size=1.0):
    import torch
    nk, nq = sum(s for s, _ in rows), sum(s - o for s, o in rows)
    kv = la.queries(nk, heads, 256, seed, 1.0)
    return la.queries(nq, heads, 192, seed + 1, size), kv[..., :128], la.queries(nk, 1, 64, seed + 2, 1.0)[:, 0], kv[..., 128:]


def _run(rows, heads, q, k, kr, v, scale=SCALE, plan=None, stream=None):
    import torch
    import mixed_attention_quantized_gb300 as mq
    plan = plan or mq.ExpandedPlan(heads, [r[0] for r in rows], [r[1] for r in rows], scale)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    ws.fill_(0xFF)
    out = torch.full((q.shape[0], heads, 128), float("nan"), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    plan.run(q, k, kr, v, out, ws, stream=stream)
    torch.cuda.synchronize()
    assert mq.device_error(clear=True) == 0
    return out


def _compare(rows, got, q, k, kr, v, scale=SCALE):
    import torch
    at = first = 0
    for r, (s, o) in enumerate(rows):
        key = torch.cat([k[first:first + s], kr[first:first + s, None].expand(-1, k.shape[1], -1)], -1)
        for a in range(0, s - o, 256):
            b = min(s - o, a + 256)
            vis = la.seen(1, s, o)[a:b]
            want, bound = la.attention64(q[at + a:at + b], key, v[first:first + s], vis, scale)
            la.check(got[at + a:at + b], want, bound, (r, s, o, a))
        at += s - o
        first += s


@pytest.mark.parametrize("heads", [1, 2, 5])
@pytest.mark.parametrize("rows", [[(1, 0)], [(127, 0), (128, 0), (129, 0)], [(256, 0), (257, 0), (2, 0), (300, 299)],
                                  [(700, 0)], [(1000, 200), (40, 39), (513, 256)], [(2600, 2500)], [(1300, 7), (64, 0)]])
def test_prompts_and_chunks(heads, rows):
    x = _inputs(rows, heads, 10 * heads + len(rows))
    _compare(rows, _run(rows, heads, *x), *x)


def test_many_tiles_a_cta():
    rows = [(300, 0)] * 9 + [(900, 100), (17, 0)]
    x = _inputs(rows, 32, 5)
    _compare(rows, _run(rows, 32, *x), *x)


def test_rows_of_many_kv_tiles_after_one_another():
    """Several tiles a CTA, the ends of their rows more than two KV tiles apart."""
    rows = [(700, 0), (1000, 0), (900, 500), (450, 0), (1100, 1000)]
    x = _inputs(rows, 32, 15)
    _compare(rows, _run(rows, 32, *x), *x)


def test_long_rows_are_cut_and_joined():
    rows = [(6000, 5700)]
    x = _inputs(rows, 2, 6)
    _compare(rows, _run(rows, 2, *x), *x)


def test_scores_that_move_the_reference():
    rows = [(900, 0), (1500, 1400)]
    x = _inputs(rows, 2, 7, 6.0)
    _compare(rows, _run(rows, 2, *x), *x)


def test_what_lies_behind_a_row_does_not_matter():
    """The next row's keys and values are infinite or NaN: this row's outputs keep their bits."""
    import torch
    rows = [(200, 0), (130, 0), (77, 70)]
    q, k, kr, v = _inputs(rows, 3, 8)
    k, v = k.clone(), v.clone()
    want = _run(rows, 3, q, k, kr, v)
    for bad in (float("nan"), float("inf")):
        for x in (k, v, kr):
            x[200:330] = bad
        got = _run(rows, 3, q, k, kr, v)
        assert torch.equal(got[:200], want[:200]) and torch.equal(got[330:], want[330:])


def test_strides():
    import torch
    rows = [(150, 20), (70, 0)]
    q, k, kr, v = _inputs(rows, 4, 9)
    want = _run(rows, 4, q, k, kr, v)
    wide = torch.zeros(220, 600, dtype=torch.float16, device="cuda")
    wide[:, 512:576] = kr
    outer = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # heads outermost
    assert torch.equal(want, _run(rows, 4, outer(q), outer(k), wide[:, 512:576], v.contiguous()))


def test_streams_graphs_and_updates():
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [(400, 100), (90, 0)]
    x = _inputs(rows, 6, 11)
    want = _run(rows, 6, *x)
    plan = mq.ExpandedPlan(6, [5], [0], SCALE)
    plan.update([400, 90], [100, 0])
    assert torch.equal(want, _run(rows, 6, *x, plan=plan, stream=torch.cuda.Stream()))
    ws, out = mq.alloc_workspace(plan.workspace_bytes), torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(*x, out, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, out)
    with pytest.raises(mq.MixattnError):
        plan.update([5], [0])
    graph.reset()
    plan.close()


def test_refusals():
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [(40, 0)]
    q, k, kr, v = _inputs(rows, 2, 12)
    o = torch.empty(40, 2, 128, dtype=torch.float16, device="cuda")
    for bad in ((0, [40], [0], SCALE), (2, [40], [40], SCALE), (2, [40], [-1], SCALE), (2, [], [], SCALE),
                (2, [40], [0], 0.0), (2, [40], [0], float("inf"))):
        with pytest.raises(mq.MixattnError) as e:
            mq.ExpandedPlan(*bad)
        assert e.value.status == mq.ERR_INVALID_ARG
    plan = mq.ExpandedPlan(2, [40], [0], SCALE)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    with pytest.raises(mq.MixattnError) as e:
        plan.run(q, k, kr, v, o, ws[:100])
    assert e.value.status == mq.ERR_WORKSPACE
    for args in ((q[..., :128], k, kr, v, o), (q, k[:39], kr, v, o), (q, k, kr[:, :32], v, o), (q, k, kr, v.float(), o),
                 (q, k, kr, v, o[:, :1]), (q, k.cpu(), kr, v, o)):
        with pytest.raises(ValueError):
            plan.run(*args, ws)
    with pytest.raises(mq.MixattnError) as e:
        plan.run(q, k[:1].expand(40, 2, 128), kr, v, o, ws)  # tokens on top of one another
    assert e.value.status == mq.ERR_INVALID_ARG
    plan.close()


def test_a_model_prefills_decodes_and_verifies():
    """Prompts through the expanded form, the same tokens again through the absorbed one over the cache that
    the append filled, then a tree of drafted tokens: one model, two forms, the same attention."""
    import torch
    import _trees as tr
    import mixed_attention_quantized_gb300 as mq
    heads, prompts, draft = 16, [150, 33], 5
    g = torch.Generator("cuda").manual_seed(13)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
    w_k, w_v = (rnd(heads, 512, 128) / 512 ** 0.5 for _ in range(2))
    rope = mq.Rope(64, layout=mq.ROPE_INTERLEAVED)
    total = [p + draft for p in prompts]
    cache = mq.LatentCache.allocate(sum(-(-t // 32) for t in total) + 1, fill=0xFF)
    pt = torch.full((2, 5), -1, dtype=torch.int32)
    pt[0, :5], pt[1, :2] = torch.tensor([3, 0, 6, 1, 7]), torch.tensor([5, 2])
    pt = pt.cuda()

    def step(tokens, latents, q_nope, q_pe, k_pe, positions, row_of):
        """Appends; returns the absorbed queries."""
        slots = pt[row_of, positions // 32] * 32 + positions % 32
        q = torch.empty(tokens, heads, 576, dtype=torch.float16, device="cuda")
        q[..., :512] = torch.einsum("thd,hcd->thc", q_nope.float(), w_k).half()
        mq.latent_append(cache, rope, q_pe, latents, k_pe, positions.int(), slots.int(), q[..., 512:])
        return q

    n = sum(prompts)
    c, qn, qp, kp = rnd(n, 512).half(), rnd(n, heads, 128).half(), rnd(n, heads, 64).half(), rnd(n, 64).half()
    pos = torch.cat([torch.arange(p) for p in prompts]).cuda()
    row = torch.cat([torch.full((p,), i) for i, p in enumerate(prompts)]).cuda()
    q_abs = step(n, c, qn, qp, kp, pos, row)

    # expanded: keys and values made of what the cache holds
    rows_c = mq.latent_export(cache, (pt[row, pos // 32] * 32 + pos % 32).int())
    k = torch.einsum("tc,hcd->thd", rows_c[:, :512].float(), w_k).half()
    v = torch.einsum("tc,hcd->thd", rows_c[:, :512].float(), w_v).half()
    ep = mq.ExpandedPlan(heads, prompts, [0, 0], SCALE)
    o_exp = torch.empty(n, heads, 128, dtype=torch.float16, device="cuda")
    ep.run(torch.cat([qn, q_abs[..., 512:]], -1), k, rows_c[:, 512:], v, o_exp, mq.alloc_workspace(ep.workspace_bytes))
    ap = mq.LatentPlan(cache, heads, [mq.ROW_CHUNK] * 2, prompts, [0, 0], 5, SCALE)
    o_lat = torch.empty(n, heads, 512, dtype=torch.float16, device="cuda")
    ap.run(q_abs, pt, o_lat, mq.alloc_workspace(ap.workspace_bytes))
    o_abs = torch.einsum("thc,hcd->thd", o_lat.float(), w_v)
    # each path's keys or queries and values are rounded to fp16 at other places: 2^-11 of scores of up to ~6 in
    # the exponent, and of the values
    assert float((o_exp.float() - o_abs).abs().max()) <= 2.0 ** -11 * (6 + 4) * float(v.abs().max())

    # drafted trees behind the prompts
    rng = np.random.default_rng(14)
    masks = [tr.random_tree(draft, rng) for _ in prompts]
    m = 2 * draft
    c2, qn2, qp2, kp2 = rnd(m, 512).half(), rnd(m, heads, 128).half(), rnd(m, heads, 64).half(), rnd(m, 64).half()
    row2 = torch.arange(2).repeat_interleave(draft).cuda()
    at = torch.cat([p + torch.arange(draft) for p in prompts]).cuda()  # slots behind the context
    q2 = step(m, c2, qn2, qp2, kp2, at, row2)
    tp = mq.LatentPlan(cache, heads, [mq.ROW_TREE] * 2, total, prompts, 5, SCALE)
    o2 = torch.empty(m, heads, 512, dtype=torch.float16, device="cuda")
    tp.run(q2, pt, o2, mq.alloc_workspace(tp.workspace_bytes), tree_mask=torch.from_numpy(tr.pack(masks)).cuda())
    assert mq.device_error(clear=True) == 0
    for r in range(2):
        t = torch.arange(total[r], device="cuda")
        keys = mq.latent_export(cache, (pt[r, t // 32] * 32 + t % 32).int())[:, None]
        part = slice(r * draft, (r + 1) * draft)
        want, bound = la.attention64(q2[part], keys, keys[..., :512], la.seen(3, total[r], prompts[r], masks[r]), SCALE)
        la.check(o2[part], want, bound, r)
