"""Latent plans of many rows, whose list goes through the workspace and not with the launch; plans shared by streams
and graphs; caches and keys beyond 2^31 elements."""
import numpy as np
import pytest

import _latent as la

pytestmark = pytest.mark.gpu

DECODE, CHUNK = 0, 1
SCALE = 192 ** -0.5


def _plan(cache, pt, rows, heads):
    import mixed_attention_quantized_gb300 as mq
    return mq.LatentPlan(cache, heads, [r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows], pt.shape[1], SCALE)


def _out(rows, heads):
    import torch
    return torch.full((sum(s - o for _, s, o in rows), heads, 512), float("nan"), dtype=torch.float16, device="cuda")


def _compare(cache, slots, rows, q, got):
    at = 0
    for r, (kind, s, o) in enumerate(rows):
        k = cache.data.view(-1, 576)[slots[r]][:, None]
        want, bound = la.attention64(q[at:at + s - o], k, k[..., :512], la.seen(kind, s, o), SCALE)
        la.check(got[at:at + s - o], want, bound, (r, kind, s, o))
        at += s - o


def _many(n, seed, top=200):
    rng = np.random.default_rng(seed)
    rows = []
    for i in range(n):
        s = int(rng.integers(1, top))
        rows.append((CHUNK, s, max(0, s - 3)) if i % 50 == 7 else (DECODE, s, s - 1))
    return rows


@pytest.mark.parametrize("n,heads", [(390, 16), (500, 16), (700, 2), (420, 128)])
def test_many_rows(n, heads):
    import mixed_attention_quantized_gb300 as mq
    rows = _many(n, n + heads)
    cache, pt, slots = la.paged([r[1] for r in rows], 301)
    q, out = la.queries(sum(s - o for _, s, o in rows), heads, 576, 302), _out(rows, heads)
    plan = _plan(cache, pt, rows, heads)
    ws = mq.alloc_workspace(plan.workspace_bytes)
    ws.fill_(0xFF)
    plan.run(q, pt, out, ws)
    assert mq.device_error(clear=True) == 0
    _compare(cache, slots, rows, q, out)
    plan.close()


def test_an_update_behind_a_run_that_has_not_begun():
    """The second list takes the first one's place only when the first run has it; and back to a short list."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    lists = [_many(500, 311), _many(650, 312, 120), _many(3, 313)]
    seqs = [max(r[i][1] for r in lists if i < len(r)) for i in range(650)]
    cache, pt, slots = la.paged(seqs, 314)
    plan = _plan(cache, pt[:500], lists[0], 16)
    side, todo = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    for i, rows in enumerate(lists):
        if i:
            plan.update([r[0] for r in rows], [r[1] for r in rows], [r[2] for r in rows], pt.shape[1])
        q, out = la.queries(sum(s - o for _, s, o in rows), 16, 576, 315 + i), _out(rows, 16)
        ws, table = mq.alloc_workspace(plan.workspace_bytes), pt[:len(rows)].contiguous()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(30_000_000)  # some 15 ms
        plan.run(q, table, out, ws, stream=side)
        todo.append((rows, q, out, ws, table))
    torch.cuda.synchronize()
    assert mq.device_error(clear=True) == 0
    for rows, q, out, _, _ in todo:
        _compare(cache, [x[:r[1]] for x, r in zip(slots, rows)], rows, q, out)
    plan.close()


@pytest.mark.parametrize("n", [4, 500])
def test_one_plan_on_two_streams_and_in_two_graphs(n):
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = _many(n, 321, 900)
    cache, pt, slots = la.paged([r[1] for r in rows], 322)
    q = [la.queries(sum(s - o for _, s, o in rows), 16, 576, 323 + i) for i in range(2)]
    plan = _plan(cache, pt, rows, 16)
    ws = [mq.alloc_workspace(plan.workspace_bytes) for _ in range(2)]
    want = [_out(rows, 16) for _ in range(2)]
    for i in range(2):
        plan.run(q[i], pt, want[i], ws[0])  # (one after the other over one workspace)
    _compare(cache, slots, rows, q[0], want[0])
    streams, out = [torch.cuda.Stream() for _ in range(2)], [_out(rows, 16) for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for i in range(2):
            plan.run(q[i], pt, out[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            plan.run(q[i], pt, out[i], ws[0])
    for i in (0, 1, 1, 0, 1):
        out[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[i], want[i])
    assert mq.device_error(clear=True) == 0
    for g in graphs:
        g.reset()
    plan.close()


def test_a_cache_of_more_than_2_to_the_32_elements():
    """Append, export and both row kinds in the last pages of 9 GB."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    pages, rows, heads = 245000, [(DECODE, 700, 699), (CHUNK, 90, 85)], 16
    cache = mq.LatentCache.allocate(pages, fill=None)
    need = [22, 3]
    pt = torch.zeros(2, 22, dtype=torch.int32)
    pt[0], pt[1, :3] = pages - 25 + torch.arange(22), pages - 3 + torch.arange(3)
    assert int(pt[0, 0]) * 32 * 576 > 2 ** 32
    pt = pt.cuda()
    pos = torch.cat([torch.arange(s) for _, s, _ in rows]).cuda()
    row = torch.cat([torch.full((s,), i) for i, (_, s, _) in enumerate(rows)]).cuda()
    slots = (pt[row, pos // 32] * 32 + pos % 32).int()
    x = la.queries(790, 1, 576, 331, 1.0)[:, 0]
    mq.latent_append(cache, mq.Rope(64), None, x[:, :512], x[:, 512:], pos.int(), slots)
    kept = mq.latent_export(cache, slots)
    assert torch.equal(kept[:, :512], x[:, :512]) and torch.equal(kept, cache.data.view(-1, 576)[slots.long()])
    q, out = la.queries(6, heads, 576, 332), _out(rows, heads)
    plan = _plan(cache, pt, rows, heads)
    plan.run(q, pt, out, mq.alloc_workspace(plan.workspace_bytes))
    assert mq.device_error(clear=True) == 0
    _compare(cache, [slots[:700].long(), slots[700:].long()], rows, q, out)
    plan.close()


def test_expanded_keys_of_more_than_2_to_the_31_elements():
    import torch
    import mixed_attention_quantized_gb300 as mq
    s, o, heads = 70000, 69990, 128
    g = torch.Generator("cuda").manual_seed(341)
    kv = torch.empty(s, heads, 256, dtype=torch.float16, device="cuda").normal_(generator=g)
    assert kv.numel() > 2 ** 31
    q, kr = la.queries(s - o, heads, 192, 342, 1.0), la.queries(s, 1, 64, 343, 1.0)[:, 0]
    out = torch.empty(s - o, heads, 128, dtype=torch.float16, device="cuda")
    plan = mq.ExpandedPlan(heads, [s], [o], SCALE)
    plan.run(q, kv[..., :128], kr, kv[..., 128:], out, mq.alloc_workspace(plan.workspace_bytes))
    assert mq.device_error(clear=True) == 0
    for h in (0, 77, 127):
        key = torch.cat([kv[:, h:h + 1, :128], kr[:, None]], -1)
        want, bound = la.attention64(q[:, h:h + 1], key, kv[:, h:h + 1, 128:], la.seen(CHUNK, s, o), SCALE)
        la.check(out[:, h:h + 1], want, bound, h)
    plan.close()
