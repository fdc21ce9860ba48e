"""One plan run on several streams and updated while some of those runs have not begun: each has the list it was called
with."""
import numpy as np
import pytest

import _latent as la

pytestmark = pytest.mark.gpu

SLEEP = 30_000_000  # cycles, some 15 ms


def _paged(rows):
    import torch
    import mixed_attention_quantized_gb300 as mq
    pages = sum(-(-s // 32) for s in rows)
    cache = mq.KVCache.allocate(pages, 2, 128, mq.Q8_0, mq.Q8_0)
    n = pages * 32
    g = torch.Generator("cuda").manual_seed(401)
    k, v = (torch.randn(n, 2, 128, device="cuda", generator=g).half() for _ in range(2))
    mq.kv_append_quant(cache, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
    pt, at = np.zeros((len(rows), max(-(-s // 32) for s in rows)), dtype=np.int32), 0
    for i, s in enumerate(rows):
        pt[i, :-(-s // 32)] = at + np.arange(-(-s // 32))
        at += -(-s // 32)
    pt = torch.from_numpy(pt).cuda()

    def batch(seqs, seed):
        off = [s - 1 if i % 3 else max(0, s - 40) for i, s in enumerate(seqs)]
        kinds = [0 if i % 3 else 1 for i in range(len(seqs))]
        table = pt[:len(seqs)].contiguous()
        q = torch.randn(sum(s - o for s, o in zip(seqs, off)), 8, 128, device="cuda",
                        generator=torch.Generator("cuda").manual_seed(seed)).half()
        return (kinds, seqs, off, pt.shape[1]), (q, table), q.shape

    return batch, lambda args: mq.Plan(cache, 8, *args), (lambda plan, x, out, ws, s: plan.run(*x, out, ws, stream=s))


def _latent(rows):
    import mixed_attention_quantized_gb300 as mq
    cache, pt, _ = la.paged(rows, 402)

    def batch(seqs, seed):
        q = la.queries(len(seqs), 16, 576, seed)
        return ([0] * len(seqs), seqs, [s - 1 for s in seqs], pt.shape[1]), (q, pt[:len(seqs)].contiguous()), (len(seqs), 16, 512)

    return (batch, lambda args: mq.LatentPlan(cache, 16, *args, 0.07),
            lambda plan, x, out, ws, s: plan.run(*x, out, ws, stream=s))


def _expanded(rows):
    import mixed_attention_quantized_gb300 as mq

    def batch(seqs, seed):
        n = sum(seqs)
        kv = la.queries(n, 16, 256, seed, 1.0)
        x = (la.queries(n, 16, 192, seed + 1, 1.0), kv[..., :128], la.queries(n, 1, 64, seed + 2, 1.0)[:, 0], kv[..., 128:])
        return (seqs, [0] * len(seqs)), x, (n, 16, 128)

    return batch, lambda args: mq.ExpandedPlan(16, *args, 0.07), (lambda plan, x, out, ws, s: plan.run(*x, out, ws, stream=s))


@pytest.mark.parametrize("make,rows", [(_paged, 60), (_latent, 600), (_expanded, 50)])
@pytest.mark.parametrize("streams", [2, 11])
def test_an_update_waits_for_every_streams_copy(make, rows, streams):
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(403)
    first, second = ([int(x) for x in rng.integers(1, 300, n)] for n in (rows, rows - 5))
    batch, plan_of, call = make([max(a, b) for a, b in zip(first, second + [1] * 5)])
    jobs = [batch(first, 410 + 5 * i) for i in range(streams)] + [batch(second, 409)]

    def fresh(job, ws_bytes):
        return torch.full(job[2], float("nan"), dtype=torch.float16, device="cuda"), mq.alloc_workspace(ws_bytes)

    want = []
    for job in jobs:
        plan = plan_of(job[0])
        out, ws = fresh(job, plan.workspace_bytes)
        call(plan, job[1], out, ws, None)
        torch.cuda.synchronize()
        want.append(out)
        plan.close()
    plan = plan_of(jobs[0][0])
    bufs = [fresh(job, plan.workspace_bytes) for job in jobs[:-1]]
    side = [torch.cuda.Stream() for _ in range(streams)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side[0]):
        torch.cuda._sleep(SLEEP)  # the first run begins after all the others
    for job, (out, ws), s in zip(jobs, bufs, side):
        call(plan, job[1], out, ws, s)
    plan.update(*jobs[-1][0])
    last = fresh(jobs[-1], plan.workspace_bytes)
    call(plan, jobs[-1][1], *last, None)
    torch.cuda.synchronize()
    assert mq.device_error(clear=True) == 0
    for got, w in zip([b[0] for b in bufs] + [last[0]], want):
        assert torch.equal(got, w)
    plan.close()


def test_a_plan_closed_behind_runs_that_have_not_begun():
    import torch
    import mixed_attention_quantized_gb300 as mq
    rows = [int(x) for x in np.random.default_rng(404).integers(1, 300, 600)]
    batch, plan_of, call = _latent(rows)
    job = batch(rows, 420)
    plan, outs, side = plan_of(job[0]), [], [torch.cuda.Stream() for _ in range(2)]
    bufs = [(torch.zeros(job[2], dtype=torch.float16, device="cuda"), mq.alloc_workspace(plan.workspace_bytes)) for _ in side]
    torch.cuda.synchronize()
    with torch.cuda.stream(side[0]):
        torch.cuda._sleep(SLEEP)
    for (out, ws), s in zip(bufs, side):
        call(plan, job[1], out, ws, s)
    plan.close()
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][0], bufs[1][0]) and mq.device_error(clear=True) == 0
