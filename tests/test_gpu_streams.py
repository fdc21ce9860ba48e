"""Calls given a stream other than the current one: what they allocate belongs to that stream (the
allocator hands a freed block out again in the order of its own stream only), and they compute what
they compute on the current stream."""
import numpy as np
import pytest

import _page8 as ref
import test_gpu_page8 as base

pytestmark = pytest.mark.gpu


def _stream_of(t):
    """The stream in whose order the allocator reuses the tensor's memory."""
    import torch
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


def _case(fmt, hq=8, hkv=2, d=128):
    import torch
    rows, kinds = [(300, 299), (400, 200), (70, 66)], [0, 1, 1]
    cache, pt, row_slots = base._filled(fmt, rows, hkv, d, 401)
    q = np.random.default_rng(402).standard_normal((205, hq, d)).astype(np.float16)
    return cache, torch.from_numpy(pt).cuda(), rows, kinds, torch.from_numpy(q).cuda(), row_slots


@pytest.mark.parametrize("fmt", [1, ref.I8, ref.E4M3])
def test_outputs_belong_to_the_given_stream(fmt, monkeypatch):
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache, pt, rows, kinds, q, row_slots = _case(fmt)
    seqs, offs = [r[0] for r in rows], [r[1] for r in rows]
    rope = mq.Rope(128)
    n = q.shape[0]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    skip = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots = torch.from_numpy(np.asarray(row_slots[0][:50], dtype=np.int32)).cuda()
    k = q[:, :2].contiguous()
    made = []
    alloc = mq.alloc_workspace
    monkeypatch.setattr(mq, "alloc_workspace", lambda *a, **kw: made.append(alloc(*a, **kw)) or made[-1])
    calls = [lambda s: mq.rope_apply(rope, q, pos, stream=s),
             lambda s: mq.rope_append(cache, rope, q, k, k, pos, skip, stream=s),
             lambda s: mq.kv_export_blocks(cache, 1, slots, stream=s),
             lambda s: mq.mixed_attention(cache, q, pt, seqs, offs, kinds, stream=s)]
    if fmt == 1:
        calls.append(lambda s: mq.mixed_attention_noalloc(cache, q, pt, seqs, offs, kinds, stream=s))
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    for call in calls:
        made.clear()
        want = call(None)
        assert _stream_of(want) == here.cuda_stream
        torch.cuda.synchronize()
        side.wait_stream(here)
        got = call(side)
        for t in [got] + made[1:]:
            assert _stream_of(t) == side.cuda_stream
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert torch.cuda.current_stream() == here
    assert mq.device_error(clear=True) == 0


@pytest.mark.parametrize("fmt", [1, ref.I8])
def test_a_step_on_a_side_stream(fmt):
    """Append, rotate and attend on one side stream, with outputs of the caller's and without."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache, pt, rows, kinds, q, row_slots = _case(fmt)
    rope = mq.Rope(64)
    n = q.shape[0]
    pos = torch.cat([torch.arange(o, s) for s, o in rows]).to(torch.int32).cuda()
    slots = torch.from_numpy(np.concatenate([np.asarray(r)[o:s] for r, (s, o) in zip(row_slots, rows)]).astype(np.int32)).cuda()
    k, v = torch.randn(2, n, 2, 128, device="cuda").half()
    plan = mq.Plan(cache, 8, kinds, [r[0] for r in rows], [r[1] for r in rows], pt.shape[1])
    start = [t.clone() for t in (cache.k_quant, cache.k_scale, cache.v_quant, cache.v_scale)]

    def step(stream, q_out):
        for t, x in zip((cache.k_quant, cache.k_scale, cache.v_quant, cache.v_scale), start):
            t.copy_(x)
        ws, o = mq.alloc_workspace(plan.workspace_bytes), torch.zeros_like(q)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        qr = mq.rope_append(cache, rope, q, k, v, pos, slots, q_out, stream=stream)
        plan.run(qr, pt, o, ws, stream=stream)
        torch.cuda.synchronize()
        return qr, o

    want = step(None, None)
    side = torch.cuda.Stream()
    for q_out in (None, torch.empty_like(q)):
        for a, b in zip(step(side, q_out), want):
            assert torch.equal(a, b)
    plan.close()
    assert mq.device_error(clear=True) == 0


@pytest.mark.parametrize("fmt", [1, ref.I8])
@pytest.mark.parametrize("mode", ["relaxed", "thread_local"])
def test_the_one_call_entry_point_is_not_captured(fmt, mode):
    """It frees the plan whose tile list a replay would read: refused on a capturing stream, which goes
    on capturing what it may."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache, pt, rows, kinds, q, _ = _case(fmt)
    seqs, offs = [r[0] for r in rows], [r[1] for r in rows]
    ws = mq.alloc_workspace(mq.workspace_bytes(cache, 8, kinds, seqs, offs, pt.shape[1]))
    want = mq.mixed_attention(cache, q, pt, seqs, offs, kinds, workspace=ws)
    o, rope = torch.zeros_like(q), mq.Rope(128)
    pos = torch.arange(q.shape[0], dtype=torch.int32, device="cuda")
    turned, kept = mq.rope_apply(rope, q, pos), torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode=mode):
        with pytest.raises(mq.MixattnError) as e:
            mq.mixed_attention(cache, q, pt, seqs, offs, kinds, o=o, workspace=ws)
        mq.rope_apply(rope, q, pos, kept)
    assert e.value.status == mq.ERR_UNSUPPORTED
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, turned) and not o.any()
    assert torch.equal(mq.mixed_attention(cache, q, pt, seqs, offs, kinds, workspace=ws), want)
