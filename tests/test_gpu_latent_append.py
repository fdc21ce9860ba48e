"""The latent cache's append, with rotary positions, and its export.

A rotated fp16 element is off by its own rounding (2^-11 of the value, 2^-25 among the smallest) and
by the fp32 cosines and products, under 2^-20 of m (|a| + |b|) for a pair (a, b)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _turned(x, pos, rope, interleaved):
    """(rotated fp64, bound) of [n, ..., 64]."""
    info = rope.info()
    f, m = np.array(info["frequencies"]), info["mscale"]
    a = pos.astype(np.float64).reshape(-1, *([1] * (x.ndim - 2)), 1) * f
    c, s = np.cos(a) * m, np.sin(a) * m
    x = x.astype(np.float64)
    u, v = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y0, y1, size = u * c - v * s, v * c + u * s, (np.abs(u) + np.abs(v)) * m
    if interleaved:
        y, size = np.stack([y0, y1], -1).reshape(x.shape), np.repeat(size, 2, axis=-1)
    else:
        y, size = np.concatenate([y0, y1], -1), np.concatenate([size, size], -1)
    return y, 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 2.0 ** -20 * size


def _close(got, want, bound):
    assert (np.abs(got.astype(np.float64) - want) <= bound).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", [0, 2])
@pytest.mark.parametrize("n,heads", [(1, 1), (1, 128), (7, 3), (70, 16), (33, 128), (300, 0), (2501, 8), (2503, 0),
                                     (1300, 33)])
def test_append(interleaved, scaling, n, heads):
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(100 * n + heads)
    rope = mq.Rope(64, layout=int(interleaved), scaling=scaling, factor=8.0, original_ctx=4096, low=1.0, high=32.0)
    cache = mq.LatentCache.allocate(n // 32 + 4, fill=0x3C)
    before = cache.data.clone()
    slots = rng.permutation(cache.num_pages * 32)[:n].astype(np.int32)
    if n > 5:
        slots[[1, 4]] = -1
    pos = rng.integers(0, 300000, n).astype(np.int32)
    c = rng.standard_normal((n, 512)).astype(np.float16)
    proj = rng.standard_normal((n, 576)).astype(np.float16)
    q = rng.standard_normal((n, max(heads, 1), 192)).astype(np.float16)
    t = lambda x: torch.from_numpy(x).cuda()
    qd, buf = t(q), torch.full((n, max(heads, 1), 576), 7.0, dtype=torch.float16, device="cuda")
    out = mq.latent_append(cache, rope, qd[..., 128:] if heads else None, t(c), t(proj)[:, 512:], t(pos), t(slots),
                           buf[..., 512:] if heads else None)
    assert mq.device_error() == 0
    flat, old = cache.data.view(-1, 576).cpu().numpy(), before.view(-1, 576).cpu().numpy()
    kept = slots >= 0
    assert np.array_equal(flat[slots[kept], :512], c[kept])
    y, bound = _turned(proj[:, 512:], pos, rope, interleaved)
    _close(flat[slots[kept], 512:], y[kept], bound[kept])
    rest = np.setdiff1d(np.arange(len(flat)), slots[kept])
    assert np.array_equal(flat[rest].view(np.uint16), old[rest].view(np.uint16))
    if heads:
        y, bound = _turned(q[..., 128:], pos, rope, interleaved)
        _close(buf[..., 512:].cpu().numpy(), y, bound)
        assert bool((buf[..., :512] == 7).all()) and out.data_ptr() == buf[..., 512:].data_ptr()
        again = qd.clone()
        mq.latent_append(cache, rope, again[..., 128:], t(c), t(proj)[:, 512:], t(pos), t(slots), again[..., 128:])
        assert torch.equal(again[..., 128:], buf[..., 512:]) and torch.equal(again[..., :128], qd[..., :128])
        # heads outermost
        tok = qd[..., 128:].transpose(0, 1).contiguous().transpose(0, 1)
        assert torch.equal(mq.latent_append(cache, rope, tok, t(c), t(proj)[:, 512:], t(pos), t(slots)), buf[..., 512:])
    else:
        assert out is None
    got = mq.latent_export(cache, t(slots[kept]))
    assert np.array_equal(got.cpu().numpy().view(np.uint16), flat[slots[kept]].view(np.uint16))


def test_slots_outside_the_cache_are_skipped_and_reported():
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache = mq.LatentCache.allocate(2)
    x = torch.ones(3, 576, dtype=torch.float16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    mq.latent_append(cache, mq.Rope(64), None, x[:, :512], x[:, 512:], pos,
                     torch.tensor([5, 64, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    assert mq.device_error(clear=True) == mq.DEVERR_SLOT
    assert float(cache.data.float().sum()) == 576
    out = mq.latent_export(cache, torch.tensor([5, 64, -1], dtype=torch.int32, device="cuda"))
    assert mq.device_error(clear=True) == mq.DEVERR_SLOT
    assert bool((out[0] == 1).all())


def test_elements_that_are_not_finite_stay():
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache = mq.LatentCache.allocate(1)
    x = torch.zeros(1, 576, dtype=torch.float16, device="cuda")
    x[0, 3], x[0, 4], x[0, 512] = float("inf"), float("nan"), float("nan")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    mq.latent_append(cache, mq.Rope(64), None, x[:, :512], x[:, 512:], i, i)
    row = cache.data[0, 0].float()
    assert row[3] == float("inf") and bool(row[4].isnan()) and bool(row[512].isnan()) and float(row[1]) == 0


def test_refusals():
    import torch
    import mixed_attention_quantized_gb300 as mq
    cache, rope = mq.LatentCache.allocate(4), mq.Rope(64)
    n = 4
    q = torch.zeros(n, 8, 192, dtype=torch.float16, device="cuda")
    x = torch.zeros(n, 576, dtype=torch.float16, device="cuda")
    i = torch.arange(n, dtype=torch.int32, device="cuda")
    good = dict(q_rope=q[..., 128:], c_new=x[:, :512], k_rope=x[:, 512:], positions=i, slot_mapping=i)

    def call(**kw):
        return mq.latent_append(cache, kw.pop("rope", rope), **{**good, **kw})

    call()
    for bad in (dict(q_rope=q[..., :128]), dict(q_rope=q[:3, :, 128:]), dict(c_new=x[:, :500]), dict(k_rope=x[:, 500:]),
                dict(c_new=x[:, :512].float()), dict(positions=i.long()), dict(slot_mapping=i[:3]),
                dict(q_out=q[:, :4, 128:]), dict(c_new=x[:, :512].cpu()), dict(q_rope=q[..., 128:].cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    flat = torch.zeros(n * 8 * 64 + 64, dtype=torch.float16, device="cuda")
    dense = flat[:n * 8 * 64].view(n, 8, 64)
    for bad in (dict(rope=mq.Rope(32)), dict(q_rope=dense, q_out=flat[64:].view(n, 8, 64)),
                dict(q_rope=flat[4:4 + n * 8 * 64].view(n, 8, 64)), dict(q_rope=dense[:1].expand(n, 8, 64))):
        with pytest.raises(mq.MixattnError) as e:
            call(**bad)
        assert e.value.status == mq.ERR_INVALID_ARG
    with pytest.raises(mq.MixattnError):
        mq.LatentCache.allocate(4, latent_dim=256)
