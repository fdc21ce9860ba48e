"""Rotary positions on the GPU against fp64: alone, and on the way into every cache format.

An fp16 output is off by its own rounding (2^-11 of the value, 2^-25 among the smallest
numbers) and by the fp32 cosines and products: those are within 2^-22, the angle they
are taken of within 2^-24 radians, each product and sum within 2^-24, so
under 2^-20 of m (|a| + |b|) for a pair (a, b)."""
import numpy as np
import pytest

import _page8 as ref
import oracle

pytestmark = pytest.mark.gpu

SCALINGS = {"none": {}, "linear": dict(factor=4.0),
            "ramp": dict(factor=8.0, original_ctx=4096, low=1.0, high=32.0),
            "bands": dict(factor=8.0, original_ctx=8192, low=1.0, high=4.0)}


def _rope(rot, interleaved, scaling, base=10000.0):
    import mixed_attention_quantized_gb300 as mq
    kind = {"none": 0, "linear": 1, "ramp": 2, "bands": 3}[scaling]
    kw = SCALINGS[scaling]
    r = mq.Rope(rot, layout=int(interleaved), base=base, scaling=kind, **kw)
    f, m = ref.frequencies(rot, scaling, base, kw.get("factor", 1.0), kw.get("original_ctx", 0), kw.get("low", 0.0),
                           kw.get("high", 0.0))
    return r, f, m


def _size(x, rot, interleaved, m):
    """m (|a| + |b|) of each element's pair; 0 past rot."""
    s = np.zeros(x.shape)
    a = np.abs(x.astype(np.float64))
    if interleaved:
        t = a[..., 0:rot:2] + a[..., 1:rot:2]
        s[..., 0:rot:2] = s[..., 1:rot:2] = t
    else:
        t = a[..., :rot // 2] + a[..., rot // 2:rot]
        s[..., :rot // 2] = s[..., rot // 2:rot] = t
    return s * m


def _half_tolerance(want, size):
    return 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -20 * size


def _positions(n, rng):
    p = rng.integers(0, 1 << 20, size=n)
    special = [0, 1, 262143, 2 ** 31 - 1, 31, 32, -1, -(2 ** 31)]
    p[:min(n, len(special))] = special[:min(n, len(special))]
    return p.astype(np.int32)


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 16), (128, 96), (64, 64), (64, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,scaling", [(1, 1, "none"), (7, 5, "ramp"), (70, 32, "bands"), (33, 67, "linear")])
def test_rope_apply(d, rot, interleaved, n, heads, scaling):
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(n * 1000 + rot)
    x = (rng.standard_normal((n, heads, d)) * 3).astype(np.float16)
    pos = _positions(n, rng)
    r, f, m = _rope(rot, interleaved, scaling)
    want = ref.rotate(x, pos, f, m, rot, interleaved)
    xd, pd = torch.from_numpy(x).cuda(), torch.from_numpy(pos).cuda()
    out = torch.full((n, heads, d), float("nan"), dtype=torch.float16, device="cuda")
    mq.rope_apply(r, xd, pd, out)
    got = out.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= _half_tolerance(want, _size(x, rot, interleaved, m))).all()
    # elements past rot are copied, in place gives the same, the input stays
    np.testing.assert_array_equal(got[..., rot:], x[..., rot:].astype(np.float64))
    np.testing.assert_array_equal(xd.cpu().numpy(), x)
    mq.rope_apply(r, xd, pd, xd)
    assert torch.equal(xd, out)


def test_rope_apply_on_slices_of_one_projection():
    """Queries and keys as strided slices, in place; what lies between stays as it was."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(5)
    n, hq, hkv, d = 37, 4, 2, 128
    qkv = rng.standard_normal((n, (hq + 2 * hkv) * d)).astype(np.float16)
    pos = _positions(n, rng)
    r, f, m = _rope(d, False, "none")
    buf = torch.from_numpy(qkv).cuda()
    q = buf[:, :hq * d].view(n, hq, d)
    k = buf[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    pd = torch.from_numpy(pos).cuda()
    assert mq.rope_apply(r, q, pd, q).data_ptr() == buf.data_ptr()
    mq.rope_apply(r, k, pd, k)
    got = buf.cpu().numpy()
    x = qkv[:, :(hq + hkv) * d].reshape(n, hq + hkv, d)
    want = ref.rotate(x, pos, f, m, d, False)
    err = np.abs(got[:, :(hq + hkv) * d].reshape(x.shape).astype(np.float64) - want)
    assert (err <= _half_tolerance(want, _size(x, d, False, m))).all()
    np.testing.assert_array_equal(got[:, (hq + hkv) * d:], qkv[:, (hq + hkv) * d:])


def test_far_positions_keep_their_angle():
    """Relative rotation: R(p) x . R(p + 7) y depends on the 7 alone, at any p."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(9)
    x, y = rng.standard_normal((2, 1, 1, 128)).astype(np.float16)
    r, _, _ = _rope(128, False, "none")
    starts = np.array([0, 1000, 262144, 10_000_000, 2_000_000_000], dtype=np.int64)
    n = len(starts)

    def turned(v, p):
        t = torch.from_numpy(np.repeat(v, n, axis=0)).cuda()
        return mq.rope_apply(r, t, torch.from_numpy(p.astype(np.int32)).cuda()).cpu().numpy().astype(np.float64)

    dots = (turned(x, starts) * turned(y, starts + 7)).sum(axis=(1, 2))
    # two roundings to fp16 a product: 2^-10 of |x||y|, over 128 of them
    assert np.ptp(dots) <= 2 * 2.0 ** -10 * (np.abs(x.astype(np.float64)) + 0.1).sum() * 4


def test_saturates_and_no_tokens():
    import torch
    import mixed_attention_quantized_gb300 as mq
    r, _, _ = _rope(64, False, "none")
    x = torch.full((2, 1, 64), 65504.0, dtype=torch.float16, device="cuda")
    out = mq.rope_apply(r, x, torch.tensor([1, 3], dtype=torch.int32, device="cuda"))
    assert torch.isfinite(out).all()
    e = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    mq.rope_apply(r, e, torch.empty(0, dtype=torch.int32, device="cuda"), e)


FORMATS = [(0, 0), (1, 1), (2, 2), (1, 2), (2, 1), (3, 3), (4, 4)]


def _canonical(cache, which, slots):
    """Values [n, heads, d] of cache slots, and their steps, from the exported blocks."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    fmt = cache.k_fmt if which == 0 else cache.v_fmt
    blk = mq.kv_export_blocks(cache, which, torch.from_numpy(slots).cuda()).cpu().numpy()
    n, h = blk.shape[:2]
    if fmt in (ref.I8, ref.E4M3):
        d = blk[..., :4].copy().view(np.float32).astype(np.float64)
        v = ref.raw_codes(fmt, np.ascontiguousarray(blk[..., 4:]))
        return (v * d).reshape(n, h, -1), np.broadcast_to(d, v.shape).reshape(n, h, -1)
    v = oracle.dequantize(fmt, blk).astype(np.float64).reshape(n, h, -1)
    if fmt == 0:
        return v, np.zeros(v.shape)
    d = np.abs(blk[..., :2].copy().view(np.float16).astype(np.float64))
    return v, np.broadcast_to(d, d.shape[:-1] + (32,)).reshape(n, h, -1)


@pytest.mark.parametrize("fmts", FORMATS)
@pytest.mark.parametrize("d,rot,interleaved,scaling", [(128, 128, False, "none"), (64, 32, True, "ramp"),
                                                       (128, 96, False, "bands"), (128, 64, True, "none")])
@pytest.mark.parametrize("n,hq,hkv", [(1, 4, 1), (75, 6, 3)])
def test_rope_append(fmts, d, rot, interleaved, scaling, n, hq, hkv):
    import torch
    import mixed_attention_quantized_gb300 as mq
    rng = np.random.default_rng(n + rot)
    buf = rng.standard_normal((n, (hq + 2 * hkv) * d)).astype(np.float16)
    pos = _positions(n, rng)
    pages = 6
    slots = (rng.permutation(pages)[:-(-n // 32)].repeat(32)[:n] * 32 + np.arange(n) % 32).astype(np.int32)
    if n > 1:
        slots[[3, 40]] = -1  # padding: query rotated, key dropped
    r, f, m = _rope(rot, interleaved, scaling)
    cache = mq.KVCache.allocate(pages, hkv, d, fmts[0], fmts[1], fill=0xFF)
    bd = torch.from_numpy(buf).cuda()
    q, k, v = (bd[:, a * d:b * d].view(n, b - a, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
    out = mq.rope_append(cache, r, q, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda())
    assert mq.device_error(clear=True) == 0
    x = buf[:, :hq * d].reshape(n, hq, d)
    want = ref.rotate(x, pos, f, m, rot, interleaved)
    got = out.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= _half_tolerance(want, _size(x, rot, interleaved, m))).all()

    keep = slots >= 0
    xk = buf[:, hq * d:(hq + hkv) * d].reshape(n, hkv, d)[keep]
    xv = buf[:, (hq + hkv) * d:].reshape(n, hkv, d)[keep]
    for which, fmt, want, slack in ((0, fmts[0], ref.rotate(xk, pos[keep], f, m, rot, interleaved),
                                     2.0 ** -20 * _size(xk, rot, interleaved, m)),
                                    (1, fmts[1], xv.astype(np.float64), 0.0)):
        got, step = _canonical(cache, which, slots[keep])
        if fmt == 0:
            tol = _half_tolerance(want, 0) if which == 0 else 0.0
        elif fmt == 2:  # a code off the range's short end is a whole step off; the scale is rounded to fp16
            tol = step * (1.0 + 8 * 2.0 ** -11 + 1e-5)
        elif fmt == ref.E4M3:
            tol = np.maximum(2.0 ** -4 * np.abs(want), step * 2.0 ** -10) * (1 + 1e-5)
        else:  # half a step, and for Q8_0 the fp16 rounding of a scale that multiplies up to 127
            tol = step * (0.5 + (127 * 2.0 ** -11 if fmt == 1 else 0) + 1e-4)
        assert (np.abs(got - want) <= tol + slack + 1e-7).all(), (which, np.abs(got - want).max())

    # values go the way of the plain append, bit for bit
    plain = mq.KVCache.allocate(pages, hkv, d, fmts[0], fmts[1], fill=0xFF)
    mq.kv_append_quant(plain, k.contiguous(), v.contiguous(), torch.from_numpy(slots).cuda())
    assert torch.equal(plain.v_quant, cache.v_quant)
    if fmts[1]:
        assert torch.equal(plain.v_scale, cache.v_scale)


@pytest.mark.parametrize("fmt", [1, 3])
def test_rope_append_without_queries_and_bad_slots(fmt):
    import torch
    import mixed_attention_quantized_gb300 as mq
    mq.device_error(clear=True)
    r, f, m = _rope(64, False, "none")
    cache = mq.KVCache.allocate(2, 1, 64, fmt, fmt, fill=0x5A)
    k = torch.ones(3, 1, 64, dtype=torch.float16, device="cuda")
    pos = torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda")
    assert mq.rope_append(cache, r, None, k, k, pos, torch.tensor([64, 3, -7], dtype=torch.int32, device="cuda")) is None
    torch.cuda.synchronize()
    assert mq.device_error(clear=True) == mq.DEVERR_SLOT
    got, step = _canonical(cache, 0, np.array([3], dtype=np.int32))
    want = ref.rotate(np.ones((1, 1, 64)), np.array([1]), f, m, 64, False)
    assert (np.abs(got - want) <= 0.6 * step + 1e-6).all()
    # position 0 is the identity: the plain append's bytes
    a, b = (mq.KVCache.allocate(2, 1, 64, fmt, fmt) for _ in range(2))
    x = torch.randn(32, 1, 64, device="cuda").half()
    s = torch.arange(32, dtype=torch.int32, device="cuda")
    mq.rope_append(a, r, None, x, x, torch.zeros_like(s), s)
    mq.kv_append_quant(b, x, x, s)
    assert torch.equal(a.k_quant, b.k_quant) and torch.equal(a.k_scale, b.k_scale)
