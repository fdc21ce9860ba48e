"""What the fused rotary append makes of infinities, NaN and values past the fp16 range."""
import numpy as np
import pytest

import _page8 as ref
import oracle
from test_gpu_rope import _half_tolerance, _rope, _size

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fk,fv", [(0, 0), (1, 1), (1, 2), (2, 1), (2, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_elements_that_are_not_finite(fk, fv, interleaved):
    """Q8_0 and Q4_0 keys: NaN counts as 0, infinities and rotated values past the fp16 range
    saturate.  fp16 keys keep NaN.  Values go in as the plain append takes them."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    n, hkv, d, rot = 40, 2, 128, 64
    rng = np.random.default_rng(9)
    rope, f, m = _rope(rot, interleaved, "none")
    k, v = rng.standard_normal((2, n, hkv, d)).astype(np.float16)
    pos = np.zeros(n, dtype=np.int32)  # no turn: a pair's two elements stay apart
    pos[30:] = 1
    k[3, 0, 5], k[4, 1, 70], k[5, 0, 100] = np.inf, -np.inf, np.nan  # rotated and copied elements
    k[30, 0, :rot] = 60000  # 60000 (cos 1 + sin 1) is past the range
    v[6, 1, 40], v[7, 0, 3] = np.inf, np.nan
    slots = rng.permutation(64)[:n].astype(np.int32)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    a = mq.KVCache.allocate(2, hkv, d, fk, fv)
    b = mq.KVCache.allocate(2, hkv, d, fk, fv)
    mq.rope_append(a, rope, None, dev(k), dev(v), dev(pos), dev(slots))
    mq.kv_append_quant(b, dev(k), dev(v), dev(slots))
    assert mq.device_error(clear=True) == 0
    s = dev(slots)
    got_v, plain_v = (mq.kv_export_blocks(c, 1, s).cpu().numpy() for c in (a, b))
    np.testing.assert_array_equal(got_v, plain_v)
    got = mq.kv_export_blocks(a, 0, s).cpu().numpy()
    want = ref.rotate(np.nan_to_num(k.astype(np.float64), nan=0.0, posinf=ref.F16_MAX, neginf=-ref.F16_MAX), pos, f, m, rot,
                      interleaved)
    want = np.clip(want, -ref.F16_MAX, ref.F16_MAX)
    partner = 4 if interleaved else 5 + rot // 2
    want[3, 0, 5], want[3, 0, partner] = ref.F16_MAX, 0  # infinity times cos 0; plus infinity times sin 0, a NaN
    if fk == 0:
        x = got.view(np.float16).astype(np.float64).reshape(n, hkv, d)
        assert np.isnan(x[5, 0, 100]) and np.isnan(x[3, 0, partner]) and x[4, 1, 70] == -np.inf
        assert (x[30, 0] == ref.F16_MAX).any()
        ok = np.isfinite(x)
        assert (~ok).sum() == 3
        assert (np.abs(x - want)[ok] <= _half_tolerance(want, _size(want, rot, interleaved, m))[ok]).all()
    else:
        x = oracle.dequantize(fk, got).reshape(n, hkv, d)
        assert np.isfinite(x).all()
        # fp32 scale rounded to fp16 (2^-11 of the value), a code's half step; Q4_0's largest code
        # is one short on the far side of zero: a whole step there
        top = np.abs(want).reshape(n, hkv, d // 32, 32).max(axis=-1, keepdims=True)
        step = top / (127.0 if fk == 1 else 8.0)
        tol = (0.5 if fk == 1 else 1.0) * step * (1 + 2.0 ** -10) + top * 2.0 ** -11 + 2.0 ** -24 * (127 if fk == 1 else 8)
        err = np.abs(x - want).reshape(n, hkv, d // 32, 32)
        assert (err <= tol).all()


@pytest.mark.parametrize("mscale", [1.0, 1.25])
@pytest.mark.parametrize("interleaved", [False, True])
def test_cosines_and_sines_to_fp32(interleaved, mscale):
    """Pairs (a, b) that nearly cancel, a cos w = b sin w to about 2^-21, lay bare the last bits of the
    cosine and the sine: each has to be fp32's nearest but for less than half of half an ulp, the larger
    product and the result are rounded once more."""
    import torch
    import mixed_attention_quantized_gb300 as mq
    n, rot = 600, 128
    rng = np.random.default_rng(31)
    rope = mq.Rope(rot, layout=int(interleaved), mscale=mscale)
    f = np.array(rope.info()["frequencies"])
    pos = rng.integers(0, 4096, n).astype(np.int32)
    w = pos[:, None] * f  # fp64: within 2^-41
    c, s = mscale * np.cos(w), mscale * np.sin(w)
    # the a of 11 bits for which b = a c / s (or the other way round) is nearest to 11 bits
    big = np.abs(c) >= np.abs(s)
    r = np.where(big, s, c) / np.where(big, c, s)  # |r| <= 1; the larger factor's partner is a r
    best = np.full((n, rot // 2), np.inf)
    x = np.zeros((2, n, rot // 2))
    for lead in range(1024, 2048):
        exact = lead * r
        at = np.exp2(np.floor(np.log2(np.maximum(np.abs(exact), 1e-3))) - 10)
        near = np.round(exact / at) * at
        left = np.abs(near - exact)
        better = (left < best) & (np.abs(near) >= 1)
        best = np.where(better, left, best)
        x[0] = np.where(better, np.where(big, near, lead), x[0])
        x[1] = np.where(better, np.where(big, lead, near), x[1])
    x *= 16
    a, b = x
    want = a * c - b * s
    assert np.median(np.abs(want) / np.maximum(np.abs(a * c), 1)) < 2.0 ** -18
    k = np.zeros((n, 1, rot), dtype=np.float16)
    first, second = (np.s_[0::2], np.s_[1::2]) if interleaved else (np.s_[:rot // 2], np.s_[rot // 2:])
    k[:, 0, first], k[:, 0, second] = a, b
    assert (k[:, 0, first] == a).all() and (k[:, 0, second] == b).all()
    got = mq.rope_apply(rope, torch.from_numpy(k).cuda(), torch.from_numpy(pos).cuda()).cpu().numpy()
    got = got[:, 0, first].astype(np.float64)
    half = lambda v: np.spacing(np.abs(v).astype(np.float32)).astype(np.float64) / 2
    tol = 1.5 * (np.abs(a) * half(c) + np.abs(b) * half(s)) + half(a * c) + half(want)
    tol += 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    used = np.isfinite(best)
    assert used.mean() > 0.5
    assert (np.abs(got - want) <= tol)[used].all(), (np.abs(got - want) / tol)[used].max()
