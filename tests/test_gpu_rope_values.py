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
