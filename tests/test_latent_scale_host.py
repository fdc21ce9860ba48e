"""The range of softmax_scale, ends included (no GPU: what passes the checks may still lack a device)."""
import ctypes

import pytest

import mixed_attention_quantized_gb300 as mq


def _status(scale):
    lib, one = mq.load(), mq._i32_array([5])
    desc = mq.LatentCacheDesc(4, 32, 512, 64, 1 << 20)
    out = []
    for form in range(2):
        h, ws = ctypes.c_void_p(0), ctypes.c_size_t(0)
        if form:
            st = lib.mixattn_expanded_plan_create(ctypes.byref(h), 4, scale, 1, one, mq._i32_array([0]), ctypes.byref(ws))
            destroy = lib.mixattn_expanded_plan_destroy
        else:
            st = lib.mixattn_latent_plan_create(ctypes.byref(h), ctypes.byref(desc), 4, scale, 1, mq._i32_array([0]), one,
                                                mq._i32_array([4]), 1, ctypes.byref(ws))
            destroy = lib.mixattn_latent_plan_destroy
        if h.value:
            destroy(h)
        out.append(st)
    return out


@pytest.mark.parametrize("scale", [1e-20, 1e6, 0.07, 1.0])
def test_inside(scale):
    assert mq.ERR_INVALID_ARG not in _status(scale)


@pytest.mark.parametrize("scale", [0.9e-20, 1.01e6, 0.0, -1.0, float("inf"), float("nan")])
def test_outside(scale):
    assert _status(scale) == [mq.ERR_INVALID_ARG] * 2
