"""Expanded plans of so many heads that a token's output passes 2^31 elements are refused before they allocate (no GPU):
the kernel counts them in 32 bits."""
import ctypes

import pytest

import mixed_attention_quantized_gb300 as mq


@pytest.mark.parametrize("heads", [(1 << 16) + 1, 1 << 24])
@pytest.mark.parametrize("seqs,offs", [((2,), (0,)), ((9,), (8,))])
def test_too_many_heads(heads, seqs, offs):
    h, ws = ctypes.c_void_p(0), ctypes.c_size_t(0)
    st = mq.load().mixattn_expanded_plan_create(ctypes.byref(h), heads, 0.07, 1, mq._i32_array(seqs), mq._i32_array(offs),
                                                ctypes.byref(ws))
    assert st == mq.ERR_UNSUPPORTED and not h.value
