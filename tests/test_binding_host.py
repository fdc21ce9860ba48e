"""What a user's program may do with the binding's objects around its calls (no GPU)."""
import copy
import ctypes
import pickle

import pytest

import mixed_attention_quantized_gb300 as mq

torch = pytest.importorskip("torch")


def _used_cache():
    cache = mq.KVCache.allocate(4, 2, 64, mq.Q8_0, mq.Q8_0, device="cpu", fill=7)
    cache.note = "kept"
    # a call that the library answers without a GPU (no tokens) has the descriptor made and kept
    st = mq.load().mixattn_kv_append_quant(cache._ref(), None, None, None, 0, None)
    assert st == mq.OK
    return cache


@pytest.mark.parametrize("how", [copy.deepcopy, copy.copy, lambda c: pickle.loads(pickle.dumps(c))])
def test_a_used_cache_can_be_copied(how):
    cache = _used_cache()
    other = how(cache)
    assert (other.num_pages, other.head_dim, other.k_fmt, other.note) == (4, 64, mq.Q8_0, "kept")
    for name in ("k_quant", "k_scale", "v_quant", "v_scale"):
        assert torch.equal(getattr(other, name), getattr(cache, name))
    # each describes its own planes
    for c in (cache, other):
        d = ctypes.cast(c._ref(), ctypes.POINTER(mq.KVCacheDesc)).contents
        assert d.k_quant == c.k_quant.data_ptr() and d.v_scale == c.v_scale.data_ptr()


def test_a_cache_whose_planes_change_is_described_anew():
    cache = _used_cache()
    cache.k_quant = cache.k_quant.clone()
    d = ctypes.cast(cache._ref(), ctypes.POINTER(mq.KVCacheDesc)).contents
    assert d.k_quant == cache.k_quant.data_ptr()
