"""Latent caches on the host: sizes, and what the C entry points refuse before any launch."""
import ctypes

import pytest

import mixed_attention_quantized_gb300 as mq

FAKE = 1 << 20  # 256-byte aligned, never dereferenced on the host


def _desc(pages=64, page=32, latent=512, rope=64, data=FAKE):
    return mq.LatentCacheDesc(pages, page, latent, rope, data)


def test_cache_bytes():
    f = mq.load().mixattn_latent_cache_bytes
    assert f(ctypes.byref(_desc(10, data=0))) == 10 * 32 * 576 * 2
    for bad in (dict(pages=0), dict(page=16), dict(latent=256), dict(rope=32), dict(pages=1 << 27)):
        assert f(ctypes.byref(_desc(**bad))) == 0


def _append(desc=None, rope=None, heads=4, q=None, q_out=None, c=FAKE, cs=512, k=FAKE, ks=64, pos=FAKE, slots=FAKE, n=3):
    q = q or mq.HeadsDesc(FAKE, 4 * 192, 192)
    q_out = q_out or mq.HeadsDesc(2 * FAKE, 4 * 576, 576)
    rope = rope or mq.Rope(64)
    return mq.load().mixattn_latent_append(ctypes.byref(desc or _desc()), rope._handle, heads, ctypes.byref(q),
                                           ctypes.byref(q_out), c, cs, k, ks, pos, slots, n, None)


def test_append_refuses_before_it_launches():
    assert _append(n=0) == mq.OK
    heads = mq.HeadsDesc
    for bad in (dict(desc=_desc(data=0)), dict(desc=_desc(data=FAKE + 128)), dict(rope=mq.Rope(32)), dict(heads=-1),
                dict(n=-1), dict(c=0), dict(c=FAKE + 8), dict(cs=500), dict(cs=516), dict(k=0), dict(ks=56), dict(pos=0),
                dict(slots=0), dict(q=heads(0, 768, 192)), dict(q=heads(FAKE + 2, 768, 192)), dict(q=heads(FAKE, 100, 192)),
                dict(q=heads(FAKE, 768, 56)), dict(q=heads(FAKE, 768, -192)), dict(q=heads(FAKE, 192, 192)),
                dict(q_out=heads(FAKE + 64, 4 * 576, 576))):
        assert _append(**bad) == mq.ERR_INVALID_ARG, bad
    assert _append(desc=_desc(page=16)) == mq.ERR_UNSUPPORTED
    assert _append(heads=1 << 17) == mq.ERR_UNSUPPORTED


def _plan(cache=None, heads=16, scale=0.07, kinds=(0,), seqs=(100,), offs=(99,), pages=4):
    h, ws = ctypes.c_void_p(0), ctypes.c_size_t(0)
    st = mq.load().mixattn_latent_plan_create(ctypes.byref(h), ctypes.byref(cache or _desc()), heads, scale, len(seqs),
                                              mq._i32_array(kinds), mq._i32_array(seqs), mq._i32_array(offs), pages,
                                              ctypes.byref(ws))
    if h.value:
        mq.load().mixattn_latent_plan_destroy(h)
    return st


def test_plans_refuse_before_they_allocate():
    for bad in (dict(heads=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0), dict(offs=(98,)),
                dict(seqs=(0,), offs=(-1,)), dict(kinds=(1,), offs=(100,)), dict(kinds=(2,)), dict(kinds=(7,)),
                dict(pages=3), dict(pages=0), dict(seqs=(65 * 32,), offs=(65 * 32 - 1,), pages=100),
                dict(kinds=(), seqs=(), offs=()), dict(cache=_desc(data=0)), dict(cache=_desc(pages=-1))):
        assert _plan(**bad) == mq.ERR_INVALID_ARG, bad
    for bad in (dict(heads=129), dict(kinds=(3,), seqs=(1025,), offs=(0,), pages=40), dict(cache=_desc(latent=256))):
        assert _plan(**bad) == mq.ERR_UNSUPPORTED, bad


@pytest.mark.parametrize("bad", [dict(heads=0), dict(scale=0.0), dict(seqs=(5,), offs=(5,)), dict(seqs=(5,), offs=(-1,)),
                                 dict(seqs=(), offs=()), dict(heads=1 << 20, seqs=(1 << 20,), offs=(0,))])
def test_expanded_plans_refuse_before_they_allocate(bad):
    kw = {**dict(heads=4, scale=0.07, seqs=(40,), offs=(0,)), **bad}
    h, ws = ctypes.c_void_p(0), ctypes.c_size_t(0)
    st = mq.load().mixattn_expanded_plan_create(ctypes.byref(h), kw["heads"], kw["scale"], len(kw["seqs"]),
                                                mq._i32_array(kw["seqs"]), mq._i32_array(kw["offs"]), ctypes.byref(ws))
    assert st == mq.ERR_INVALID_ARG and not h.value


def test_runs_refuse_a_missing_plan():
    lib = mq.load()
    assert lib.mixattn_latent_run(None, FAKE, FAKE, None, 0, FAKE, FAKE, 1 << 20, None) == mq.ERR_INVALID_ARG
    q = mq.HeadsDesc(FAKE, 192, 192)
    assert lib.mixattn_expanded_run(None, ctypes.byref(q), ctypes.byref(q), FAKE, 64, ctypes.byref(q), FAKE, FAKE, 1 << 20,
                                    None) == mq.ERR_INVALID_ARG
    assert lib.mixattn_latent_plan_update(None, 1, None, None, None, 1, None) == mq.ERR_INVALID_ARG


def test_a_cache_whose_data_changes_is_looked_at_again():
    import copy
    import torch
    c = mq.LatentCache(2)
    x = torch.zeros(2 * 32 * 576, dtype=torch.float16)
    c.data = x.view(2, 32, 576)
    assert c._ref()._obj.data == x.data_ptr()
    for bad in (c.data.view(torch.bfloat16), x.view(32, 576, 2).permute(2, 0, 1), x.view(2, 576, 32), x.view(1, 64, 576)):
        c.data = bad  # the same memory
        with pytest.raises(ValueError):
            c._ref()
    c.data = torch.ones(2, 32, 576, dtype=torch.float16)
    assert c._ref()._obj.data == c.data.data_ptr()
    assert bool((copy.deepcopy(c).data == 1).all())
