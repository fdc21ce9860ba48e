"""Host side of the page-scaled 8-bit formats and of rotary positions (no GPU): sizes,
refusals, the frequency tables, and the reference the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

import _page8 as ref
import mixed_attention_quantized_gb300 as mq

FAKE = 1 << 20  # aligned non-null "device" address; never dereferenced on the host
NUL = ctypes.c_void_p(0)


def _p(off=0):
    return ctypes.c_void_p(FAKE + off)


def _desc(fk=mq.I8_PAGE, fv=mq.I8_PAGE, pages=64, hkv=2, d=128):
    return mq.cache_desc(pages, hkv, d, fk, fv, FAKE, FAKE, FAKE, FAKE)


def test_e4m3_reference_matches_torch():
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(codes, ref.e4m3_values().astype(np.float32))
    y = np.concatenate([np.linspace(-448, 448, 100001), np.linspace(-0.05, 0.05, 20001)]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ref.e4m3_round(y.astype(np.float64)).astype(np.float32), want)


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
def test_reference_append_keeps_half_a_step(fmt):
    rng = np.random.default_rng(fmt)
    x = rng.standard_normal((32, 2, 64)) * np.exp2(rng.integers(-6, 6, size=(32, 1, 1)))
    c = ref.PageCache(fmt, 1, 2, 64)
    c.append(x, np.arange(32))
    d = c.scale[0].astype(np.float64)[None, :, None]
    got = c.values()[0].transpose(1, 0, 2)
    step = d if fmt == ref.I8 else np.maximum(np.abs(x) * 2.0 ** -3, d * 2.0 ** -9)
    assert (np.abs(got - x) <= step / 2 * (1 + 1e-5)).all()
    top = np.abs(x).max(axis=(0, 2))
    if fmt == ref.I8:
        np.testing.assert_allclose(c.scale[0], top / 127, rtol=1e-6)
    else:
        assert (top <= 448 * c.scale[0]).all() and (top > 224 * c.scale[0]).all()


def test_reference_scale_is_the_least_power_of_two():
    for a in (448.0, np.nextafter(np.float32(448), np.float32(500)), 447.9, 1.0, 0.875, 0.8750001, 2.0 ** -24, 65504.0):
        d = float(ref.scale_for(ref.E4M3, np.array([a]))[0])
        assert math.log2(d) == int(math.log2(d)) and np.float32(a) <= 448 * d and np.float32(a) > 224 * d


def test_cache_bytes_of_page_scaled_formats():
    for f in (mq.I8_PAGE, mq.E4M3_PAGE):
        total, planes = mq.kv_cache_bytes(mq.cache_desc(10, 8, 128, f, f))
        assert planes == [10 * 8 * 32 * 128, 10 * 8 * 4] * 2 and total == sum(planes)
    # a page-scaled format pairs only with itself
    for other in (mq.F16, mq.Q8_0, mq.Q4_0, mq.E4M3_PAGE):
        assert mq.kv_cache_bytes(mq.cache_desc(10, 8, 128, mq.I8_PAGE, other))[0] == 0
        assert mq.kv_cache_bytes(mq.cache_desc(10, 8, 128, other, mq.I8_PAGE))[0] == 0
    assert mq.kv_cache_bytes(mq.cache_desc(10, 8, 128, 5, 5))[0] == 0
    assert mq.block_bytes(mq.I8_PAGE) == 36 and mq.row_bytes(mq.E4M3_PAGE, 64) == 64


def test_page_scaled_refusals():
    lib = mq.load()
    d = _desc()
    assert lib.mixattn_kv_append_quant(ctypes.byref(d), NUL, NUL, NUL, 0, NUL) == mq.OK
    assert lib.mixattn_kv_append_quant(ctypes.byref(d), NUL, _p(), _p(), 3, NUL) == mq.ERR_INVALID_ARG
    mixed = _desc(mq.I8_PAGE, mq.E4M3_PAGE)
    assert lib.mixattn_kv_append_quant(ctypes.byref(mixed), _p(), _p(), _p(), 3, NUL) == mq.ERR_UNSUPPORTED
    no_scale = _desc()
    no_scale.v_scale = 0
    assert lib.mixattn_kv_append_quant(ctypes.byref(no_scale), _p(), _p(), _p(), 3, NUL) == mq.ERR_INVALID_ARG
    # the entry point without allocations does not build these formats' tiles
    one = mq._i32_array([0]), mq._i32_array([1])
    st = lib.mixattn_mixed_attention_noalloc(ctypes.byref(d), 8, _p(), _p(), 4, 1, one[1], one[0], one[0], _p(), NUL)
    assert st == mq.ERR_UNSUPPORTED
    # a workspace is sized for every row kind
    ws = ctypes.c_size_t(0)
    for kind, seq, off in ((0, 100, 99), (1, 100, 96), (1, 100, 0), (1, 1, 0)):
        assert lib.mixattn_workspace_bytes(ctypes.byref(d), 8, 1, mq._i32_array([kind]), mq._i32_array([seq]),
                                           mq._i32_array([off]), 4, ctypes.byref(ws)) == mq.OK
        assert ws.value > 0


SCALINGS = [("none", mq.ROPE_SCALE_NONE, {}),
            ("linear", mq.ROPE_SCALE_LINEAR, dict(factor=4.0)),
            ("ramp", mq.ROPE_SCALE_RAMP, dict(factor=8.0, original_ctx=4096, low=1.0, high=32.0)),
            ("bands", mq.ROPE_SCALE_BANDS, dict(factor=8.0, original_ctx=8192, low=1.0, high=4.0))]


@pytest.mark.parametrize("rot", [16, 32, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("name,kind,kw", SCALINGS)
def test_frequencies(rot, base, name, kind, kw):
    r = mq.Rope(rot, base=base, scaling=kind, **kw)
    got = r.info()
    f, m = ref.frequencies(rot, name, base, kw.get("factor", 1.0), kw.get("original_ctx", 0), kw.get("low", 0.0),
                           kw.get("high", 0.0))
    np.testing.assert_allclose(got["frequencies"], f, rtol=1e-12)
    assert got["mscale"] == pytest.approx(m, rel=1e-12)
    assert mq.Rope(rot, base=base, scaling=kind, mscale=0.5, **kw).info()["mscale"] == 0.5


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), mq.ERR_INVALID_ARG), (dict(rot_dim=144), mq.ERR_INVALID_ARG),
    (dict(rot_dim=24), mq.ERR_UNSUPPORTED), (dict(rot_dim=10), mq.ERR_UNSUPPORTED),
    (dict(rot_dim=64, layout=2), mq.ERR_INVALID_ARG), (dict(rot_dim=64, base=1.0), mq.ERR_INVALID_ARG),
    (dict(rot_dim=64, base=float("nan")), mq.ERR_INVALID_ARG), (dict(rot_dim=64, mscale=-1.0), mq.ERR_INVALID_ARG),
    (dict(rot_dim=64, scaling=4), mq.ERR_INVALID_ARG),
    (dict(rot_dim=64, scaling=1, factor=0.0), mq.ERR_INVALID_ARG),
    (dict(rot_dim=64, scaling=2, factor=0.5, original_ctx=64, low=1.0, high=2.0), mq.ERR_INVALID_ARG),
    (dict(rot_dim=64, scaling=2, factor=2.0, original_ctx=0, low=1.0, high=2.0), mq.ERR_INVALID_ARG),
    (dict(rot_dim=64, scaling=3, factor=2.0, original_ctx=64, low=2.0, high=2.0), mq.ERR_INVALID_ARG),
    (dict(rot_dim=64, scaling=3, factor=2.0, original_ctx=64, low=0.0, high=2.0), mq.ERR_INVALID_ARG)])
def test_rope_create_refusals(kw, status):
    with pytest.raises(mq.MixattnError) as e:
        mq.Rope(**kw)
    assert e.value.status == status


def test_rope_apply_refusals():
    lib = mq.load()
    h = mq.Rope(64)._handle

    def go(rope=h, x=FAKE, xs=512, out=FAKE + (1 << 20), os_=512, pos=FAKE, n=3, heads=4, d=128):
        return lib.mixattn_rope_apply(rope, ctypes.c_void_p(x), xs, ctypes.c_void_p(out), os_, ctypes.c_void_p(pos), n,
                                      heads, d, NUL)

    assert go(n=0, x=0, out=0, pos=0) == mq.OK
    assert go(rope=NUL) == mq.ERR_INVALID_ARG
    assert go(n=-1) == mq.ERR_INVALID_ARG
    assert go(heads=0) == mq.ERR_INVALID_ARG
    assert go(d=96) == mq.ERR_UNSUPPORTED
    for kw in (dict(x=0), dict(out=0), dict(pos=0), dict(x=FAKE + 8), dict(out=FAKE + 2), dict(pos=FAKE + 2),
               dict(xs=511), dict(xs=504), dict(xs=516), dict(os_=256), dict(xs=1 << 40)):
        assert go(**kw) == mq.ERR_INVALID_ARG, kw
    # overlaps: shifted rows, in place with another stride
    assert go(out=FAKE + 16) == mq.ERR_INVALID_ARG
    assert go(out=FAKE + 1024 + 512) == mq.ERR_INVALID_ARG
    assert go(out=FAKE, os_=1024) == mq.ERR_INVALID_ARG
    assert go(xs=1024, os_=1024, out=FAKE + 1040) == mq.ERR_INVALID_ARG
    # a table for heads of 128 on heads of 64
    assert lib.mixattn_rope_apply(mq.Rope(128)._handle, _p(), 512, _p(1 << 20), 512, _p(), 3, 4, 64, NUL) == \
        mq.ERR_INVALID_ARG


def test_rope_append_refusals():
    lib = mq.load()
    h = mq.Rope(128)._handle
    c = _desc()

    def go(cache=c, rope=h, hq=4, q=FAKE, qs=512, qo=FAKE + (1 << 20), qos=512, k=FAKE, ks=256, v=FAKE, vs=256, pos=FAKE,
           slots=FAKE, n=3):
        v_ = ctypes.c_void_p
        return lib.mixattn_rope_append(ctypes.byref(cache), rope, hq, v_(q), qs, v_(qo), qos, v_(k), ks, v_(v), vs,
                                       v_(pos), v_(slots), n, NUL)

    assert go(n=0, q=0, k=0, pos=0) == mq.OK
    assert go(rope=NUL) == mq.ERR_INVALID_ARG
    assert go(cache=_desc(mq.I8_PAGE, mq.E4M3_PAGE)) == mq.ERR_UNSUPPORTED
    assert go(cache=_desc(d=64)) == mq.ERR_INVALID_ARG  # rot 128 > head_dim 64
    for kw in (dict(hq=-1), dict(n=-1), dict(q=0), dict(qo=0), dict(k=0), dict(v=0), dict(pos=0), dict(slots=0),
               dict(k=FAKE + 4), dict(v=FAKE + 2), dict(ks=128), dict(vs=260), dict(qs=256), dict(qos=511),
               dict(qo=FAKE + 32), dict(slots=FAKE + 1)):
        assert go(**kw) == mq.ERR_INVALID_ARG, kw


def test_python_wrappers_check_shapes():
    torch = pytest.importorskip("torch")
    r = mq.Rope(64)
    x = torch.zeros(3, 4, 128, dtype=torch.float16)
    pos = torch.zeros(3, dtype=torch.int32)
    for bad in (x.float(), x[:2], x.transpose(1, 2), x[:, :, ::2], x[0]):
        with pytest.raises(ValueError):
            mq.rope_apply(r, bad, pos)
    with pytest.raises(ValueError):
        mq.rope_apply(r, x, pos.long())
    with pytest.raises(ValueError):
        mq.rope_apply(r, x, pos, out=torch.zeros(3, 4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):  # not on a GPU
        mq.rope_apply(r, x, pos)
    cache = mq.KVCache(4, 4, 128, mq.I8_PAGE, mq.I8_PAGE, k_quant=x)
    with pytest.raises(ValueError):
        mq.rope_append(cache, r, x, x[:, :2], x, pos, pos)
    with pytest.raises(ValueError):
        mq.rope_append(cache, r, x, x, x, pos, pos[:2])
