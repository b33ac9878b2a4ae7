"""Refusals of the drafting and rotary entry points: bad arguments are found on the host, before any launch."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_349_b200 as pa
from paged_kv_cache_349_b200._lib import lib

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED = pa.PA_OK, pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


def ptr(addr=0x10000):
    return P(addr)


def caller(fn, names, **ok):
    assert set(names) == set(ok)

    def call(**kw):
        a = dict(ok, **kw)
        return fn(*(a[n] for n in names))
    return call


def test_decode_tree_refusals():
    names = ("out q qs kt ks vt vs T k v bt maxb lens cu masks B maxlen maxn Hq Hkv d bs NB scale pt ws wsb flag "
             "stream").split()
    call = caller(lib.pa_decode_tree, names, out=ptr(), q=ptr(), qs=1024, kt=ptr(), ks=256, vt=ptr(), vs=256, T=8,
                  k=ptr(), v=ptr(), bt=ptr(), maxb=4, lens=ptr(), cu=ptr(), masks=ptr(), B=2, maxlen=64, maxn=4, Hq=8,
                  Hkv=2, d=128, bs=16, NB=64, scale=0.1, pt=-1, ws=None, wsb=0, flag=None, stream=None)
    assert call(B=0) == OK and call(T=0) == OK
    for bad in (dict(B=-1), dict(T=-1), dict(maxlen=-1), dict(maxn=-1), dict(maxn=0), dict(NB=0), dict(maxb=-1)):
        assert call(**bad) == INVALID, bad
    for name in ("out", "q", "kt", "vt", "k", "v", "bt", "lens", "cu"):
        assert call(**{name: None}) == INVALID, name
    for name in ("out", "q", "kt", "vt", "k", "v"):
        assert call(**{name: ptr(0x10008)}) == INVALID, name
    for bad in (dict(qs=1016), dict(qs=1028), dict(ks=255), dict(ks=248), dict(vs=260), dict(vs=-256)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(bs=12), dict(Hq=6, Hkv=4), dict(Hq=32, Hkv=2), dict(NB=1 << 30), dict(B=70000)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (-0.1, math.inf, math.nan):
        assert call(scale=bad) == INVALID, bad
    assert call(pt=128, maxlen=257) == INVALID  # needs a workspace
    assert call(pt=64) == INVALID and call(pt=16) == INVALID  # partitions are multiples of 128 tokens


def test_tree_masks_refusals():
    names = "masks pos parents cu lens B T maxn flag stream".split()
    call = caller(lib.pa_tree_masks, names, masks=ptr(), pos=None, parents=ptr(), cu=ptr(), lens=ptr(), B=2, T=8, maxn=4,
                  flag=None, stream=None)
    assert call(B=0) == OK and call(T=0) == OK
    for bad in (dict(B=-1), dict(T=-1), dict(maxn=-1), dict(maxn=0), dict(masks=None), dict(parents=None),
                dict(cu=None), dict(lens=None)):
        assert call(**bad) == INVALID, bad
    assert call(maxn=pa.PA_TREE_MAX_NODES + 1) == UNSUPPORTED


def test_extend_tables_refusals():
    names = "bt maxb lens add lens_out B bs NB free nfree cur cur_out slots pos cu T cu_rows path maxp flag stream".split()
    call = caller(lib.pa_extend_tables, names, bt=ptr(), maxb=4, lens=ptr(), add=ptr(), lens_out=ptr(), B=2, bs=16, NB=64,
                  free=ptr(), nfree=9, cur=ptr(), cur_out=ptr(), slots=ptr(), pos=None, cu=ptr(), T=8, cu_rows=None,
                  path=None, maxp=0, flag=None, stream=None)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(T=-1), dict(maxb=-1), dict(NB=0), dict(nfree=-1), dict(maxp=-1), dict(cu_rows=ptr()),
                dict(path=ptr()), dict(NB=1 << 28), dict(maxb=1 << 28), dict(maxb=(1 << 27) - 1)):
        assert call(**bad) == INVALID, bad
    for name in ("bt", "lens", "add", "lens_out", "free", "cur", "cur_out", "slots", "cu"):
        assert call(**{name: None}) == INVALID, name
    assert call(bs=12) == UNSUPPORTED


ROPE = "q qs qo qos Hq k ks".split()


def test_rope_refusals():
    names = ROPE + "ko kos Hkv pos turns rot inter gain T d stream".split()
    call = caller(lib.pa_rope, names, q=ptr(), qs=1024, qo=ptr(), qos=1024, Hq=8, k=ptr(), ks=256, ko=ptr(), kos=256,
                  Hkv=2, pos=ptr(), turns=ptr(), rot=128, inter=0, gain=1.0, T=3, d=128, stream=None)
    assert call(T=0) == OK
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(Hq=0, Hkv=0), dict(pos=None), dict(turns=None), dict(qs=1016),
                dict(qos=1020), dict(ks=252), dict(kos=128), dict(q=ptr(0x10008)), dict(qo=ptr(0x10004))):
        assert call(**bad) == INVALID, bad
    for name in ("q", "qo", "k", "ko"):
        assert call(**{name: None}) == INVALID, name
    for bad in (dict(d=80), dict(rot=0), dict(rot=24), dict(rot=144), dict(rot=-16), dict(Hq=70000)):
        assert call(**bad) == UNSUPPORTED, bad


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_and_cache_refusals(fp8):
    names = ROPE + "v vs Hkv kc vc slots NB bs pos turns rot inter gain T d".split()
    names += ["sk", "sv"] * fp8 + ["flag", "stream"]
    ok = dict(q=ptr(), qs=1024, qo=ptr(), qos=1024, Hq=8, k=ptr(), ks=256, v=ptr(), vs=256, Hkv=2, kc=ptr(), vc=ptr(),
              slots=ptr(), NB=8, bs=16, pos=ptr(), turns=ptr(), rot=64, inter=1, gain=1.0, T=3, d=128, flag=None,
              stream=None)
    if fp8:
        ok.update(sk=0.5, sv=0.5)
    call = caller(lib.pa_rope_and_cache_fp8 if fp8 else lib.pa_rope_and_cache, names, **ok)
    assert call(T=0) == OK
    for bad in (dict(T=-1), dict(Hkv=0), dict(NB=0), dict(v=None), dict(kc=None), dict(vc=None), dict(slots=None),
                dict(vs=248), dict(kc=ptr(0x10008)), dict(pos=None), dict(q=None), dict(k=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=80), dict(bs=24), dict(rot=8)):
        assert call(**bad) == UNSUPPORTED, bad
    if fp8:
        for bad in (dict(sk=0.0), dict(sv=-1.0), dict(sk=math.inf), dict(sv=math.nan)):
            assert call(**bad) == INVALID, bad


def test_rope_frequency_refusals():
    f = lib.pa_rope_frequencies
    turns, gain = (ctypes.c_double * 64)(), ctypes.c_float()

    def call(rot=128, base=1e4, kind=0, factor=8.0, orig=4096.0, low=1.0, high=32.0, t=turns, g=ctypes.byref(gain)):
        return f(t, g, rot, base, kind, factor, orig, low, high)

    assert call() == OK
    assert call(t=None) == INVALID and call(g=None) == INVALID
    for bad in (dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                dict(kind=1, factor=0.5), dict(kind=1, factor=math.nan), dict(kind=2, rot=2), dict(kind=3, orig=0.0),
                dict(kind=3, low=0.0), dict(kind=3, low=32.0), dict(kind=4, high=0.5), dict(kind=4, high=math.inf)):
        assert call(**bad) == INVALID, bad
    assert call(kind=5) == UNSUPPORTED and call(kind=-1) == UNSUPPORTED


def test_rope_frequencies_against_the_formulas():
    """Each scaling against its formula in numpy; 1e-12 relative: a few fp64 operations of pow and log."""
    R, base, s, orig = 128, 500000.0, 8.0, 8192.0
    i = np.arange(R // 2)
    f = base ** (-2.0 * i / R)

    def check(got, want, gain=1.0):
        t, g = got
        assert np.allclose(t.numpy() * 2 * np.pi, want, rtol=1e-12, atol=0)
        assert g == np.float32(gain)

    check(pa.pa_rope_frequencies(R, base), f)
    check(pa.pa_rope_frequencies(R, base, "linear", s), f / s)
    check(pa.pa_rope_frequencies(R, base, "ntk", s), (base * s ** (R / (R - 2))) ** (-2.0 * i / R))
    # by wavelength: pairs that turn fewer than `low` times are slowed, more than `high` kept
    n = orig * f / (2 * np.pi)
    w = np.clip((n - 1.0) / 3.0, 0, 1)
    check(pa.pa_rope_frequencies(R, base, "by_wavelength", s, orig), (1 - w) * f / s + w * f)
    # by parts: the pair number at which a pair turns r times within orig
    at = [R * math.log(orig / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), R - 1)
    w = np.clip((i - lo) / (hi - lo), 0, 1)
    check(pa.pa_rope_frequencies(R, base, "by_parts", s, orig), w * f / s + (1 - w) * f, 0.1 * math.log(s) + 1)
    with pytest.raises(ValueError):
        pa.pa_rope_frequencies(R, base, "cubic")
    with pytest.raises(pa.PaError):
        pa.pa_rope_frequencies(R, 0.5)


def test_tree_workspace_size_of_unsplit_calls():
    assert pa.pa_decode_tree_workspace_size(4, 32, 8, 2, 128, 16, 4096, 8, -1) == 0
    assert pa.pa_decode_tree_workspace_size(0, 0, 8, 2, 128, 16, 4096, 8, 0) == 0
    assert pa.pa_decode_tree_workspace_size(4, 32, 8, 2, 128, 16, 0, 8, 0) == 0
    assert pa.pa_decode_tree_workspace_size(4, 32, 8, 2, 128, 16, 512, 8, 0) == 0  # a few tiles: never cut
    assert pa.pa_decode_tree_workspace_size(4, 32, 8, 2, 128, 16, 256, 8, 128) == 0
    assert pa.pa_decode_tree_workspace_size(4, 32, 8, 2, 128, 16, 4096, 8, 0) > 0


def test_decode_tree_scales():
    """A scale is accepted up to where scale * log2(e) leaves fp32.  The scale is looked at before the batch, which is
    too large here, so that no call goes on."""
    def call(scale):
        return lib.pa_decode_tree(ptr(), ptr(), 1024, ptr(), 256, ptr(), 256, 8, ptr(), ptr(), ptr(), 4, ptr(), ptr(), ptr(),
                                  70000, 64, 4, 8, 2, 128, 16, 64, scale, -1, None, 0, None, None)

    for good in (0.0, 1e-45, 1.0, 2.3e38):
        assert call(good) == UNSUPPORTED, good
    for bad in (2.4e38, 2.9e38, math.inf, math.nan, -1e-45):
        assert call(bad) == INVALID, bad


def test_rope_in_place_needs_one_stride():
    """A row written in place at another stride would land on rows that are still to be read."""
    names = ROPE + "ko kos Hkv pos turns rot inter gain T d stream".split()
    call = caller(lib.pa_rope, names, q=ptr(), qs=1024, qo=ptr(0x20000), qos=1024, Hq=8, k=ptr(0x30000), ks=256, ko=ptr(0x40000),
                  kos=256, Hkv=2, pos=ptr(), turns=ptr(), rot=128, inter=0, gain=1.0, T=3, d=128, stream=None)
    assert call(qo=ptr(), qos=1032) == INVALID and call(qo=ptr(), qs=2048) == INVALID
    assert call(ko=ptr(0x30000), kos=264) == INVALID and call(ko=ptr(0x30000), ks=512) == INVALID
    names = ROPE + "v vs Hkv kc vc slots NB bs pos turns rot inter gain T d flag stream".split()
    call = caller(lib.pa_rope_and_cache, names, q=ptr(), qs=1024, qo=ptr(), qos=1032, Hq=8, k=ptr(0x30000), ks=256,
                  v=ptr(0x40000), vs=256, Hkv=2, kc=ptr(0x50000), vc=ptr(0x60000), slots=ptr(), NB=8, bs=16, pos=ptr(),
                  turns=ptr(), rot=64, inter=1, gain=1.0, T=3, d=128, flag=None, stream=None)
    assert call() == INVALID
