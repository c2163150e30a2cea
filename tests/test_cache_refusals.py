"""What the cache's entry points refuse, on the host: nothing is launched (no GPU needed)."""
import ctypes
import os
import shutil

import pytest

EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -7
P = ctypes.c_void_p(1 << 20)                                                    # never read
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD4 = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def q2():
    import dequant_gemv_q2_gb300 as m
    if not os.path.exists(m.lib_path()):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("libq2.so not built and nvcc not available")
        m._build.build()
    m.load()
    return m


def _kv(q2, **kw):
    f = dict(k=P, v=P, page_stride=4096, token_stride=256, head_stride=128, npages=9, page_size=16, kv_heads=2, head_dim=128,
             table=P, table_stride=4, max_pages=4)
    return q2._KV(**{**f, **kw})


def _kv4(q2, **kw):
    f = dict(k=P, v=P, page_stride=2048, token_stride=128, head_stride=64, ks=P, vs=P, s_page_stride=64, s_token_stride=4,
             s_head_stride=2, npages=9, page_size=16, kv_heads=2, head_dim=128, group=64, table=P, table_stride=4, max_pages=4)
    return q2._KV4(**{**f, **kw})


CACHE = [(dict(page_size=0), ESHAPE), (dict(npages=-1), ESHAPE), (dict(max_pages=-1), ESHAPE), (dict(kv_heads=0), ESHAPE), (dict(head_dim=96), ESHAPE),
         (dict(page_stride=-16), ESHAPE), (dict(table_stride=3), ESHAPE), (dict(max_pages=1 << 28, table_stride=1 << 28), ESHAPE),
         (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(table=None), EINVAL), (dict(k=ODD), EALIGN), (dict(v=ODD), EALIGN),
         (dict(table=ODD4), EALIGN), (dict(token_stride=260), EALIGN), (dict(head_stride=4), EALIGN)]
CACHE4 = CACHE + [(dict(group=128), ESHAPE), (dict(group=0), ESHAPE), (dict(ks=None), EINVAL), (dict(vs=None), EINVAL), (dict(ks=ODD), EALIGN),
                  (dict(s_token_stride=-2), ESHAPE), (dict(s_token_stride=3), EALIGN), (dict(s_head_stride=1), EALIGN), (dict(page_stride=2056), EALIGN)]


def _each_cache(q2, call):
    for make, bad in ((_kv, CACHE), (_kv4, CACHE4)):
        four = make is _kv4
        for kw, status in bad:
            assert call(four, ctypes.byref(make(q2, **kw))) == status, (four, kw)
        assert call(four, None) == EINVAL


@pytest.mark.parametrize("four", [False, True])
def test_append(q2, four):
    L = q2.load()
    fn = L.q2_append4 if four else L.q2_append
    kv = (_kv4 if four else _kv)(q2)

    def call(kv=kv, bounds=None, q=P, ldq=1024, qo=P, ldqo=1024, heads=8, k=P, ldk=256, v=P, ldv=256, starts=None, lens=P, batch=2, ntok=2, rope=None):
        r = None if rope is None else ctypes.byref(q2._Rope(**{**dict(table=P, positions=100, rot=64, interleaved=0), **rope}))
        return fn(kv if kv is None else ctypes.byref(kv), bounds, q, ldq, qo, ldqo, heads, k, ldk, v, ldv, starts, lens, batch, ntok, r, None)

    assert call(batch=0, ntok=0) == 0 and call(starts=P, ntok=0) == 0
    assert call(k=None) == EINVAL and call(v=None) == EINVAL and call(lens=None) == EINVAL and call(qo=None) == EINVAL and call(q=None) == EINVAL
    assert call(ntok=3) == ESHAPE and call(batch=-1) == ESHAPE and call(batch=1025, ntok=1025) == ESHAPE and call(ntok=-1, starts=P) == ESHAPE
    assert call(heads=0) == ESHAPE and call(heads=65537) == ESHAPE and call(ldq=1016) == ESHAPE and call(ldqo=8) == ESHAPE
    assert call(ldk=248) == ESHAPE and call(ldv=0) == ESHAPE
    assert call(q=ODD) == EALIGN and call(qo=ODD) == EALIGN and call(k=ODD) == EALIGN and call(v=ODD) == EALIGN and call(ldk=260) == EALIGN
    assert call(ldq=1028) == EALIGN and call(starts=ODD4, ntok=2) == EALIGN and call(lens=ODD4) == EALIGN and call(bounds=ODD) == EALIGN
    for rope, status in ((dict(rot=8), ESHAPE), (dict(rot=24), ESHAPE), (dict(rot=144), ESHAPE), (dict(positions=-1), ESHAPE), (dict(table=None), EINVAL),
                         (dict(table=ODD), EALIGN)):
        assert call(rope=rope) == status
    make = _kv4 if four else _kv
    assert call(make(q2, page_size=24), bounds=P) == ESHAPE and call(make(q2, page_size=96), bounds=P) == ESHAPE


def test_caches(q2):
    L = q2.load()
    _each_cache(q2, lambda four, kv: (L.q2_append4 if four else L.q2_append)(kv, None, None, 0, None, 0, 0, P, 256, P, 256, None, P, 2, 2, None, None))
    _each_cache(q2, lambda four, kv: (L.q2_read4 if four else L.q2_read)(kv, P, 256, P, 256, None, P, 2, 2, None))
    _each_cache(q2, lambda four, kv: (L.q2_select4 if four else L.q2_select)(kv, P, P, 1024, P, 2, 8, 4, 0, 1, P, None))


@pytest.mark.parametrize("four", [False, True])
def test_read(q2, four):
    L = q2.load()
    fn, kv = (L.q2_read4, _kv4(q2)) if four else (L.q2_read, _kv(q2))
    call = lambda k=P, ldk=256, v=P, ldv=256, starts=None, lens=P, batch=2, ntok=2: \
        fn(ctypes.byref(kv), k, ldk, v, ldv, starts, lens, batch, ntok, None)  # noqa: E731
    assert call(batch=0, ntok=0) == 0 and call(k=None, v=None) == 0 and call(starts=P, ntok=0) == 0
    assert call(lens=None) == EINVAL and call(ntok=1) == ESHAPE and call(ldk=248) == ESHAPE and call(ldv=8) == ESHAPE
    assert call(k=ODD) == EALIGN and call(v=ODD) == EALIGN and call(ldv=260) == EALIGN and call(starts=ODD4) == EALIGN


def test_attend4_and_blocks(q2):
    L = q2.load()

    def call4(q=P, ldq=1024, lens=P, batch=2, heads=8, sel=None, nsel=0, scale=0.1, out=P, ldo=1024, ws=P, wsb=1 << 30, **kv):
        return L.q2_attend4(ctypes.byref(_kv4(q2, **kv)), q, ldq, lens, batch, heads, sel, nsel, scale, out, ldo, ws, wsb, None)

    def call16(q=P, ldq=1024, lens=P, batch=2, heads=8, sel=P, nsel=3, scale=0.1, out=P, ldo=1024, ws=P, wsb=1 << 30, **kv):
        return L.q2_attend_blocks(ctypes.byref(_kv(q2, **kv)), q, ldq, lens, batch, heads, sel, nsel, scale, out, ldo, ws, wsb, None)

    for call in (call4, call16):
        assert call(batch=0) == 0
        assert call(q=None) == EINVAL and call(lens=None) == EINVAL and call(out=None) == EINVAL and call(k=None) == EINVAL and call(table=None) == EINVAL
        assert call(scale=float("inf")) == EINVAL and call(scale=float("nan")) == EINVAL
        assert call(heads=7) == ESHAPE and call(heads=130) == ESHAPE and call(batch=1025) == ESHAPE and call(head_dim=96) == ESHAPE
        assert call(page_size=0) == ESHAPE and call(ldq=1016) == ESHAPE and call(ldo=8) == ESHAPE and call(table_stride=3) == ESHAPE
        assert call(max_pages=1 << 28, table_stride=1 << 28) == ESHAPE
        assert call(q=ODD) == EALIGN and call(out=ODD) == EALIGN and call(k=ODD) == EALIGN and call(ldq=1028) == EALIGN and call(lens=ODD4) == EALIGN
        assert call(ws=None) == EWORKSPACE and call(wsb=100) == EWORKSPACE and call(ws=ctypes.c_void_p((1 << 20) + 16)) == EALIGN
    assert call4(sel=P) == ESHAPE and call4(nsel=2) == ESHAPE and call4(sel=ODD4, nsel=2) == EALIGN and call4(sel=P, nsel=-1) == ESHAPE
    assert call4(group=16) == ESHAPE and call4(ks=None) == EINVAL and call4(s_page_stride=1 << 33) == ESHAPE and call4(page_stride=1 << 37) == ESHAPE
    assert call16(sel=None) == EINVAL and call16(nsel=0) == ESHAPE and call16(sel=ODD4) == EALIGN
    assert L.q2_attend4(None, P, 0, P, 1, 8, None, 0, 0.1, P, 0, P, 1 << 30, None) == EINVAL


@pytest.mark.parametrize("four", [False, True])
def test_select(q2, four):
    L = q2.load()
    fn, make = (L.q2_select4, _kv4) if four else (L.q2_select, _kv)

    def call(bounds=P, q=P, ldq=1024, lens=P, batch=2, heads=8, nsel=4, first=0, last=1, sel=P, **kv):
        return fn(ctypes.byref(make(q2, **kv)), bounds, q, ldq, lens, batch, heads, nsel, first, last, sel, None)

    assert call(batch=0) == 0
    assert call(bounds=None) == EINVAL and call(q=None) == EINVAL and call(lens=None) == EINVAL and call(sel=None) == EINVAL
    assert call(nsel=0) == ESHAPE and call(nsel=32769) == ESHAPE and call(first=-1) == ESHAPE and call(last=-1) == ESHAPE and call(first=4) == ESHAPE
    assert call(heads=7) == ESHAPE and call(heads=130) == ESHAPE and call(batch=1025) == ESHAPE and call(ldq=1016) == ESHAPE
    assert call(page_size=24) == ESHAPE and call(page_size=96) == ESHAPE
    assert call(max_pages=32769, table_stride=32769, page_size=64) == ESHAPE                    # more blocks than it holds
    assert call(bounds=ODD) == EALIGN and call(q=ODD) == EALIGN and call(ldq=1028) == EALIGN and call(lens=ODD4) == EALIGN and call(sel=ODD4) == EALIGN
