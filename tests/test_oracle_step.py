"""Pins of the oracles of the decode step's operators around the products:
closed forms and special cases of ``oracle.int4`` and ``oracle.norm``, and the
4-bit packer's device layout (no GPU needed)."""
import ctypes
import os
import shutil

import numpy as np
import pytest

import synth
from oracle import attend as oatt, int4 as oint4, norm as onorm
from tests import _blob


@pytest.fixture(scope="module")
def q2():
    import dequant_gemv_q2_gb300 as m
    if not os.path.exists(m.lib_path()):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("libq2.so not built and nvcc not available")
        m._build.build()
    m.load()
    return m


def test_int4_decode_of_one_byte():
    # byte 0x2f: column 0 holds 15, column 1 holds 2
    code = np.full((1, 16), 0x2F, dtype=np.uint8)
    scale = np.array([[0.5]], dtype=np.float16)
    w = oint4.decode_f64(code, scale, None, 32)
    assert np.array_equal(w[0, 0::2], np.full(16, 0.5 * 7)) and np.array_equal(w[0, 1::2], np.full(16, 0.5 * -6))
    w = oint4.decode_f64(code, scale, np.array([[15]], dtype=np.uint8), 32)
    assert (w[0, 0::2] == 0).all() and (w[0, 1::2] == 0.5 * -13).all()


def test_norm_closed_forms():
    x = np.array([[3.0, 4.0]])
    h, y = onorm.rmsnorm_f64(x, np.ones(2), 0.0)
    assert np.array_equal(h, x) and np.allclose(y, x / np.sqrt(12.5), rtol=1e-15)
    h, y = onorm.rmsnorm_f64(x, np.array([1.0, 2.0]), 0.0, residual=-x)
    assert (h == 0).all() and np.isnan(y).all()                    # 0 / sqrt(0): eps is what avoids it
    q, s = onorm.quantise_f64(np.array([[0.0, 0.0], [2.54, -1.0]]))
    assert np.array_equal(q, [[0, 0], [127, -50]]) and s[0] == 0 and s[1] == 0.02


def test_attend_closed_forms():
    v = np.arange(12.0).reshape(3, 2, 2)
    k = np.zeros((3, 2, 2))
    q = np.ones((4, 2))
    o, S, Q = oatt.attend_f64(q, k, v, 0.5)                        # equal scores: the mean
    assert np.allclose(o[:2], v[:, 0].mean(0)) and np.allclose(o[2:], v[:, 1].mean(0)) and np.allclose(S, o) and (Q == 0).all()
    k[1, 0] = np.log(2)                                            # head 0: weights 1, 2, 1 at scale 1/2
    assert np.allclose(oatt.attend_f64(q, k, v, 0.5)[0][:2], (v[0, 0] + 2 * v[1, 0] + v[2, 0]) / 4)
    assert (oatt.attend_f64(q, k[:0], v[:0], 0.5)[0] == 0).all()
    pool = np.arange(8.0).reshape(4, 2, 1, 1)
    assert oatt.gather(pool, np.array([3, 0]), 3).ravel().tolist() == [6, 7, 0]


def test_attend_refusals(q2):
    L = q2.load()
    n = ctypes.c_size_t(0)
    p = ctypes.c_void_p(1 << 20)                                                # never read
    assert L.q2_attend_workspace_bytes(2, 7, 2, 128, ctypes.byref(n)) == -2     # heads do not divide
    assert L.q2_attend_workspace_bytes(2, 8, 2, 96, ctypes.byref(n)) == -2
    assert L.q2_attend_workspace_bytes(1025, 8, 2, 128, ctypes.byref(n)) == -2
    assert L.q2_attend_workspace_bytes(2, 130, 2, 128, ctypes.byref(n)) == -2   # 65 heads to one
    assert L.q2_attend_workspace_bytes(2, 8, 2, 128, None) == -1

    def call(q=p, ldq=1024, nk=None, nv=None, ldn=0, lens=p, batch=2, heads=8, scale=0.1, out=p, ldo=1024, ws=p, wsb=1 << 30, **kv):
        f = dict(k=p, v=p, page_stride=4096, token_stride=256, head_stride=128, npages=9, page_size=16, kv_heads=2,
                 head_dim=128, table=p, table_stride=4, max_pages=4)
        f.update(kv)
        return L.q2_attend(ctypes.byref(q2._KV(**f)), q, ldq, nk, nv, ldn, lens, batch, heads, scale, out, ldo, ws, wsb, None)

    odd = ctypes.c_void_p((1 << 20) + 8)
    assert call(batch=0) == 0
    assert call(q=None) == -1 and call(lens=None) == -1 and call(out=None) == -1 and call(k=None) == -1 and call(table=None) == -1
    assert call(nk=p) == -1 and call(scale=float("inf")) == -1 and call(scale=float("nan")) == -1
    assert call(page_size=0) == -2 and call(npages=-1) == -2 and call(ldq=1023) == -2 and call(ldo=8) == -2
    assert call(table_stride=3) == -2 and call(nk=p, nv=p, ldn=8) == -2 and call(page_stride=-8) == -2
    assert call(max_pages=1 << 28, table_stride=1 << 28) == -2                  # more tokens than 32 bits count
    assert call(q=odd) == -3 and call(k=odd) == -3 and call(ldq=1028) == -3 and call(token_stride=260) == -3
    assert call(lens=ctypes.c_void_p((1 << 20) + 2)) == -3
    assert call(ws=None) == -7 and call(wsb=100) == -7 and call(ws=ctypes.c_void_p((1 << 20) + 16)) == -3


def _codes(blob, R, C, group):
    """(code values, zero points) read back from the packed layout, one element at a time."""
    h = _blob.header(blob)
    nblk, gpb = int(h["nblock"]), 128 // group
    items = _blob.section(blob, 0).reshape(-1, 1024 + gpb * 32 + (gpb * 16 if h["layout"] else 0))
    w = items[:, :1024].copy().view("<u4").reshape(-1, 2, 32, 4)
    sc = items[:, 1024: 1024 + gpb * 32].copy().view(np.float16).reshape(-1, 8, gpb, 2)
    zr = items[:, 1024 + gpb * 32:].reshape(-1, 8, gpb, 2) if h["layout"] else None
    order = [0, 0, 8, 8, 1, 1, 9, 9]
    q = np.zeros((R, C), dtype=np.int64)
    s = np.zeros((R, C // group), dtype=np.float16)
    z = np.full((R, C // group), 8, dtype=np.int64)
    for r in range(R):
        for c in range(C):
            it, cc, half = (r // 16) * nblk + c // 128, c % 128, (r // 8) % 2
            step = cc // 16
            v = int(w[it, step // 4, (r % 8) * 4 + (cc % 8) // 2, step % 4])
            nib = [n for n in range(8) if order[n] == cc % 2 + cc % 16 // 8 * 8 and n % 2 == half][0]
            q[r, c] = (v >> (4 * nib)) & 15
            s[r, c // group] = sc[it, r % 8, cc // group, half]
            if zr is not None:
                z[r, c // group] = zr[it, r % 8, cc // group, half]
    return q, s, z


@pytest.mark.parametrize("R,C,group,zeros", [(33, 160, 32, True), (16, 192, 64, False), (70, 384, 128, True)])
def test_int4_layout_round_trip(q2, R, C, group, zeros):
    d = synth.int4(R, C, group, 41, zeros)
    blob = q2.q2_pack_int4(d["code"], d["scale"], d["zero"], group)
    h = _blob.header(blob)
    assert (h["fmt"], h["R"], h["C"], h["reserved"]) == (5, R, C, group)
    q, s, z = _codes(blob, R, C, group)
    want = np.stack([d["code"] & 15, d["code"] >> 4], axis=-1).reshape(R, C)
    assert np.array_equal(q, want) and np.array_equal(s, d["scale"])
    assert np.array_equal(z, d["zero"]) if zeros else (z == 8).all()


def test_int4_pack_and_bind_refusals(q2):
    L = q2.load()
    n = ctypes.c_size_t(0)
    N = ctypes.byref(n)
    assert L.q2_pack_int4(None, None, None, 4, 128, 48, None, N) == -1          # group
    assert L.q2_pack_int4(None, None, None, 4, 160, 64, None, N) == -2          # C % group
    assert L.q2_pack_int4(None, None, None, 0, 128, 64, None, N) == -2          # R
    assert L.q2_pack_int4(None, None, None, 4, 128, 64, None, None) == -1
    d = synth.int4(5, 128, 64, 42)
    zero = d["zero"].copy()
    zero[4, 1] = 16
    with pytest.raises(q2.Q2Error) as e:
        q2.q2_pack_int4(d["code"], d["scale"], zero, 64)
    assert e.value.status == -1
    with pytest.raises(q2.Q2Error) as e:
        q2.q2_pack_int4(d["code"], d["scale"][:, :1], None, 64)
    assert e.value.status == -2
    blob = q2.q2_pack_int4(d["code"], d["scale"], d["zero"], 64)
    h, dev, x = ctypes.c_void_p(), ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
    for field, value in (("reserved", 48), ("nblock", 9), ("nslice", 7), ("layout", 0), ("layout", 2)):
        bad = blob.copy()
        hdr = np.frombuffer(bad[:_blob.HEADER.itemsize].tobytes(), dtype=_blob.HEADER).copy()
        hdr[field] = value
        bad[:_blob.HEADER.itemsize] = np.frombuffer(hdr.tobytes(), dtype=np.uint8)
        assert L.q2_bind(bad.ctypes.data, dev, ctypes.byref(h)) == -6, field
    assert L.q2_bind(blob.ctypes.data, dev, ctypes.byref(h)) == 0
    assert L.q2_workspace_bytes(h, 64, N) == 0 and n.value == 0
    assert L.q2_bytes(h, 1, N) == 0 and n.value == 2 * (1024 + 64 + 32)              # Rpad 32: two row tiles
    assert L.q2_gemv(1, h, x, x, 1, None) == -4
    assert L.q2_gemv(5, h, x, x, 65, None) == -5
    assert L.q2_gemv(5, h, ctypes.c_void_p((1 << 21) + 8), x, 1, None) == -3
    assert L.q2_gemv_x8(h, x, None, x, 1, None) == -1
    assert L.q2_gemv_x8(h, x, x, x, 0, None) == -5
    assert L.q2_gemv_x8(h, x, ctypes.c_void_p((1 << 21) + 2), x, 1, None) == -3
    L.q2_unbind(h)
    b = synth.bpdq(32, 256, 43)
    bq = q2.q2_pack_bpdq(b["plane0"], b["plane1"], b["coef"])
    assert L.q2_bind(bq.ctypes.data, dev, ctypes.byref(h)) == 0
    assert L.q2_gemv_x8(h, x, x, x, 1, None) == -4                              # 8-bit x needs 4-bit weights
    L.q2_unbind(h)


def test_norm_refusals(q2):
    L = q2.load()
    p = [ctypes.c_void_p(1 << k) for k in range(20, 28)]                        # never read
    call = lambda x=p[0], ldx=64, n=2, heads=1, C=64, r=None, ro=None, w=p[1], eps=1e-6, y=p[2], ldy=64, y8=None, s8=None: \
        L.q2_rmsnorm(x, ldx, n, heads, C, r, ro, w, eps, y, ldy, y8, s8, None)  # noqa: E731
    assert call(n=0) == 0                                                       # nothing to do
    assert call(n=-1) == -1 and call(x=None) == -1 and call(w=None) == -1 and call(y=None) == -1
    assert call(y8=p[3]) == -1                                                  # no scales
    assert call(r=p[3]) == -1 and call(ro=p[3]) == -1                           # both or neither
    assert call(eps=-1.0) == -1 and call(eps=float("nan")) == -1
    assert call(C=0) == -2 and call(C=32769, ldx=40000, ldy=40000) == -2 and call(heads=0) == -2
    assert call(ldx=63) == -2 and call(heads=2) == -2 and call(ldy=63) == -2
    assert call(x=ctypes.c_void_p((1 << 20) + 1)) == -3
    assert call(y8=p[3], s8=ctypes.c_void_p((1 << 24) + 2)) == -3
