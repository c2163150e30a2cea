"""``Q2_INT4`` products (``q2_gemv``, ``q2_gemv_x8``) against the f64 oracle.

A group's products are exact in fp32 (a small integer times an fp16 or an
8-bit integer); the tensor cores add them in fp32, each addition at most
2^-23 of the sum of magnitudes S_g of its group off (truncation), group of
them; the group sums are scaled and added with at most C / group + 16 further
roundings of 2^-24.  y is rounded once.  So with S = sum |w x|:
|y - ref| <= 2^-11 |ref| + 2^-25 + (2 group + C / group + 16) 2^-24 S,
and for 8-bit x, whose group sums are exact, without the term 2 group.
(Up to 16 tokens the kernels take the zero point off a group's sum; the bound
for that is wider, see test_gpu_int4_limits.py, and these inputs stay inside
this one.)
"""
import numpy as np
import pytest

import synth
from oracle import int4 as oint4, matvec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _matrix(q2, R, C, group, seed, zeros=True):
    d = synth.int4(R, C, group, seed, zeros)
    return q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], group)), \
        oint4.decode_f64(d["code"], d["scale"], d["zero"], group)


def _check(y, w, x, group, exact_groups=False):
    ref, S = matvec.gemv(w, x), matvec.abs_bound(w, x)
    k = w.shape[1] // group + 16 + (0 if exact_groups else 2 * group)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + k * 2.0 ** -24 * S
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} outside; worst {(err / tol).max():.2f}x"


SHAPES = [(1, 32, 32), (16, 128, 128), (17, 96, 32), (40, 192, 64), (129, 640, 128), (200, 1056, 32), (333, 4096, 128),
          (128, 17408, 64), (4096, 4096, 128), (520, 5120, 64)]


@pytest.mark.parametrize("R,C,group", SHAPES)
@pytest.mark.parametrize("ntok", [1, 2, 3, 8, 9, 16, 17, 32, 33, 64])
def test_parity(q2, R, C, group, ntok):
    pk, w = _matrix(q2, R, C, group, R + C + group, zeros=(R + ntok) % 2 == 0)
    x = synth.activations(ntok, C, 900 + ntok)
    _check(pk.gemv(torch.from_numpy(x).cuda()), w, x, group)
    x8, xs = synth.activations8(ntok, C, 901 + ntok)
    y = pk.gemv_x8(torch.from_numpy(x8).cuda(), torch.from_numpy(xs).cuda())
    _check(y, w, x8 * xs.astype(np.float64)[:, None], group, exact_groups=True)


def test_decode_is_exact(q2):
    for R, C, group, zeros in [(50, 416, 32, True), (33, 256, 128, False)]:
        pk, w = _matrix(q2, R, C, group, 77, zeros)
        got = pk.decode().view(torch.float32).view(R, C).cpu().numpy()
        assert np.array_equal(got.astype(np.float64), w)


def test_every_weight_is_where_it_belongs(q2):
    """One-hot tokens: y[t] is column c of W, exactly."""
    R, C, group = 48, 384, 64
    pk, w = _matrix(q2, R, C, group, 78)
    for c0 in range(0, C, 64):
        x = np.zeros((64, C), dtype=np.float16)
        x[np.arange(64), c0 + np.arange(64)] = 1
        want = w[:, c0: c0 + 64].T.astype(np.float16)
        assert np.array_equal(pk.gemv(torch.from_numpy(x).cuda()).cpu().numpy(), want)
        for t in (0, 13, 63):
            one = pk.gemv(torch.from_numpy(x[t: t + 1]).cuda()).cpu().numpy()
            assert np.array_equal(one[0], want[t])


@pytest.mark.parametrize("ntok", [1, 5, 16, 64])
@pytest.mark.parametrize("x8", [False, True])
def test_stays_inside_its_buffers(q2, ntok, x8):
    R, C, G = 201, 1056, 512
    pk, w = _matrix(q2, R, C, 32, 79)
    ybuf = torch.full((G + ntok * R + G,), 0x5A5A, dtype=torch.int16, device="cuda")
    y = ybuf[G: G + ntok * R].view(torch.float16).view(ntok, R)
    if x8:
        xn, xs = synth.activations8(ntok, C, 80)
        xbuf = torch.full((G + ntok * C + G,), 127, dtype=torch.int8, device="cuda")
        sbuf = torch.full((4 + ntok + 4,), float("nan"), device="cuda")
        sbuf[4: 4 + ntok] = torch.from_numpy(xs)
        xd = xbuf[G: G + ntok * C].view(ntok, C)
        xd.copy_(torch.from_numpy(xn))
        pk.gemv_x8(xd, sbuf[4: 4 + ntok], y)
        _check(y, w, xn * xs.astype(np.float64)[:, None], 32, exact_groups=True)
    else:
        xn = synth.activations(ntok, C, 80)
        xbuf = torch.full((G + ntok * C + G,), float("nan"), dtype=torch.float16, device="cuda")
        xd = xbuf[G: G + ntok * C].view(ntok, C)
        xd.copy_(torch.from_numpy(xn))
        pk.gemv(xd, y)
        _check(y, w, xn, 32)
    yb = ybuf.cpu().numpy()
    assert (yb[:G] == 0x5A5A).all() and (yb[G + ntok * R:] == 0x5A5A).all()


@pytest.mark.parametrize("ntok", [1, 8, 24])
def test_nonfinite_activations_stay_in_their_token(q2, ntok):
    R, C = 96, 512
    pk, w = _matrix(q2, R, C, 128, 81)
    x = synth.activations(ntok, C, 82)
    x[ntok - 1, 301] = np.inf
    y = pk.gemv(torch.from_numpy(x).cuda()).cpu().numpy()
    assert not np.isfinite(y[ntok - 1]).any()
    if ntok > 1:
        _check(torch.from_numpy(y[:-1]), w, x[:-1], 128)
    x8, xs = synth.activations8(ntok, C, 83)
    xs[ntok - 1] = np.nan
    y = pk.gemv_x8(torch.from_numpy(x8).cuda(), torch.from_numpy(xs).cuda()).cpu().numpy()
    assert np.isnan(y[ntok - 1]).all() and np.isfinite(y[: ntok - 1]).all()


def test_same_result_twice_and_on_another_stream(q2):
    pk, w = _matrix(q2, 1000, 4096, 128, 84)
    for ntok in (1, 7, 64):
        x = torch.from_numpy(synth.activations(ntok, 4096, 85)).cuda()
        a, b = pk.gemv(x), torch.empty((ntok, 1000), dtype=torch.float16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        pk.gemv(x, b, stream=side)
        side.synchronize()
        assert torch.equal(a, b)


def test_in_a_chain_with_2_bit_weights(q2):
    """qkv in BPDQ, then a 4-bit projection of its outputs, as one chain."""
    d = synth.bpdq(512, 256, 86)
    from oracle import bpdq as obpdq
    a = q2.Packed(q2.q2_pack_bpdq(d["plane0"], d["plane1"], d["coef"]), ntok_max=1)
    b, wb = _matrix(q2, 300, 512, 64, 87)
    x = torch.from_numpy(synth.activations(1, 256, 88)).cuda()
    y0 = torch.empty((1, 512), dtype=torch.float16, device="cuda")
    y1 = torch.empty((1, 300), dtype=torch.float16, device="cuda")
    for look in (0, 2):
        q2.Chain([(a, x, y0), (b, y0, y1)], 1, lookahead=look).run()
        torch.cuda.synchronize()
        _check(y1, wb, y0.cpu().numpy(), 64)
    wa = obpdq.decode_f64(d["plane0"], d["plane1"], d["coef"])
    xn = x.cpu().numpy()
    assert matvec.passes(y0.cpu().numpy(), matvec.gemv(wa, xn), matvec.abs_bound(wa, xn)).all()


def test_binding_refuses_what_it_would_misread(q2):
    pk, _ = _matrix(q2, 64, 256, 64, 89)
    x8 = torch.zeros((3, 256), dtype=torch.int8, device="cuda")
    xs = torch.ones(3, device="cuda")
    for bad in ((x8.half(), xs), (x8[:, :128], xs), (x8, xs[:2]), (x8, xs.half()), (x8.cpu(), xs),
                (torch.zeros((65, 256), dtype=torch.int8, device="cuda"), torch.ones(65, device="cuda"))):
        with pytest.raises(q2.Q2Error):
            pk.gemv_x8(*bad)
