"""``q2_rmsnorm`` against the f64 oracle.

The kernel computes in fp32 from the fp16 inputs and rounds each output once.
Relative error of y before that rounding: the sum of squares adds at most 32
terms in a row and 10 levels of a tree, (32 + 10 + 1) * 2^-24, halved by the
root; the division, the root (2 units), two products and the addition of the
residual are under 8 * 2^-24.  So |y - ref| <= (2^-11 + 2^-18) |ref| + 2^-25
(half the smallest fp16), scales to 2^-18 relative, and y8 * scale8 within
(1/2 + 127 * 2^-17) scale8 of ref.
"""
import numpy as np
import pytest

from oracle import norm as onorm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EPS = 1e-6
REL = 2.0 ** -18


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _draw(ntok, heads, C, seed, gap=0):
    rng = np.random.default_rng(seed)
    wide = rng.normal(size=(ntok, heads * C + gap)).astype(np.float16)
    wide[:, rng.integers(0, heads * C, size=2)] *= np.float16(30)
    x = wide[:, : heads * C].reshape(ntok, heads, C)
    w = (1 + 0.3 * rng.normal(size=C)).astype(np.float16)
    r = rng.normal(size=(ntok, heads, C)).astype(np.float16)
    return wide, x, w, r


def _close16(got, ref):
    got = got.cpu().numpy().astype(np.float64)
    tol = (2.0 ** -11 + REL) * np.abs(ref) + 2.0 ** -25
    assert (np.abs(got - ref) <= tol).all(), f"worst {(np.abs(got - ref) / tol).max():.2f}x"


def _close8(q, s, y):
    _, sref = onorm.quantise_f64(y)
    q, s = q.cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64)
    assert (np.abs(s - sref) <= REL * sref).all()
    assert (np.abs(q * s[..., None] - y) <= (0.5 + 127 * 2.0 ** -17) * s[..., None]).all()
    assert (np.abs(q) <= 127).all()


@pytest.mark.parametrize("C", [1, 7, 64, 128, 130, 256, 264, 512, 1000, 4096, 4099, 5120, 8192, 8200, 17408, 32768, 32767])
@pytest.mark.parametrize("ntok", [1, 5])
def test_all_outputs(q2, C, ntok):
    wide, x, w, r = _draw(ntok, 1, C, C + ntok)
    n = q2.RmsNorm(w, EPS)
    xd, rd = torch.from_numpy(x[:, 0].copy()).cuda(), torch.from_numpy(r[:, 0].copy()).cuda()
    q8 = torch.zeros((ntok, C), dtype=torch.int8, device="cuda")
    s8 = torch.zeros(ntok, device="cuda")
    ro, out = torch.empty_like(rd), torch.empty_like(xd)
    n.apply(xd, residual=rd, residual_out=ro, out=out, out8=q8, scale8=s8)
    h, y = onorm.rmsnorm_f64(x[:, 0], w, EPS, r[:, 0])
    _close16(ro, h)
    _close16(out, y)
    _close8(q8, s8, y)
    # without a residual, fp16 only
    _close16(n.apply(xd), onorm.rmsnorm_f64(x[:, 0], w, EPS)[1])


@pytest.mark.parametrize("heads,C,gap", [(40, 128, 2048), (8, 128, 24), (3, 64, 5), (2, 100, 0), (5, 256, 8), (4, 513, 3)])
def test_heads_of_a_strided_projection_in_place(q2, heads, C, gap):
    wide, x, w, _ = _draw(9, heads, C, heads * C, gap)
    d = torch.from_numpy(wide).cuda()
    view = d[:, : heads * C].unflatten(1, (heads, C))
    q2.RmsNorm(w, EPS).apply(view, out=view)
    _close16(view, onorm.rmsnorm_f64(x, w, EPS)[1])
    assert np.array_equal(d[:, heads * C:].cpu().numpy(), wide[:, heads * C:])       # the gap is not touched


@pytest.mark.parametrize("off", [1, 4, 8])
def test_misaligned_rows(q2, off):
    C = 4096
    _, x, w, r = _draw(3, 1, C, 70 + off)
    buf = torch.full((3 * C + 16,), float("nan"), dtype=torch.float16, device="cuda")
    xd = buf[off: off + 3 * C].view(3, C)
    xd.copy_(torch.from_numpy(x[:, 0].copy()))
    rd = torch.from_numpy(r[:, 0].copy()).cuda()
    out = q2.RmsNorm(w, EPS).apply(xd, residual=rd)
    h, y = onorm.rmsnorm_f64(x[:, 0], w, EPS, r[:, 0])
    _close16(out, y)
    _close16(rd, h)                                                                    # the residual was updated in place


@pytest.mark.parametrize("C,ntok", [(65, 40), (127, 33), (255, 9), (510, 21), (513, 700), (4099, 400), (5125, 333), (8201, 160), (17401, 5)])
@pytest.mark.parametrize("offs", [(0, 0, 0, 0), (1, 2, 3, 5), (7, 7, 7, 7)])
def test_rows_that_begin_anywhere(q2, C, ntok, offs):
    """Odd widths, each tensor at its own offset inside a buffer whose other elements have to stay as they are."""
    _, x, w, r = _draw(ntok, 1, C, C + ntok)
    sizes = {"x": x[:, 0], "r": r[:, 0], "y": None, "q": None}
    bufs, views = {}, {}
    for (name, data), off in zip(sizes.items(), offs):
        dt = torch.int8 if name == "q" else torch.float16
        bufs[name] = torch.full((ntok * C + 32,), 77, dtype=dt, device="cuda")
        views[name] = bufs[name][off: off + ntok * C].view(ntok, C)
        if data is not None:
            views[name].copy_(torch.from_numpy(data.copy()))
    s8 = torch.zeros(ntok, device="cuda")
    q2.RmsNorm(w, EPS).apply(views["x"], residual=views["r"], out=views["y"], out8=views["q"], scale8=s8)
    h, y = onorm.rmsnorm_f64(x[:, 0], w, EPS, r[:, 0])
    _close16(views["r"], h)
    _close16(views["y"], y)
    _close8(views["q"], s8, y)
    assert np.array_equal(views["x"].cpu().numpy(), x[:, 0])
    for name, off in zip(sizes, offs):
        assert (bufs[name][:off] == 77).all() and (bufs[name][off + ntok * C:] == 77).all()
    # 8 bits alone, and fp16 alone in place
    q2.RmsNorm(w, EPS).apply(views["x"], out8=views["q"], scale8=s8)
    y = onorm.rmsnorm_f64(x[:, 0], w, EPS)[1]
    _close8(views["q"], s8, y)
    q2.RmsNorm(w, EPS).apply(views["x"], out=views["x"])
    _close16(views["x"], y)


def test_rows_do_not_depend_on_the_batch(q2):
    _, x, w, r = _draw(64, 1, 5120, 80)
    n = q2.RmsNorm(w, EPS)
    xd, rd = torch.from_numpy(x[:, 0].copy()).cuda(), torch.from_numpy(r[:, 0].copy()).cuda()
    whole = n.apply(xd, residual=rd, residual_out=torch.empty_like(rd))
    for t in (0, 31, 63):
        one = n.apply(xd[t: t + 1], residual=rd[t: t + 1].clone())
        assert torch.equal(one[0], whole[t])


def test_zero_rows_and_nonfinite_rows(q2):
    C = 512
    x = torch.ones((4, C), dtype=torch.float16, device="cuda")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 500] = float("inf")
    q8, s8 = torch.zeros((4, C), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    out = torch.empty_like(x)
    q2.RmsNorm(np.ones(C, dtype=np.float16), EPS).apply(x, out=out, out8=q8, scale8=s8)
    assert (out[0] == 0).all() and s8[0] == 0 and (q8[0] == 0).all()
    assert torch.isnan(out[1]).all() and not torch.isfinite(s8[1]) and not torch.isfinite(s8[2])
    assert not torch.isfinite(q8[1:3].float() * s8[1:3, None]).any()
    assert torch.equal(out[3], x[3]) and (q8[3] == 127).all()


def test_no_rows_and_another_stream(q2):
    n = q2.RmsNorm(np.ones(128, dtype=np.float16), EPS)
    assert n.apply(torch.empty((0, 128), dtype=torch.float16, device="cuda")).shape == (0, 128)
    x = torch.randn(7, 128, device="cuda").half()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    n.apply(x, out=out, stream=side)
    side.synchronize()
    _close16(out, onorm.rmsnorm_f64(x.cpu().numpy(), np.ones(128), EPS)[1])


def test_binding_refuses_what_it_would_misread(q2):
    n = q2.RmsNorm(np.ones(128, dtype=np.float16), EPS)
    x = torch.zeros((4, 128), dtype=torch.float16, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x.cpu()), dict(x=x[:, :64]), dict(x=x.t().contiguous().t()),
                dict(x=x, residual=x[:2]), dict(x=x, out8=x.to(torch.int8)), dict(x=x, out=x.float()),
                dict(x=x, residual_out=x.clone())):
        with pytest.raises(q2.Q2Error):
            n.apply(**bad)
