"""What ``Packed.gemv``, ``Chain`` and ``Rotation.apply`` would misread is refused on the host, before any launch; shapes
that hold the same rows are taken."""
import numpy as np
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
R, C = 96, 512


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _handles(q2):
    d, e = synth.int4(R, C, 64, 950, True), synth.bpdq(R, C, 951)
    return [q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], 64)),
            q2.Packed(q2.q2_pack_bpdq(e["plane0"], e["plane1"], e["coef"]))]


def _bad_rows(width):
    """fp16 [3][width] as the C call would read it, in every way wrong."""
    new = lambda *shape, dtype=torch.float16: torch.zeros(shape, dtype=dtype, device="cuda")
    return [new(3, width, dtype=torch.int8), new(3, width, dtype=torch.float32), new(3, width).cpu(), new(3, width - 8),
            new(3, width + 8), new(3, 2 * width)[:, :width], new(width, 3).t(), new(3, 2, width)]


def test_gemv(q2):
    x = torch.from_numpy(synth.activations(3, C, 952)).cuda()
    for pk in _handles(q2):
        want = pk.gemv(x)
        for bad in _bad_rows(C):
            with pytest.raises(q2.Q2Error):
                pk.gemv(bad)
        for bad in _bad_rows(R) + [torch.zeros((2, R), dtype=torch.float16, device="cuda")]:
            with pytest.raises(q2.Q2Error):
                pk.gemv(x, bad)
        with pytest.raises(q2.Q2Error):
            pk.gemv(x[0, : C - 8])
        # the same rows in other shapes
        assert torch.equal(pk.gemv(x.view(3, 4, C // 4)), want)
        flat, more = torch.zeros(3 * R, dtype=torch.float16, device="cuda"), torch.full((5, R), 7.0, dtype=torch.float16, device="cuda")
        assert torch.equal(pk.gemv(x, flat).view(3, R), want)
        pk.gemv(x, more)
        assert torch.equal(more[:3], want) and (more[3:] == 7).all()


def test_chain(q2):
    a = _handles(q2)[1]
    x, y = torch.zeros((3, C), dtype=torch.float16, device="cuda"), torch.zeros((3, R), dtype=torch.float16, device="cuda")
    for bad in _bad_rows(C):
        with pytest.raises(q2.Q2Error):
            q2.Chain([(a, x, y), (a, bad, y)], 3)
    for bad in _bad_rows(R):
        with pytest.raises(q2.Q2Error):
            q2.Chain([(a, x, bad)], 3)
    with pytest.raises(q2.Q2Error):
        q2.Chain([(a, x, y)], 4)
    q2.Chain([(a, x, y)], 2, 0).run()


def test_rotation(q2):
    inp = synth.rotation(1024, 1024, 953)
    rot = q2.Rotation(inp["signs"], inp["q"], 1024, 1024)
    x = torch.zeros((3, 1024), dtype=torch.float16, device="cuda")
    for bad in _bad_rows(1024):
        with pytest.raises(q2.Q2Error):
            rot.apply(bad)
        with pytest.raises(q2.Q2Error):
            rot.apply(x, bad)
    assert rot.apply(x[0]).shape == (1, 1024)
