"""``Q2_INT4`` products whose columns are split over a cluster: many launches one behind another give the same bits.

Every CTA of a cluster reads the others' sums and leaves only when they have read its own; the sums are added in a fixed
order, so any launch has to repeat the first one's output, which is checked against the oracle with test_gpu_int4.py's
bound.
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


@pytest.mark.parametrize("R,C", [(128, 512), (130, 1024), (640, 2176), (1000, 4096), (2048, 3200)])
@pytest.mark.parametrize("ntok", [3, 8, 11, 16, 17, 33, 64])
def test_launches_repeat(q2, R, C, ntok):
    d = synth.int4(R, C, 64, 900 + R, True)
    pk = q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], 64))
    x = synth.activations(ntok, C, 901)
    x8, xs = synth.activations8(ntok, C, 902)
    xd, x8d, xsd = (torch.from_numpy(a).cuda() for a in (x, x8, xs))
    w = oint4.decode_f64(d["code"], d["scale"], d["zero"], 64)
    for call, xn, k in ((lambda: pk.gemv(xd), x, 128), (lambda: pk.gemv_x8(x8d, xsd), x8 * xs.astype(np.float64)[:, None], 0)):
        ys = torch.stack([call() for _ in range(40)])
        ref, S = matvec.gemv(w, xn), matvec.abs_bound(w, xn)
        tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (k + C // 64 + 16) * 2.0 ** -24 * S
        assert (np.abs(ys[0].cpu().numpy().astype(np.float64) - ref) <= tol).all()
        assert (ys == ys[0]).all()
