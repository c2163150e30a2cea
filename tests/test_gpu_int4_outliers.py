"""``Q2_INT4`` products with a few activations far above the rest, as projections behind a gate have them, over weights
that are zero there (q = z): they must not show in the output, at any token count.

A group's products (q - z) x are exact in fp32 and summed on the tensor cores, each addition at most 2^-23 of the sum
of magnitudes of its group off: the bound of test_gpu_int4.py with S = sum |w x|, to which an outlier over a zero weight
adds nothing, |y - ref| <= 2^-11 |ref| + 2^-25 + (2 group + C / group + 16) 2^-24 S.
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


@pytest.mark.parametrize("ntok", [1, 2, 3, 8, 9, 16, 17, 64])
@pytest.mark.parametrize("C,group", [(128, 32), (256, 128), (1024, 64)])
@pytest.mark.parametrize("zeros", [False, True])
def test_outliers_over_zero_weights(q2, ntok, C, group, zeros):
    R, big = 512, [5, C // 2 + 8]                              # one outlier in an even column of either half
    d = synth.int4(R, C, group, 800 + C, zeros)
    z = d["zero"] if zeros else np.full((R, C // group), 8, dtype=np.uint8)
    x = synth.activations(ntok, C, 801)
    for c, value in zip(big, (6e4, -2e4)):
        byte = d["code"][:, c // 2]
        at = z[:, c // group]
        d["code"][:, c // 2] = (byte & 0x0F) | at << 4 if c % 2 else (byte & 0xF0) | at
        x[:, c] = value
    w = oint4.decode_f64(d["code"], d["scale"], d["zero"], group)
    assert (w[:, big] == 0).all()
    y = q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], group)).gemv(torch.from_numpy(x).cuda())
    ref, S = matvec.gemv(w, x), matvec.abs_bound(w, x)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (2 * group + C // group + 16) * 2.0 ** -24 * S
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} outside; worst {(err / tol).max():.2f}x"
