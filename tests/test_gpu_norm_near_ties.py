"""The 8-bit output of ``q2_rmsnorm`` is rint(y / scale8) to the last step, values near n + 1/2 among them.

With eps = 0 and x = +-1 the mean of squares is exactly 1, so y is +-weight, exactly, and scale8 = fp32(max / 127):
what y8 has to be follows in fp32 without a tolerance.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _weights(C, unit, rng):
    """Odd multiples of `unit` under a maximum of 254 units (y / scale8 is n + 1/2 up to rounding), then random ones."""
    w = rng.uniform(-254, 254, size=C) * unit
    half = np.arange(1, 254, 2) * unit
    n = min(C - 1, 127)
    w[:n], w[n] = rng.permutation(half)[:n], 254 * unit
    return rng.permutation(w).astype(np.float16)


@pytest.mark.parametrize("C", [64, 128, 256, 500, 512, 1000, 4096, 4099, 8192, 8200, 17408, 17401])
@pytest.mark.parametrize("unit", [7 / 256, 13 / 256, 7 / 1024])
@pytest.mark.parametrize("ntok", [3, 400])
def test_values_near_ties(q2, C, unit, ntok):
    rng = np.random.default_rng(C + ntok)
    w = _weights(C, unit, rng)
    x = torch.from_numpy(rng.choice([-1.0, 1.0], size=(ntok, C)).astype(np.float16)).cuda()
    q8, s8 = torch.zeros((ntok, C), dtype=torch.int8, device="cuda"), torch.zeros(ntok, device="cuda")
    q2.RmsNorm(w, 0.0).apply(x, out8=q8, scale8=s8)
    y = x.cpu().numpy().astype(np.float32) * w.astype(np.float32)
    s = np.float32(np.abs(w).max()) / np.float32(127)
    assert (s8.cpu().numpy() == s).all()
    assert np.array_equal(q8.cpu().numpy(), np.rint(y / s).astype(np.int8))
