"""All-zero rows of ``q2_rmsnorm`` give zeros and scale8 = 0 whatever eps is, 0 included; the other rows are as ever."""
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


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-6])
@pytest.mark.parametrize("C", [1, 100, 128, 512, 4096, 4099, 17408])
def test_zero_rows(q2, C, eps):
    x = torch.ones((5, C), dtype=torch.float16, device="cuda")
    x[1], x[4, 0] = 0, float("nan")
    r = torch.zeros_like(x)
    q8, s8 = torch.ones((5, C), dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda")
    out = torch.ones_like(x)
    q2.RmsNorm(np.full(C, 2, dtype=np.float16), eps).apply(x, residual=r, out=out, out8=q8, scale8=s8)
    assert (r[1] == 0).all() and (out[1] == 0).all() and (q8[1] == 0).all() and s8[1] == 0
    assert (out[[0, 2, 3]] == 2).all() and (q8[[0, 2, 3]] == 127).all()
    assert torch.isnan(out[4]).all() and not torch.isfinite(s8[4])
