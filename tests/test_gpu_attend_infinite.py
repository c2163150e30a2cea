"""Infinite values in the cache: an output's column with one is infinite, of its sign, in ``q2_attend`` as in the
definition (a probability is positive, and positive times infinity is infinity); with both signs it is NaN.  Other
columns, heads and sequences are as without.  Probabilities here are above 2^-30 of the largest.
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


@pytest.mark.parametrize("D,group", [(64, 1), (128, 4), (128, 12), (256, 8)])
@pytest.mark.parametrize("n", [1, 40, 900])
def test_infinite_values(q2, D, group, n):
    rng = np.random.default_rng(n + D)
    page, H = 16, 2
    need = -(-n // page)
    k, v = (rng.normal(size=(2 * need, page, H, D)).astype(np.float16) for _ in range(2))
    q = rng.normal(size=(2, H * group, D)).astype(np.float16)
    table = np.arange(2 * need, dtype=np.int32).reshape(2, need)
    dev = lambda a: torch.from_numpy(a).cuda()
    lens = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    run = lambda: q2.PagedKV(dev(k), dev(v), dev(table), H * group).attend(dev(q), lens).cpu().numpy()
    clean = run()
    rows = v.reshape(2, need * page, H, D)[0]                 # sequence 0; sequence 1 stays as it is
    want = clean.copy()
    for i, t in enumerate(sorted({0, n // 2, n - 1})):        # a token with any probability, head 0 and head 1
        rows[t, 0, 3 + i], rows[t, 1, 9 + i] = np.inf, -np.inf
        want[0, :group, 3 + i], want[0, group:, 9 + i] = np.inf, -np.inf
    if n > 1:
        rows[0, 0, 20], rows[n - 1, 0, 20] = np.inf, -np.inf
        want[0, :group, 20] = np.nan
    assert np.array_equal(run(), want, equal_nan=True)
