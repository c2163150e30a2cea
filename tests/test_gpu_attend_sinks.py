"""``q2_attend`` where one token's score stands far above the rest and its value row is zero: the output is made of
probabilities far below 1.

The bound is that of test_gpu_attend.py, |o - ref| <= 2^-11 |ref| + 2^-25 + 2 (e + 2^-19 + n / 16 2^-23) sum p |v|
with e = 2 (D + 8) 2^-23 Q + 2^-21; the sink adds nothing to sum p |v|, so every probability has to be right
relative to itself.  (A probability is two fp16 numbers of 2^15 p: 2^-20.7 of itself, or 2^-40 of the largest, which
at the widest gap here is 2^-11 of each and of either sign: 2^-14 and less of a sum of 8000, inside 2 e.)
"""
import numpy as np
import pytest

from oracle import attend as oatt

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _run(q2, n, D, group, gap, sinks, page=16, kv_heads=2, seed=0):
    """Keys with small scores, those of `sinks` with scores `gap` above them (natural logarithm) and values of zero."""
    rng = np.random.default_rng(seed)
    need = -(-n // page)
    k = rng.normal(size=(need, page, kv_heads, D)) * 0.1
    v = 500 + 100 * rng.normal(size=(need, page, kv_heads, D))
    q = rng.choice([-1.0, 1.0], size=(1, kv_heads * group, D))
    q[0] = np.repeat(q[0, ::group], group, axis=0)                 # the heads of a group look for the same key
    for t in sinks:
        k[t // page, t % page] = q[0, ::group] * gap * D ** -0.5   # scale q.k = gap
        v[t // page, t % page] = 0
    k, v, q = (a.astype(np.float16) for a in (k, v, q))
    table = rng.permutation(need).astype(np.int32)[None]
    dev = lambda a: torch.from_numpy(a).cuda()
    inv = np.argsort(table[0])                                      # page i of the sequence lies at table[0][i]
    kv = q2.PagedKV(dev(k[inv]), dev(v[inv]), dev(table), kv_heads * group)
    got = kv.attend(dev(q), torch.tensor([n], dtype=torch.int32, device="cuda"))[0].cpu().numpy().astype(np.float64)
    flat = [a.reshape(-1, kv_heads, D)[:n] for a in (k, v)]
    ref, S, Q = oatt.attend_f64(q[0], *flat, D ** -0.5)
    e = 2 * (D + 8) * 2.0 ** -23 * Q[:, None] + 2.0 ** -21 + 2.0 ** -19 + n / 16 * 2.0 ** -23
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2 * e * S
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst {(err / tol).max():.2f}x, {(err / np.abs(ref)).max():.2e} relative"


@pytest.mark.parametrize("gap", [9, 12, 14, 16, 17, 18, 20])
@pytest.mark.parametrize("D,group", [(64, 4), (128, 4), (128, 16), (256, 2)])
@pytest.mark.parametrize("where", ["first", "each warp's first tile", "last"])
def test_a_long_sequence_behind_a_sink(q2, gap, D, group, where):
    n = 8192
    sinks = {"first": [0], "each warp's first tile": [0, 16, 32, 48], "last": [n - 1]}[where]
    _run(q2, n, D, group, gap, sinks, seed=gap)


@pytest.mark.parametrize("gap", [12, 15])
@pytest.mark.parametrize("n", [2, 17, 64, 200])
def test_a_short_sequence_behind_a_sink(q2, gap, n):
    _run(q2, n, 128, 4, gap, [0], page=24, seed=n)
