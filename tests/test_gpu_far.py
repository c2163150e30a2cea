"""Offsets beyond 2^31 elements: the norm's and the cache's, in sparse use of large buffers.

Tolerances as in the operators' own tests: the norm's row is compared with
the same row at a small offset (bit-identical), attention with the same
sequences in a small pool (bit-identical: pages do not change the order of
the sums).
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


def test_norm_rows_far_apart(q2):
    C, ld, n = 520, 2 ** 30 + 8, 4
    rng = np.random.default_rng(50)
    x = torch.from_numpy(rng.normal(size=(n, C)).astype(np.float16)).cuda()
    norm = q2.RmsNorm(rng.normal(size=C).astype(np.float16))
    want = norm.apply(x)
    big = torch.empty((n - 1) * ld + C, dtype=torch.float16, device="cuda")
    far = big.as_strided((n, C), (ld, 1))
    far.copy_(x)
    assert torch.equal(norm.apply(far), want)
    norm.apply(x, out=far)
    assert torch.equal(far, want)


@pytest.mark.parametrize("order", ["token", "head"])
def test_pages_far_apart(q2, order):
    page, H, G, D, lens = 16, 8, 4, 128, [77, 1, 300]
    each, rng = page * H * D, np.random.default_rng(51)
    P = 2 ** 31 // each + 40                             # the last pages begin past 2^31 elements
    need = [-(-n // page) for n in lens]
    shape = (lambda p: (p, page, H, D)) if order == "token" else (lambda p: (p, H, page, D))
    seen = (lambda t: t) if order == "token" else (lambda t: t.transpose(1, 2))
    near = [torch.from_numpy(rng.normal(size=shape(sum(need))).astype(np.float16)).cuda() for _ in range(2)]
    far = [torch.empty(shape(P), dtype=torch.float16, device="cuda") for _ in range(2)]
    ids = torch.arange(sum(need))
    for a, b in zip(far, near):
        a[P - sum(need):].copy_(b)
    q = torch.from_numpy(rng.normal(size=(3, H * G, D)).astype(np.float16)).cuda()
    new = [torch.from_numpy(rng.normal(size=(3, H, D)).astype(np.float16)).cuda() for _ in range(2)]
    out = []
    for pools, first in ((near, 0), (far, P - sum(need))):
        table, at = torch.zeros((3, max(need)), dtype=torch.int32), 0
        for b, m in enumerate(need):
            table[b, :m] = ids[at: at + m] + first
            at += m
        kv = q2.PagedKV(seen(pools[0]), seen(pools[1]), table.cuda(), q_heads=H * G)
        out.append(kv.attend(q, torch.tensor(lens, dtype=torch.int32, device="cuda"), *new).clone())
    assert torch.isfinite(out[0]).all() and torch.equal(out[0], out[1])
    for a, b in zip(far, near):                          # the new rows as well
        assert torch.equal(a[P - sum(need):], b)
