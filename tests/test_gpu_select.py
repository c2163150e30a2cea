"""``q2_select`` against the f64 oracle: the selections are equal, ties and all.

The oracle's scores are sums of at most 256 exact products in f64, rounded to
fp32; the kernel's are summed to 2^-36 of the magnitudes.  Both round to the same
fp32 number unless the exact score is within that of the middle of two, which
none of these inputs' is.
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


class Case:
    def __init__(self, lens, kv_heads, q_group, D, page=64, seed=0, bits=16):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.G, self.D, self.page = lens, kv_heads, q_group, D, page
        B, sub = len(lens), -(-page // 64)
        need = [-(-max(n, 0) // page) for n in lens]
        P = sum(need) + 2
        ids = rng.permutation(P)
        self.table = np.full((B, max(need + [1]) + 1), -7, dtype=np.int32)
        at = 0
        for b in range(B):
            self.table[b, : need[b]] = ids[at: at + need[b]]
            at += need[b]
        self.bounds = np.sort(rng.normal(size=(P, sub, kv_heads, 2, D)), axis=3).astype(np.float16)
        self.q = rng.normal(size=(B, kv_heads * q_group, D)).astype(np.float16)
        self.bits = bits

    def cache(self, q2):
        P, dev = self.bounds.shape[0], "cuda"
        self.dbounds, self.dtable = torch.from_numpy(self.bounds).cuda(), torch.from_numpy(self.table).cuda()
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        wide = torch.zeros((len(self.lens), self.H * self.G * self.D + 16), dtype=torch.float16, device=dev)
        self.dq = wide[:, : self.H * self.G * self.D].unflatten(1, (self.H * self.G, self.D))
        self.dq.copy_(torch.from_numpy(self.q))
        shape = (P, self.page, self.H)
        if self.bits == 16:
            k = torch.empty(shape + (self.D,), dtype=torch.float16, device=dev)
            return q2.PagedKV(k, k, self.dtable, self.H * self.G, bounds=self.dbounds)
        k, ks = torch.empty(shape + (self.D // 2,), dtype=torch.uint8, device=dev), torch.empty(shape + (self.D // 32, 2), dtype=torch.float16, device=dev)
        return q2.PagedKV4(k, ks, k, ks, self.dtable, self.H * self.G, bounds=self.dbounds)

    def scores(self, b, h):
        first = np.arange(0, max(self.lens[b], 0), 64)
        bound = self.bounds[self.table[b, first // self.page], first % self.page // 64, h].astype(np.float64)
        q = self.q[b, h * self.G: (h + 1) * self.G].astype(np.float64)
        with np.errstate(invalid="ignore", over="ignore"):
            u = np.maximum(q[:, None] * bound[None, :, 0], q[:, None] * bound[None, :, 1]).sum(2).astype(np.float32)
        bad = ~np.isfinite(u).all(0)
        return np.where(bad, np.inf, np.where(np.isfinite(u), u, 0).max(0) if len(first) else 0)

    def expect(self, n, first, last):
        out = np.full((len(self.lens), self.H, n), -1, dtype=np.int32)
        for b in range(len(self.lens)):
            for h in range(self.H):
                s = self.scores(b, h).astype(np.float64)
                m = len(s)
                s = np.where(s == np.inf, 1e300, s)
                s[: first] = np.inf
                if last:
                    s[max(0, m - last):] = np.inf
                best = np.sort(np.argsort(-s, kind="stable")[:n])
                out[b, h, : len(best)] = best
        return out

    def check(self, q2, n, first=0, last=1):
        got = self.cache(q2).select(self.dq, self.dlens, n, first=first, last=last).cpu().numpy()
        want = self.expect(n, first, last)
        assert got.shape == want.shape
        off = [(b, h) for b in range(len(self.lens)) for h in range(self.H) if not np.array_equal(got[b, h], want[b, h])]
        assert not off, f"{off[:5]}: {got[off[0]]} not {want[off[0]]}"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_group", [1, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("n,first,last", [(1, 0, 1), (1, 0, 0), (8, 1, 1), (13, 2, 3), (4, 4, 0)])
def test_ragged_batch(q2, D, q_group, n, first, last):
    c = Case([0, 1, 64, 65, 640, 900, 8000, 513], 2, q_group, D, 64, D + q_group + n)
    c.check(q2, n, first, last)
    assert q2.device_errors() == 0


@pytest.mark.parametrize("page", [1, 16, 32, 64, 128, 256, 4096])
@pytest.mark.parametrize("bits", [16, 4])
def test_page_sizes(q2, page, bits):
    Case([5000, 77, 1300], 3, 4, 128, page, page, bits).check(q2, 9)


@pytest.mark.parametrize("lens,kv_heads,n", [([131072], 8, 64), ([1 << 20], 1, 2048), ([40000] * 3, 1, 1), ([6400] * 40, 8, 99), ([64 * 1000], 2, 999),
                                             ([64 * 1000], 2, 1000), ([64 * 1000], 2, 1001)])
def test_long_sequences_and_large_selections(q2, lens, kv_heads, n):
    Case(lens, kv_heads, 4, 64, 256, n).check(q2, n, min(1, n - 1), 1)


def test_equal_scores_go_to_the_lower_block(q2):
    c = Case([64 * 500, 64 * 300], 2, 4, 128, 64, 1)
    c.bounds[:] = c.bounds[:1]                          # all alike
    c.check(q2, 20, 0, 0)
    c.check(q2, 20, 2, 5)
    rng = np.random.default_rng(2)
    c.bounds[:] = c.bounds[rng.integers(0, 7, size=len(c.bounds))] * np.float16(1)
    c.bounds[rng.integers(0, len(c.bounds), 30)] *= np.float16(1.5)
    for n in (1, 7, 100, 299):
        c.check(q2, n, 0, 0)
    c.bounds[:] = 0
    c.bounds[::2] = np.float16(-0.0)                    # zero is zero
    c.check(q2, 11, 0, 0)


def test_scores_a_hair_apart(q2):
    """Bounds that differ by a step in one small column, below large ones that cancel: an fp32 sum would not tell them apart."""
    c = Case([64 * 400], 1, 2, 128, 64, 3)
    c.bounds[:] = c.bounds[:1]
    c.bounds[:, 0, 0, :, 5], c.bounds[:, 0, 0, :, 70] = 30000.0, -30000.0
    c.q[0, :, 5] = c.q[0, :, 70] = 100.0
    rng = np.random.default_rng(4)
    c.bounds[:, 0, 0, 1, 17] = np.float16(0.25) + np.float16(2.0 ** -12) * rng.permutation(len(c.bounds)).astype(np.float16)
    c.q[0, :, 17] = 2.0 ** -9
    c.check(q2, 50, 0, 0)


def test_what_is_not_finite_comes_first(q2):
    c = Case([64 * 200], 2, 3, 128, 64, 5)
    pages = c.table[0, :200]
    c.bounds[pages[17], 0, 0, 1, 3] = np.nan
    c.bounds[pages[50], 0, 1, 0, 100], c.bounds[pages[50], 0, 1, 1, 100] = -np.inf, np.inf
    c.bounds[pages[90], 0, 0] = [[-65504.0], [65504.0]]
    c.check(q2, 3, 0, 0)
    c.check(q2, 3, 1, 1)
    assert 17 in c.expect(3, 1, 1)[0, 0]
    c.q[0, 1, 7] = np.nan                               # every block is then
    c.check(q2, 4, 0, 1)


def test_wrong_lengths_and_pages(q2):
    c = Case([6400, 6400, 6400], 2, 4, 64, 64, 6)
    want = c.expect(5, 0, 1)
    cache = c.cache(q2)
    c.dlens[0], c.dlens[1] = -3, c.table.shape[1] * 64 + 1
    got = cache.select(c.dq, c.dlens, 5).cpu().numpy()
    assert q2.device_errors() == q2.ERR_LENGTH and (got[:2] == -1).all() and np.array_equal(got[2], want[2])
    c.dlens.fill_(6400)
    c.dtable[1, 31] = -1
    got = cache.select(c.dq, c.dlens, 5).cpu().numpy()
    assert q2.device_errors() == q2.ERR_PAGE and (got[1] == 31).any(1).all() and np.array_equal(got[::2], want[::2])


def test_given_output_captured_and_on_another_stream(q2):
    c = Case([6400, 100, 20000], 2, 4, 128, 64, 7)
    cache, want = c.cache(q2), torch.from_numpy(c.expect(12, 0, 1)).cuda()
    guard = torch.full((3 * 2 * 12 + 64,), 99, dtype=torch.int32, device="cuda")
    out = guard[32:-32].view(3, 2, 12)
    assert cache.select(c.dq, c.dlens, 12, out=out) is out and torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.select(c.dq, c.dlens, 12, out=out)
    out.zero_()
    graph.replay()
    assert torch.equal(out, want) and (guard[:32] == 99).all() and (guard[-32:] == 99).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cache.select(c.dq, c.dlens, 12, stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_binding_refuses_what_it_would_misread(q2):
    c = Case([640, 100], 2, 4, 64, 64, 8)
    cache = c.cache(q2)
    ok = dict(q=c.dq, lens=c.dlens, blocks=4)
    for kw in (dict(blocks=0), dict(blocks=2, first=2), dict(first=-1), dict(last=-1), dict(q=c.dq.float()), dict(q=c.dq[:, :4]),
               dict(lens=c.dlens.long()), dict(lens=c.dlens[:1]), dict(out=torch.zeros((2, 2, 5), dtype=torch.int32, device="cuda")),
               dict(out=torch.zeros((2, 2, 4), device="cuda"))):
        with pytest.raises(q2.Q2Error):
            cache.select(**{**ok, **kw})
    bare = q2.PagedKV(cache.k, cache.k, c.dtable, 8)
    with pytest.raises(q2.Q2Error):
        bare.select(**ok)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("large", [1.0, 64.0, 1024.0, 16384.0])
def test_keys_below_the_normal_numbers(q2, D, large):
    """Bounds of a few steps of fp16's smallest, under queries of which one column is larger than the others: the tensor cores
    align such numbers as if they were 2^-14, so what they drop is far above 2^-23 of the products.  All scores here are
    multiples of 2^-30 below 2^-9, exact in fp32; equal ones go to the lower block."""
    c = Case([64 * 2000, 64 * 333], 2, 4, D, 64, 9)
    rng = np.random.default_rng(10)
    c.bounds[:] = np.sort(rng.integers(-16, 17, size=c.bounds.shape), axis=3) * 2.0 ** -24
    c.bounds[..., 5::32] = 2.0 ** -24                   # (the error's bound takes columns 32 apart together)
    c.q[:] = np.rint(rng.normal(size=c.q.shape) * 64) / 64
    c.q[..., 5] = large
    for n in (1, 50, 300):
        c.check(q2, n, 0, 0)
    c.q[:], c.bounds[:] = c.q * 2.0 ** -20, c.bounds * 2.0 ** 10            # the queries are, and the keys hardly
    c.check(q2, 50, 0, 0)
