"""``q2_attend`` against the f64 oracle.

A score is a sum of D products, exact in fp32, added by the tensor cores with
at most 2^-23 of the sum of magnitudes each; times scale * log2(e) (two
roundings) and minus the maximum it is off by at most
d = (D + 4) 2^-23 Q, Q = the largest scale * sum |q k|, plus 2^-24 of its own
value (at most 2 Q); exp2 adds 2^-22 relative.  So every probability has a
relative error of e = 2 (D + 8) 2^-23 Q + 2^-21 at most, and the joins of
warps and CTAs a few more exp2 and roundings: + 2^-19.  The numerators add
terms of p = hi + lo (2^-22), one step of at most 2^-23 of the sum of
magnitudes per 16 tokens, at most n / 16 of them.  Together
|o - ref| <= 2^-11 |ref| + 2^-25 + 2 (e + 2^-19 + n / 16 2^-23) sum p |v|.
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


class Case:
    """A cache whose unused places hold NaN, queries and new rows inside one wider buffer."""

    def __init__(self, lens, kv_heads, group, D, page, seed, order="token", new=False, spare=0, peak=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.G, self.D, self.page, self.new = lens, kv_heads, group, D, page, new
        B, HQ = len(lens), kv_heads * group
        need = [-(-max(n, 0) // page) for n in lens]
        P = sum(need) + 2
        ids = rng.permutation(P)
        self.k, self.v = (np.full((P, page, kv_heads, D), np.nan, dtype=np.float16) for _ in range(2))
        self.table = np.full((B, max(need + [1]) + spare), -7, dtype=np.int32)      # never to be used
        at = 0
        for b, n in enumerate(lens):
            self.table[b, : need[b]] = ids[at: at + need[b]]
            at += need[b]
            for t in range(n - (1 if new else 0)):
                pg = self.table[b, t // page]
                self.k[pg, t % page], self.v[pg, t % page] = rng.normal(size=(2, kv_heads, D)) * peak
        self.wide = rng.normal(size=(B, (HQ + 2 * kv_heads) * D + 8)).astype(np.float16)
        self.q = self.wide[:, : HQ * D].reshape(B, HQ, D)
        self.nk = self.wide[:, HQ * D: (HQ + kv_heads) * D].reshape(B, kv_heads, D)
        self.nv = self.wide[:, (HQ + kv_heads) * D: (HQ + 2 * kv_heads) * D].reshape(B, kv_heads, D)
        self.scale = D ** -0.5
        # on the GPU
        d = [torch.from_numpy(x).cuda() for x in (self.k, self.v)]
        if order == "head":
            d = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in d]
        self.dk, self.dv = d
        self.dwide = torch.from_numpy(self.wide).cuda()
        self.dq = self.dwide[:, : HQ * D].unflatten(1, (HQ, D))
        self.dnk = self.dwide[:, HQ * D: (HQ + kv_heads) * D].unflatten(1, (kv_heads, D))
        self.dnv = self.dwide[:, (HQ + kv_heads) * D: (HQ + 2 * kv_heads) * D].unflatten(1, (kv_heads, D))
        self.dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dtable = torch.from_numpy(self.table).cuda()

    def cache(self, q2, **kw):
        return q2.PagedKV(self.dk, self.dv, self.dtable, self.H * self.G, **kw)

    def run(self, cache, **kw):
        if self.new:
            kw.update(new_k=self.dnk, new_v=self.dnv)
        return cache.attend(self.dq, self.dlens, scale=self.scale, **kw)

    def check(self, out):
        got = out.cpu().numpy().astype(np.float64)
        for b, n in enumerate(self.lens):
            k, v = (oatt.gather(p, self.table[b], n) for p in (self.k, self.v))
            if self.new and n:
                k[-1], v[-1] = self.nk[b], self.nv[b]
            ref, S, Q = oatt.attend_f64(self.q[b], k, v, self.scale)
            e = 2 * (self.D + 8) * 2.0 ** -23 * Q[:, None] + 2.0 ** -21 + 2.0 ** -19 + n / 16 * 2.0 ** -23
            tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2 * e * S
            err = np.abs(got[b] - ref)
            assert (err <= tol).all(), f"sequence {b} of {n} tokens: worst {(err / tol).max():.2f}x"

    def check_stored(self):
        """The cache holds the new rows where they belong, and everything else as before."""
        for pool, dev, new in ((self.k, self.dk, self.nk), (self.v, self.dv, self.nv)):
            want = pool.copy()
            for b, n in enumerate(self.lens):
                if self.new and n:
                    want[self.table[b, (n - 1) // self.page], (n - 1) % self.page] = new[b]
            assert np.array_equal(dev.cpu().numpy().view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 130, 777])
def test_one_sequence(q2, D, group, n):
    c = Case([n], 2, group, D, 16, 10 * n + group, new=n % 2 == 1)
    c.check(c.run(c.cache(q2)))
    c.check_stored()
    assert q2.device_errors() == 0


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 100, 256])
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("new", [False, True])
def test_ragged_batch_and_page_sizes(q2, page, order, new):
    c = Case([70, 0, 1, 333, 64, 0, 65, 128, 7, 0], 3, 4, 128, page, page, order, new, spare=3)
    out = c.run(c.cache(q2))
    c.check(out)
    c.check_stored()
    assert (out[1] == 0).all() and (out[5] == 0).all() and (out[9] == 0).all()
    assert q2.device_errors() == 0


@pytest.mark.parametrize("kv_heads,group,D", [(1, 16, 128), (2, 12, 64), (1, 64, 128), (1, 9, 256), (8, 5, 128), (8, 1, 64)])
def test_head_layouts(q2, kv_heads, group, D):
    c = Case([200, 31, 500], kv_heads, group, D, 32, group, new=True)
    c.check(c.run(c.cache(q2)))
    c.check_stored()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [9, 15, 16, 17, 32])
@pytest.mark.parametrize("lens,page", [([1, 17, 64], 16), ([4000, 700, 0, 33], 24)])
def test_many_query_heads_to_one(q2, D, group, lens, page):
    c = Case(lens, 2, group, D, page, group + D, new=True, peak=2.0)
    cache = c.cache(q2)
    out = c.run(cache)
    c.check(out)
    c.check_stored()
    assert torch.equal(out, c.run(cache)) and q2.device_errors() == 0


@pytest.mark.parametrize("lens", [[20000], [9000, 3, 5000], [3000] * 5])
def test_long_sequences_are_split_and_joined(q2, lens):
    c = Case(lens, 2, 4, 128, 64, len(lens), new=True)
    cache = c.cache(q2)
    out = c.run(cache)
    c.check(out)
    c.check_stored()
    for _ in range(5):                                  # the workspace is ready again, the result the same
        assert torch.equal(out, c.run(cache))


def test_large_batch(q2):
    lens = [(37 * b) % 90 for b in range(700)]
    c = Case(lens, 2, 2, 64, 16, 5, new=True)
    c.check(c.run(c.cache(q2)))
    c.check_stored()


def test_peaked_probabilities(q2):
    """Scores far apart, rising along the sequence: the maximum moves often."""
    c = Case([600, 90], 2, 4, 128, 16, 6)
    ramp = np.linspace(0.1, 12, 600)
    for b, n in enumerate(c.lens):
        for t in range(n):
            pg = c.table[b, t // 16]
            c.k[pg, t % 16] = (np.sign(c.q[b, ::4].astype(np.float64)) * ramp[t]).astype(np.float16)
    c.dk.copy_(torch.from_numpy(c.k))
    c.check(c.run(c.cache(q2)))


def test_heads_do_not_depend_on_the_batch_order(q2):
    """A sequence alone and in a batch: within the rounding of other splits."""
    c = Case([500, 40, 1000], 2, 4, 128, 16, 7)
    whole = c.run(c.cache(q2))
    for b in range(3):
        one = q2.PagedKV(c.dk, c.dv, c.dtable[b: b + 1], 8).attend(c.dq[b: b + 1], c.dlens[b: b + 1])
        assert torch.allclose(one[0].float(), whole[b].float(), rtol=2.0 ** -10, atol=1e-4)


def test_shared_pages(q2):
    """Two sequences with a common beginning, whose pages they share."""
    c = Case([100, 100], 2, 4, 64, 16, 8)
    c.table[1, :3] = c.table[0, :3]
    c.dtable.copy_(torch.from_numpy(c.table))
    c.check(c.run(c.cache(q2)))


def test_outside_pages_and_lengths_are_errors(q2):
    c = Case([100, 60, 30, 10], 2, 4, 128, 16, 9, new=True)
    P = c.k.shape[0]
    c.dtable[0, 2] = P                                  # no such page
    c.dtable[1, 3] = -1                                 # the page of the new token
    c.dlens[2] = c.table.shape[1] * 16 + 1              # more than its table row can hold
    out = c.run(c.cache(q2))
    torch.cuda.synchronize()
    assert q2.device_errors() == q2.ERR_LENGTH | q2.ERR_PAGE and q2.device_errors() == 0
    assert torch.isnan(out[:3]).all()
    keep = c.lens
    c.lens = [0, 0, 0, 10]
    c.check(torch.cat([torch.zeros_like(out[:3]), out[3:]]))
    c.lens = [100, 0, 0, 10]
    c.check_stored()                                    # the new token's own page of the first sequence is sound
    c.dlens[3] = -1
    assert torch.isnan(c.run(c.cache(q2))[3]).all() and q2.device_errors() & q2.ERR_LENGTH
    c.lens = keep


def test_stays_inside_its_buffers(q2):
    c = Case([33, 200], 2, 4, 128, 16, 11, new=True)
    probe = c.cache(q2)
    need = probe.ws.numel()
    ws = torch.full((256 + need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[256: 256 + need].zero_()
    buf = torch.full((512 + 2 * 1024 + 512,), 0x5A5A, dtype=torch.int16, device="cuda")
    out = buf[512: 512 + 2048].view(torch.float16).view(2, 8, 128)
    c.run(c.cache(q2, workspace=ws[256: 256 + need]), out=out)
    c.check(out)
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    assert (buf[:512] == 0x5A5A).all() and (buf[2560:] == 0x5A5A).all()
    with pytest.raises(q2.Q2Error):
        c.cache(q2, workspace=ws[:1024])


def test_one_workspace_for_several_shapes(q2):
    a, b = Case([5000], 2, 4, 128, 64, 12), Case([900, 20, 4000], 4, 2, 256, 16, 13, new=True)
    ws = torch.zeros(max(x.cache(q2).ws.numel() for x in (a, b)), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for x in (a, b):
            x.check(x.run(x.cache(q2, workspace=ws)))


def test_infinite_and_nan_inputs_show(q2):
    c = Case([50, 50, 50], 1, 4, 64, 16, 14)
    c.dk[int(c.table[0, 1]), 3, 0, 5] = float("nan")
    c.dv[int(c.table[1, 1]), 3, 0, 5] = float("inf")
    out = c.run(c.cache(q2)).cpu().numpy()
    assert np.isnan(out[0]).all() and not np.isfinite(out[1, :, 5]).any()
    assert np.isfinite(np.delete(out[1], 5, axis=1)).all() and np.isfinite(out[2]).all()


def test_no_sequences_and_another_stream(q2):
    c = Case([90, 17], 2, 4, 128, 16, 15, new=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache = c.cache(q2)
    torch.cuda.synchronize()
    out = c.run(cache, stream=side, out=torch.empty((2, 8, 128), dtype=torch.float16, device="cuda"))
    side.synchronize()
    c.check(out)
    empty = q2.PagedKV(c.dk, c.dv, c.dtable[:0], 8)
    assert empty.attend(c.dq[:0], c.dlens[:0]).shape == (0, 8, 128)


def test_binding_refuses_what_it_would_misread(q2):
    c = Case([20, 30], 2, 4, 128, 16, 16)
    cache = c.cache(q2)
    for q, lens, kw in ((c.dq.float(), c.dlens, {}), (c.dq[:, :4], c.dlens, {}), (c.dq, c.dlens.long(), {}),
                        (c.dq, c.dlens[:1], {}), (c.dq, c.dlens, dict(new_k=c.dnk)),
                        (c.dq, c.dlens, dict(new_k=c.dnk[:, :1], new_v=c.dnv)), (c.dq.cpu(), c.dlens, {}),
                        (c.dq, c.dlens, dict(scale=float("nan")))):
        with pytest.raises(q2.Q2Error):
            cache.attend(q, lens, **kw)
    for args in ((c.dk.float(), c.dv, c.dtable, 8), (c.dk, c.dv[:-1], c.dtable, 8), (c.dk, c.dv, c.dtable.long(), 8),
                 (c.dk, c.dv, c.dtable, 7), (c.dk[..., :96], c.dv[..., :96], c.dtable, 8), (c.dk, c.dv, c.dtable, 256)):
        with pytest.raises(q2.Q2Error):
            q2.PagedKV(*args)
