"""``q2_append``, ``q2_append4``, ``q2_read`` and ``q2_read4`` against the f64 oracle.

Keys: turned in 64 bits and rounded to fp32, then to fp16 or to 4 bits; the
kernel does the same to the last bit but where the exact value is within 2^-20
of a step of the middle of two fp32 numbers, which none of these inputs is.
Queries: two products in fp32, each off by at most 2^-24 of itself, one sum
(2^-24 of it, at most of the magnitudes) and one rounding to fp16 (2^-11 of the
value, or half of 2^-24): |err| <= 2^-11 |y| + 2^-25 + 3 * 2^-24 (|x c| + |o s|).
"""
import numpy as np
import pytest

from oracle import cache as oc

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _ordered(t, order):
    return t.transpose(1, 2).contiguous().transpose(1, 2) if order == "head" else t


class Case:
    """Sequences of `lens` tokens of which the last `counts` are new; the pools hold marks that must stay elsewhere."""

    def __init__(self, lens, counts, kv_heads=2, q_heads=6, D=128, bits=16, group=32, page=16, order="token", rot=None,
                 interleaved=False, bounds=False, seed=0, spare_rows=0, starts=True, positions=None, scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.counts, self.H, self.HQ, self.D, self.bits, self.group, self.page = lens, counts, kv_heads, q_heads, D, bits, group, page
        self.interleaved = interleaved
        B = len(lens)
        need = [-(-max(n, 0) // page) for n in lens]
        P = sum(need) + 2
        ids = rng.permutation(P).astype(np.int32)
        self.table = np.full((B, max(need + [1]) + 1), -7, dtype=np.int32)      # never to be used
        at = 0
        for b in range(B):
            self.table[b, : need[b]] = ids[at: at + need[b]]
            at += need[b]
        self.ntok = sum(counts) + spare_rows
        W = (q_heads + 2 * kv_heads) * D + 8
        self.wide = (rng.normal(size=(self.ntok, W)) * scale).astype(np.float16)
        cut = lambda a, n: self.wide[:, a * D: (a + n) * D].reshape(self.ntok, n, D)  # noqa: E731
        self.q, self.k, self.v = cut(0, q_heads), cut(q_heads, kv_heads), cut(q_heads + kv_heads, kv_heads)
        self.dwide = torch.from_numpy(self.wide).cuda()
        dcut = lambda a, n: self.dwide[:, a * D: (a + n) * D].unflatten(1, (n, D))  # noqa: E731
        self.dq, self.dk, self.dv = dcut(0, q_heads), dcut(q_heads, kv_heads), dcut(q_heads + kv_heads, kv_heads)
        rot = D if rot is None else rot
        self.angles = oc.angles_f32(rot, positions or max(lens + [1]))
        self.starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dstarts = torch.from_numpy(self.starts).cuda() if starts else None
        self.dtable = torch.from_numpy(self.table).cuda()
        shape = (P, page, kv_heads)
        if bits == 16:
            self.pools = {n: rng.integers(0, 1 << 15, size=shape + (D,)).astype(np.uint16).view(np.float16) for n in "kv"}
        else:
            self.pools = {}
            for n in ("k", "v"):
                self.pools[n] = rng.integers(0, 256, size=shape + (D // 2,)).astype(np.uint8)
                self.pools[n + "s"] = rng.normal(size=shape + (D // group, 2)).astype(np.float16)
        self.dev = {n: _ordered(torch.from_numpy(p).cuda(), order) for n, p in self.pools.items()}
        self.bounds = self.dbounds = None
        if bounds:
            self.bounds = np.sort(rng.normal(size=(P, -(-page // 64), kv_heads, 2, D)), axis=3).astype(np.float16)
            self.dbounds = torch.from_numpy(self.bounds).cuda()

    def cache(self, q2):
        d = self.dev
        if self.bits == 16:
            return q2.PagedKV(d["k"], d["v"], self.dtable, self.HQ, bounds=self.dbounds)
        return q2.PagedKV4(d["k"], d["ks"], d["v"], d["vs"], self.dtable, self.HQ, bounds=self.dbounds)

    def rope(self, q2):
        return q2.Rope(torch.from_numpy(self.angles).cuda(), self.interleaved)

    def run(self, q2, rope=True, cache=None, **kw):
        kw = {"q": self.dq, "q_out": torch.full((self.ntok, self.HQ, self.D), 7.0, dtype=torch.float16, device="cuda"), **kw}
        return (cache or self.cache(q2)).append(self.dk, self.dv, self.dlens, starts=self.dstarts,
                                                rope=self.rope(q2) if rope is True else rope, **kw)

    def turned(self, b, x):
        """(y, magnitudes) of the new rows of sequence b of x [ntok][heads][D]."""
        r = slice(self.starts[b], self.starts[b + 1])
        pos = np.arange(self.lens[b] - self.counts[b], self.lens[b])
        return oc.turn_f64(x[r], self.angles[pos], self.interleaved)

    def expect(self, keys=None, skip=()):
        """The pools and bounds afterwards."""
        want = {n: p.copy() for n, p in self.pools.items()}
        kept = None if self.bounds is None else self.bounds.copy()
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            if b in skip or not c:
                continue
            k = self.turned(b, self.k)[0] if keys is None else keys[b]
            k32 = k.astype(np.float32)
            v32 = self.v[self.starts[b]: self.starts[b + 1]].astype(np.float32)
            pos = np.arange(n - c, n)
            at = self.table[b, pos // self.page], pos % self.page
            if self.bits == 16:
                want["k"][at], want["v"][at] = k32.astype(np.float16), v32.astype(np.float16)
            else:
                for name, x in (("k", k32), ("v", v32)):
                    codes, pairs = oc.quantise(x, self.group)
                    want[name][at], want[name + "s"][at] = oc.pack(codes), pairs
            if kept is not None:
                for blk in range((n - c) // 64, (n - 1) // 64 + 1):
                    rows = k32.astype(np.float16)[(pos // 64) == blk]
                    low, high = rows.min(0), rows.max(0)
                    place = self.table[b, blk * 64 // self.page], blk * 64 % self.page // 64
                    if blk * 64 < n - c:
                        low, high = np.minimum(low, kept[place][:, 0]), np.maximum(high, kept[place][:, 1])
                    kept[place] = np.stack([low, high], axis=1)
        return want, kept

    def check_pools(self, **kw):
        want, kept = self.expect(**kw)
        for n, p in want.items():
            got = np.ascontiguousarray(self.dev[n].cpu().numpy())
            off = int((got.view(np.uint8) != p.view(np.uint8)).sum())           # bits
            assert off == 0, f"{n}: {off} of {p.nbytes} bytes differ"
        if kept is not None:
            off = int((self.dbounds.cpu().numpy() != kept).sum())
            assert off == 0, f"{off} bounds differ"

    def check_q(self, out):
        got = out.cpu().numpy()
        for b, c in enumerate(self.counts):
            r = slice(self.starts[b], self.starts[b + 1])
            y, mag = self.turned(b, self.q)
            tol = 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 3 * 2.0 ** -24 * mag
            assert (np.abs(got[r].astype(np.float64) - y) <= tol).all()
        assert (got[self.starts[-1]:] == 7).all()                               # rows behind the last sequence


FORMS = [(16, 32), (4, 32), (4, 64)]


@pytest.mark.parametrize("bits,group", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bounds", [False, True])
def test_one_token_each(q2, bits, group, D, interleaved, bounds):
    lens = [1, 2, 16, 17, 64, 65, 100, 129, 640]
    c = Case(lens, [1] * 9, D=D, bits=bits, group=group, interleaved=interleaved, bounds=bounds, seed=D + group, starts=False)
    c.check_q(c.run(q2))
    c.check_pools()
    assert q2.device_errors() == 0


@pytest.mark.parametrize("bits,group", FORMS)
@pytest.mark.parametrize("page,order,bounds", [(16, "token", True), (64, "head", True), (256, "token", True), (1, "head", True),
                                               (24, "token", False), (100, "head", False)])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (16, False), (80, False)])
def test_ragged_prompts(q2, bits, group, page, order, bounds, rot, interleaved):
    lens, counts = [300, 64, 7, 65, 200, 129, 1, 0, 66], [300, 64, 3, 1, 0, 70, 1, 0, 3]
    c = Case(lens, counts, bits=bits, group=group, page=page, order=order, bounds=bounds, rot=rot, interleaved=interleaved,
             seed=page + rot, spare_rows=5)
    c.check_q(c.run(q2))
    c.check_pools()
    assert q2.device_errors() == 0


@pytest.mark.parametrize("D,kv_heads,q_heads", [(64, 1, 1), (128, 8, 32), (256, 3, 48), (64, 8, 40), (128, 1, 61)])
@pytest.mark.parametrize("bits,group", FORMS[:2])
def test_head_layouts(q2, D, kv_heads, q_heads, bits, group):
    c = Case([130, 40], [130, 1], kv_heads, q_heads, D, bits, group, page=64, bounds=True, rot=D // 2, seed=D + kv_heads)
    c.check_q(c.run(q2))
    c.check_pools()


@pytest.mark.parametrize("bits,group", FORMS[:2])
def test_many_sequences_of_few_tokens(q2, bits, group):
    counts = [(5 * b) % 4 for b in range(1024)]
    lens = [n + (13 * b) % 70 for b, n in enumerate(counts)]
    c = Case(lens, counts, 1, 2, 64, bits, group, page=32, bounds=True, seed=3)
    c.check_q(c.run(q2))
    c.check_pools()


@pytest.mark.parametrize("bits,group", FORMS)
def test_pieces_give_what_a_whole_prompt_gives(q2, bits, group):
    """A prompt in pieces of odd lengths; the bounds come out as those of all its keys."""
    c = Case([333], [333], bits=bits, group=group, page=64, order="head", bounds=True, seed=4)
    cache, rope, at = c.cache(q2), c.rope(q2), 0
    for n in (1, 62, 1, 1, 100, 27, 64, 77):
        lens = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        cache.append(c.dk[at: at + n], c.dv[at: at + n], lens, starts=starts, rope=rope)
        at += n
    assert at == 333
    c.check_pools()
    keys = c.turned(0, c.k)[0].astype(np.float32).astype(np.float16)
    for i, want in enumerate(oc.bounds(keys)):
        assert np.array_equal(c.dbounds[int(c.table[0, i]), 0].cpu().numpy(), want)


@pytest.mark.parametrize("bits,group", FORMS)
def test_read_gives_back_what_the_rows_stand_for(q2, bits, group):
    lens = [70, 0, 1, 333, 64]
    c = Case(lens, lens, bits=bits, group=group, page=24, seed=5, spare_rows=3)
    cache = c.cache(q2)
    c.run(q2, cache=cache)
    wide = torch.full((c.ntok, c.H * c.D + 16), 7.0, dtype=torch.float16, device="cuda")
    k, v = wide[:, : c.H * c.D].unflatten(1, (c.H, c.D)), torch.full((c.ntok, c.H, c.D), 7.0, dtype=torch.float16, device="cuda")
    assert cache.read(c.dlens, starts=c.dstarts, k_out=k, v_out=v) == (k, v)
    want, _ = c.expect()
    for got, name in ((k.cpu().numpy(), "k"), (v.cpu().numpy(), "v")):
        for b, n in enumerate(lens):
            pos = np.arange(n)
            at = c.table[b, pos // c.page], pos % c.page
            ref = want[name][at] if bits == 16 else oc.value_f64(want[name][at], want[name + "s"][at]).astype(np.float32).astype(np.float16)
            assert np.array_equal(got[c.starts[b]: c.starts[b + 1]], ref)
        assert (got[c.starts[-1]:] == 7).all()
    assert (wide[:, c.H * c.D:] == 7).all()
    one, none = cache.read(c.dlens, starts=c.dstarts, k_out=v.clone())
    assert none is None and torch.equal(one, k)
    last = cache.read(c.dlens)                                                  # the last token of each; zeros for none
    for b, n in enumerate(lens):
        want_k = k[c.starts[b] + n - 1] if n else torch.zeros_like(k[0])
        assert torch.equal(last[0][b], want_k)
    assert torch.equal(cache.read(c.dlens, starts=c.dstarts, ntok=c.ntok)[1][: sum(lens)], v[: sum(lens)])
    assert q2.device_errors() == 0


def test_values_far_apart_equal_and_infinite(q2):
    """Groups of one value, of tiny and of the largest ones, with an infinity, with a NaN, and an offset beyond fp16."""
    c = Case([90], [90], 1, 1, 128, 4, 32, page=32, bounds=False, seed=6, scale=1.0)
    v, k = c.v.copy(), c.k.copy()
    v[0, 0, :32], v[1, 0, :32] = 3.0, 0.0
    v[2, 0, :32] *= np.float16(2.0 ** -20)
    v[3, 0, :2] = [65504, -65504]
    v[4, 0, 5], v[5, 0, 40], v[6, 0, 127] = np.inf, -np.inf, np.nan
    v[7, 0, :32] = np.float16(2.0 ** -24) * (np.arange(32) % 3)
    k[8] = -60000                                                               # turned: down to -84852
    c.dwide[:, 2 * 128: 3 * 128] = torch.from_numpy(v[:, 0]).cuda()
    c.dwide[:, 128: 256] = torch.from_numpy(k[:, 0]).cuda()
    c.k, c.v = k, v
    c.run(q2)
    c.check_pools()
    cache = c.cache(q2)
    got = cache.read(c.dlens, starts=c.dstarts, ntok=90)[1].cpu().numpy()
    assert np.isnan(got[4, 0, :32]).all() and np.isnan(got[5, 0, 32:64]).all() and np.isnan(got[6, 0, 96:]).all()
    assert np.isfinite(got[4, 0, 32:]).all() and (got[0, 0, :32] == 3).all()


def test_nan_keys_show_in_the_bounds(q2):
    c = Case([70], [70], 2, 2, 64, 16, page=64, bounds=True, seed=7, rot=32)
    c.dk[3, 1, 50] = float("nan")
    c.run(q2)
    lo_hi = c.dbounds[int(c.table[0, 0]), 0, 1]
    assert torch.isnan(lo_hi[:, 50]).all() and not torch.isnan(lo_hi[:, :50]).any() and not torch.isnan(lo_hi[:, 51:]).any()


@pytest.mark.parametrize("bits,group", FORMS[:2])
def test_in_place_without_queries_and_without_angles(q2, bits, group):
    c = Case([100, 20], [50, 20], bits=bits, group=group, seed=8)
    want = c.run(q2)
    got = c.dwide.clone()
    q = got[:, : c.HQ * c.D].unflatten(1, (c.HQ, c.D))
    assert c.run(q2, q=q, q_out=None) is q and torch.equal(q, want)
    assert torch.equal(got[:, c.HQ * c.D:], c.dwide[:, c.HQ * c.D:])
    c.check_pools()
    assert c.run(q2, q=None, q_out=None) is None
    c.check_pools()
    out = c.run(q2, rope=None)
    assert torch.equal(out, c.dq)                                               # a copy
    c.check_pools(keys=[c.k[c.starts[b]: c.starts[b + 1]] for b in range(2)])


@pytest.mark.parametrize("bits,group", FORMS[:2])
@pytest.mark.parametrize("starts", [False, True])
def test_a_padded_batch_leaves_its_rows(q2, bits, group, starts):
    lens = [5, 0, 70, 0]
    c = Case(lens, [1] * 4, bits=bits, group=group, seed=9, starts=starts)
    out = c.run(q2)
    assert (out[1] == 7).all() and (out[3] == 7).all()
    c.check_pools(skip=(1, 3))
    c.lens, c.counts = [5, 70], [1, 1]
    assert q2.device_errors() == 0


@pytest.mark.parametrize("bits,group", FORMS[:2])
def test_wrong_lengths_and_pages_are_errors(q2, bits, group):
    counts = [3, 70, 1, 2, 4]
    c = Case([40, 70, 33, 20, 30], counts, bits=bits, group=group, page=16, bounds=True, seed=10, positions=80)
    cap = c.table.shape[1] * 16
    for wrong in (cap + 1, -1, 2, 90):                                         # too long, negative, fewer than its rows, beyond the angles
        c.dlens[1] = wrong
        out = c.run(q2)
        assert q2.device_errors() == q2.ERR_LENGTH and torch.isnan(out[3: 73]).all() and not torch.isnan(out[:3]).any()
        c.check_pools(skip=(1,))
        if wrong != 90:                                                        # (reading needs no angles)
            k, _ = c.cache(q2).read(c.dlens, starts=c.dstarts, ntok=c.ntok)
            assert q2.device_errors() == q2.ERR_LENGTH and torch.isnan(k[3: 73]).all() and not torch.isnan(k[:3]).any()
    c.dlens[1] = 70
    c.dtable[1, 2], c.dtable[4, 0] = c.pools["k"].shape[0], -1                  # tokens 32..47 of sequence 1; none of those of sequence 4
    c.run(q2)
    assert q2.device_errors() == q2.ERR_PAGE
    k, _ = c.cache(q2).read(c.dlens, starts=c.dstarts, ntok=c.ntok)
    assert q2.device_errors() == q2.ERR_PAGE
    bad = torch.isnan(k.flatten(1)).all(1)
    assert bad[3 + 32: 3 + 48].all() and int(bad.sum()) == 16


@pytest.mark.parametrize("starts", [[0, 5, 3, 12], [-1, 4, 8, 12], [0, 4, 8, 13], [2, 2, 2, 2]])
def test_wrong_starts_are_errors(q2, starts):
    """Nothing of a sequence whose starts do not ascend within the rows; the others as they should be."""
    c = Case([20, 30, 40], [4, 4, 4], bits=16, seed=11)
    c.dstarts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    before = {n: t.clone() for n, t in c.dev.items()}
    out = c.run(q2)
    ok = [0 <= a <= b <= 12 for a, b in zip(starts, starts[1:])]
    assert q2.device_errors() == (0 if all(ok) else q2.ERR_LENGTH)
    written = (out != 7).flatten(1).any(1).cpu().tolist()
    want = [False] * 12
    for a, b, good in zip(starts, starts[1:], ok):
        for r in range(a, b) if good else ():
            want[r] = True
    assert written == want
    if not any(want):
        assert all(torch.equal(t.view(torch.int16), before[n].view(torch.int16)) for n, t in c.dev.items())


@pytest.mark.parametrize("bits,group", FORMS)
def test_captured_and_on_another_stream(q2, bits, group):
    c = Case([100, 64, 10], [1, 1, 1], bits=bits, group=group, page=64, bounds=True, seed=12, starts=False)
    cache, rope = c.cache(q2), c.rope(q2)
    out = torch.empty((3, c.HQ, c.D), dtype=torch.float16, device="cuda")
    keep = {n: t.clone() for n, t in c.dev.items()}
    kept = c.dbounds.clone()
    c.run(q2, cache=cache, rope=rope, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(q2, cache=cache, rope=rope, q_out=out)
    for _ in range(2):
        for n, t in c.dev.items():
            t.copy_(keep[n])
        c.dbounds.copy_(kept)
        out.fill_(7)
        graph.replay()
        c.check_q(out)
        c.check_pools()
    side = torch.cuda.Stream()
    for n, t in c.dev.items():
        t.copy_(keep[n])
    c.dbounds.copy_(kept)
    torch.cuda.synchronize()
    c.run(q2, cache=cache, rope=rope, q_out=out, stream=side)
    side.synchronize()
    c.check_q(out)
    c.check_pools()


def test_far_positions_and_offsets(q2):
    """Token 3 000 000 of a sequence: its angles, and a place 2^31 bytes into the pool."""
    n, page = 3_000_000, 64
    pages = n // page
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    k, v = (torch.zeros((pages, page, 3, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    rope = q2.Rope.of(128, n)
    x = torch.from_numpy(np.random.default_rng(13).normal(size=(3, 1, 3, 128)).astype(np.float16)).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cache = q2.PagedKV(k, v, table, 3)
    q = cache.append(x[0], x[1], lens, q=x[2].clone(), rope=rope)
    ang = np.stack([f((n - 1) * 10000.0 ** (-np.arange(64) / 64.0)) for f in (np.cos, np.sin)], axis=-1)[None]
    want = oc.turn_f64(x[0].cpu().numpy(), ang, False)[0]
    assert np.abs(k[-1, -1].cpu().numpy() - want[0]).max() < 2.0 ** -9 and torch.equal(v[-1, -1], x[1, 0])
    assert np.abs(q.cpu().numpy() - oc.turn_f64(x[2].cpu().numpy(), ang, False)[0]).max() < 2.0 ** -9
    assert (k.view(torch.int16)[:-1] == 0).all() and torch.equal(cache.read(lens)[0][0], k[-1, -1])


def test_binding_refuses_what_it_would_misread(q2):
    c = Case([20, 30], [1, 1], bits=4, page=16, seed=14, starts=False)
    cache, rope = c.cache(q2), c.rope(q2)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ok = dict(k=c.dk, v=c.dv, lens=c.dlens, q=c.dq, rope=rope)
    for kw in (dict(k=c.dk.float()), dict(v=c.dv[:1]), dict(k=c.dk[:, :1]), dict(lens=c.dlens.long()), dict(lens=c.dlens[:1]),
               dict(starts=starts[:2]), dict(starts=starts.long()), dict(q=c.dq[:, :4]), dict(q=c.dq.cpu()), dict(q_out=c.dq[:1]),
               dict(q=None, q_out=c.dq), dict(k=c.dk[:1], v=c.dv[:1]), dict(k=c.dk.transpose(1, 2)), dict(starts=starts.cpu())):
        with pytest.raises(q2.Q2Error):
            cache.append(**{**ok, **kw})
    d = c.dev
    args = (d["k"], d["ks"], d["v"], d["vs"], c.dtable, c.HQ)
    for i, bad in ((0, d["k"].half()), (1, d["ks"].float()), (2, d["v"][:-1]), (1, d["ks"][:, :, :, :3]), (0, d["k"][..., :24]),
                   (4, c.dtable.long()), (3, d["vs"].transpose(1, 2).contiguous().transpose(1, 2)), (5, 7)):
        with pytest.raises(q2.Q2Error):
            q2.PagedKV4(*args[:i], bad, *args[i + 1:])
    shape = (c.table.shape[0], 1, c.H, 2, c.D)
    for bad in (torch.zeros(shape, device="cuda"), torch.zeros((1,) + shape[1:], dtype=torch.float16, device="cuda")):
        with pytest.raises(q2.Q2Error):
            q2.PagedKV4(*args, bounds=bad)
    for bad in (rope.table[0], rope.table.double(), rope.table[:, ::2], rope.table.cpu()):
        with pytest.raises(q2.Q2Error):
            q2.Rope(bad)
    with pytest.raises(q2.Q2Error):                                             # 24 columns
        cache.append(**{**ok, "rope": q2.Rope(rope.table[:, :12].contiguous())})
    with pytest.raises(q2.Q2Error):
        cache.read(c.dlens, starts=starts)
    with pytest.raises(q2.Q2Error):
        cache.read(c.dlens, k_out=c.dk[:1])


@pytest.mark.parametrize("bits,group", FORMS)
@pytest.mark.parametrize("bounds", [False, True])
def test_a_prompt_among_sequences_of_few_tokens(q2, bits, group, bounds):
    """Tiles of 8 to 64 positions: what one call stores does not depend on how many tokens the others have."""
    for counts in ([1] * 20 + [70] + [2] * 9, [3, 4, 5, 150, 2, 1], [9] * 12, [0, 1, 17, 0, 33, 2]):
        lens = [n + 13 * (b % 5) if n else 0 for b, n in enumerate(counts)]
        c = Case(lens, counts, bits=bits, group=group, page=32, rot=64, bounds=bounds, seed=len(counts))
        c.check_q(c.run(q2))
        c.check_pools()
    assert q2.device_errors() == 0


@pytest.mark.parametrize("bits,group", FORMS[:2])
def test_sequences_beside_one_with_wrong_starts_are_stored(q2, bits, group):
    """Starts that descend behind sequence 1: nothing of it is stored, all of the others is, and the rows that one sequence
    alone claims are turned (sequence 0 has rows 0..8, 2 has 8..10, 3 has 11)."""
    c = Case([20, 30, 40, 10], [4, 4, 3, 1], bits=bits, group=group, bounds=True, seed=15)
    c.dstarts[1:3] = torch.tensor([9, 8], dtype=torch.int32, device="cuda")
    c.counts, c.starts = [9, 0, 3, 1], np.array([0, 9, 8, 11, 12])
    out = c.run(q2).cpu().numpy()
    assert q2.device_errors() == q2.ERR_LENGTH
    c.check_pools()
    for b, rows in ((0, range(0, 8)), (2, range(9, 11)), (3, range(11, 12))):
        y, mag = c.turned(b, c.q)
        for r in rows:
            i = r - c.starts[b]
            assert (np.abs(out[r] - y[i]) <= 2.0 ** -11 * np.abs(y[i]) + 2.0 ** -25 + 3 * 2.0 ** -24 * mag[i]).all()


@pytest.mark.parametrize("bits,group", FORMS)
@pytest.mark.parametrize("starts", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_queries_beside_padding_are_turned(q2, bits, group, starts, interleaved):
    c = Case([5, 0, 70, 0, 64], [1] * 5, bits=bits, group=group, seed=16, starts=starts, interleaved=interleaved)
    out = c.run(q2).cpu().numpy()
    for b in (0, 2, 4):
        y, mag = c.turned(b, c.q)
        assert (np.abs(out[b] - y[0]) <= 2.0 ** -11 * np.abs(y[0]) + 2.0 ** -25 + 3 * 2.0 ** -24 * mag[0]).all()
    assert (out[[1, 3]] == 7).all()
    c.check_pools(skip=(1, 3))


@pytest.mark.parametrize("bits,group", FORMS[:2])
@pytest.mark.parametrize("starts", [False, True])
def test_bounds_without_a_page_are_an_error(q2, bits, group, starts):
    """The tokens' own page is there, that of their block's first token is not: the tokens are stored, the bounds cannot be."""
    c = Case([40, 90], [1, 1], bits=bits, group=group, page=16, bounds=True, seed=17, starts=starts)
    c.dtable[0, 0] = -1
    kept = c.bounds.copy()
    c.check_q(c.run(q2))
    assert q2.device_errors() == q2.ERR_PAGE
    want, all_kept = c.expect()
    at = c.table[1, 4], 0                                                      # block 1 of sequence 1 has its bounds
    kept[at] = all_kept[at]
    assert np.array_equal(c.dbounds.cpu().numpy(), kept)
    c.bounds = None
    c.check_pools()
