"""``q2_attend4`` and ``q2_attend_blocks`` against the f64 oracle.

A score of the 4-bit cache is a sum over groups of s sum(q c) + m sum(q).  The
tensor cores take codes as numbers below fp16's normal ones, which they align as
if they were 2^-14: a product is cut off at most 2^-23 2^-14 max|q| below, where
a code's unit is 2^-24 (columns 0 and 2 of four, q over 1 and 4) or, of columns 1
and 3, 2^-20 with q over 16 and 64: 2^-13 or 2^-17 max|q| of a code each, 16 of
them per instruction, and one instruction of each kind per 32 columns: (2^-9 +
2^-13) s max|q| per 32 columns.  q over 64 is exact but below 2^-24 of the
largest 2^10: another 2^-28.  The sums in fp32 add at most (D + 8) 2^-23 of the
magnitudes M = sum |q| (s c + |m|).  So a scaled score is off by d = scale (sum
over 32 columns 2^-8 s max|q| + (D + 8) 2^-23 M), and a
probability, with exp2 and the joins, by e = 2 d + 2^-20 + 2^-19 relative.
The numerators add terms of p s = hi + lo (2^-22) times c - 8, exact, and of p (m
+ 8 s), one step of at most 2^-23 of the sum of magnitudes N = sum p (8 s + |m +
8 s|) per 16 tokens.  Together
|o - ref| <= 2^-11 |ref| + 2^-25 + 2 (e + n / 16 2^-23) N / sum p.
(The fp16 cache's tolerance is that of ``test_gpu_attend.py``.)
"""
import numpy as np
import pytest

from oracle import attend as oatt, cache as oc

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
    """A cache whose unused places hold NaN (offsets) or marks, queries inside a wider buffer."""

    def __init__(self, lens, kv_heads, q_group, D, group=32, page=16, seed=0, order="token", bits=4, spare=0, peak=1.0, shift=0.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.G, self.D, self.group, self.page, self.bits = lens, kv_heads, q_group, D, group, page, bits
        B, HQ = len(lens), kv_heads * q_group
        need = [-(-max(n, 0) // page) for n in lens]
        P = sum(need) + 2
        ids = rng.permutation(P)
        self.table = np.full((B, max(need + [1]) + spare), -7, dtype=np.int32)      # never to be used
        at = 0
        for b in range(B):
            self.table[b, : need[b]] = ids[at: at + need[b]]
            at += need[b]
        shape = (P, page, kv_heads)
        names = ("k", "v") if bits == 16 else ("k", "v", "ks", "vs")
        tail = {"k": D if bits == 16 else D // 2, "v": D if bits == 16 else D // 2}
        self.pool = {n: np.full(shape + ((tail[n],) if n in tail else (D // group, 2)), np.nan if bits == 16 or n not in tail else 0xA5,
                                dtype=np.float16 if bits == 16 or n not in tail else np.uint8) for n in names}
        for b, n in enumerate(lens):
            for t in range(max(n, 0)):
                pg, sl = self.table[b, t // page], t % page
                if bits == 16:
                    self.pool["k"][pg, sl], self.pool["v"][pg, sl] = rng.normal(size=(2, kv_heads, D)) * peak
                    continue
                for name in ("k", "v"):
                    self.pool[name][pg, sl] = rng.integers(0, 256, size=(kv_heads, D // 2))
                    s = rng.uniform(0.02, 0.4, size=(kv_heads, D // group)) * peak
                    self.pool[name + "s"][pg, sl] = np.stack([s, rng.normal(size=s.shape) * 0.3 - 7.5 * s + shift], axis=-1)
        self.wide = rng.normal(size=(B, HQ * D + 8)).astype(np.float16)
        self.q = self.wide[:, : HQ * D].reshape(B, HQ, D)
        self.scale = D ** -0.5
        ordered = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2) if order == "head" else t  # noqa: E731
        self.dev = {n: ordered(torch.from_numpy(p).cuda()) for n, p in self.pool.items()}
        self.dwide = torch.from_numpy(self.wide).cuda()
        self.dq = self.dwide[:, : HQ * D].unflatten(1, (HQ, D))
        self.dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dtable = torch.from_numpy(self.table).cuda()

    def cache(self, q2, **kw):
        d = self.dev
        if self.bits == 16:
            return q2.PagedKV(d["k"], d["v"], self.dtable, self.H * self.G, **kw)
        return q2.PagedKV4(d["k"], d["ks"], d["v"], d["vs"], self.dtable, self.H * self.G, **kw)

    def run(self, cache, **kw):
        return cache.attend(self.dq, self.dlens, scale=self.scale, **kw)

    def rows(self, name, b, tokens, h):
        """(values, magnitudes, steps per column) of one head's rows, f64 [n][D]."""
        at = self.table[b, tokens // self.page], tokens % self.page, h
        if self.bits == 16:
            x = self.pool[name][at].astype(np.float64)
            return x, np.abs(x), np.zeros_like(x)
        codes, pairs = self.pool[name][at], self.pool[name + "s"][at].astype(np.float64)
        x = oc.value_f64(codes, pairs)
        p = np.repeat(pairs, self.group, axis=-2)
        if name == "v":
            return x, 8 * p[..., 0] + np.abs(p[..., 1] + 8 * p[..., 0]), p[..., 0]
        return x, (x - p[..., 1]) + np.abs(p[..., 1]), p[..., 0]

    def check(self, out, sel=None):
        got = out.cpu().numpy().astype(np.float64)
        for b, n in enumerate(self.lens):
            for h in range(self.H):
                tokens = np.arange(n)
                if sel is not None:
                    blocks = [i for i in sel[b][h][: -(-n // 64)] if 0 <= i < -(-n // 64)]
                    tokens = np.concatenate([np.arange(64 * i, min(64 * i + 64, n)) for i in blocks] + [np.zeros(0, dtype=int)]).astype(int)
                mine = got[b, h * self.G: (h + 1) * self.G]
                if not len(tokens):
                    assert (mine == 0).all()
                    continue
                q = self.q[b, h * self.G: (h + 1) * self.G].astype(np.float64)
                k, kmag, ks = self.rows("k", b, tokens, h)
                v, vmag, _ = self.rows("v", b, tokens, h)
                s = self.scale * (q @ k.T)
                p = np.exp(s - s.max(1, keepdims=True))
                ref, l = p @ v / p.sum(1, keepdims=True), p.sum(1, keepdims=True)
                M = (np.abs(q) @ kmag.T).max(1)
                size = abs(self.scale)                  # a score's error is |scale| times that of its product q.k
                if self.bits == 16:
                    e = 2 * (self.D + 8) * 2.0 ** -23 * size * M + 2.0 ** -21 + 2.0 ** -19
                else:
                    per = np.abs(q).reshape(self.G, -1, 32).max(2) @ ks[:, ::32].T            # [G][n]
                    d = size * (2.0 ** -8 * per.max(1) + (self.D + 8) * 2.0 ** -23 * M)
                    e = 2 * d + 2.0 ** -20 + 2.0 ** -19
                N = p @ vmag / l
                tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2 * (e[:, None] + len(tokens) / 16 * 2.0 ** -23) * N
                err = np.abs(mine - ref)
                assert (err <= tol).all(), f"sequence {b} of {n} tokens, head {h}: worst {(err / tol).max():.2f}x"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("q_group", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 130, 777])
def test_one_sequence(q2, D, group, q_group, n):
    c = Case([n], 2, q_group, D, group, 16, 10 * n + q_group)
    c.check(c.run(c.cache(q2)))
    assert q2.device_errors() == 0


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 100, 256])
@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("D,group", [(128, 64), (128, 32), (64, 64), (256, 32)])
def test_ragged_batch_and_page_sizes(q2, page, order, D, group):
    c = Case([70, 0, 1, 333, 64, 0, 65, 128, 7, 0], 3, 4, D, group, page, page, order, spare=3)
    out = c.run(c.cache(q2))
    c.check(out)
    assert (out[1] == 0).all() and (out[5] == 0).all() and (out[9] == 0).all()
    assert q2.device_errors() == 0


@pytest.mark.parametrize("kv_heads,q_group,D", [(1, 16, 128), (2, 12, 64), (1, 64, 128), (1, 9, 256), (8, 5, 128), (8, 1, 64), (2, 17, 128)])
@pytest.mark.parametrize("group", [32, 64])
def test_head_layouts(q2, kv_heads, q_group, D, group):
    c = Case([200, 31, 500], kv_heads, q_group, D, group, 32, q_group)
    cache = c.cache(q2)
    out = c.run(cache)
    c.check(out)
    assert torch.equal(out, c.run(cache)) and q2.device_errors() == 0


@pytest.mark.parametrize("lens", [[20000], [9000, 3, 5000], [3000] * 5])
def test_long_sequences_are_split_and_joined(q2, lens):
    c = Case(lens, 2, 4, 128, 64, 64, len(lens), "head")
    cache = c.cache(q2)
    out = c.run(cache)
    c.check(out)
    for _ in range(5):                                  # the workspace is ready again, the result the same
        assert torch.equal(out, c.run(cache))


def test_large_batch(q2):
    c = Case([(37 * b) % 90 for b in range(700)], 2, 2, 64, 64, 16, 5)
    c.check(c.run(c.cache(q2)))


@pytest.mark.parametrize("D,group,q_group", [(128, 64, 4), (128, 32, 5), (64, 64, 12), (256, 32, 8)])
@pytest.mark.parametrize("large", [16.0, 100.0, 4000.0])
def test_queries_with_a_large_column(q2, D, group, q_group, large):
    """A score's error goes by the head's largest column, not by the terms: the bound of above holds, and the outputs are
    where an fp32 sum's would be, since a column that large decides the score."""
    c = Case([700, 64, 9], 2, q_group, D, group, 16, 30 + q_group)
    c.q[..., 5] *= np.float16(large)
    c.dwide[:, : c.q[0].size] = torch.from_numpy(c.q.reshape(3, -1)).cuda()
    c.check(c.run(c.cache(q2)))


@pytest.mark.parametrize("shift", [0.0, 100.0])
def test_peaked_probabilities_and_offsets_far_from_zero(q2, shift):
    c = Case([600, 90], 2, 4, 128, 32, 16, 6, peak=3.0, shift=shift)
    c.check(c.run(c.cache(q2)))


def test_steps_that_grow_along_the_sequence(q2):
    """The scale of the probabilities follows the largest step, over the range of fp16; the least steps come last again."""
    c = Case([640], 1, 4, 128, 64, 16, 7)
    grow = np.concatenate([2.0 ** np.linspace(-24, 4, 320), 2.0 ** np.linspace(4, -24, 320)])
    for t in range(640):
        at = c.table[0, t // 16], t % 16
        c.pool["vs"][at][..., 0] = grow[t]
        c.pool["vs"][at][..., 1] = -7.5 * grow[t]
    c.dev["vs"].copy_(torch.from_numpy(c.pool["vs"]))
    c.check(c.run(c.cache(q2)))


def test_small_probabilities_behind_a_large_one(q2):
    """A token far above the rest whose value is near zero: the output is made of the small ones."""
    n = 2000
    c = Case([n], 1, 4, 128, 64, 16, 8)
    c.pool["k"][:] = 0x77
    c.pool["ks"][..., 0], c.pool["ks"][..., 1] = 0.01, -0.07            # zero keys ..
    at = c.table[0, 0], 0
    c.q[0, :] = c.q[0, :1]
    c.dwide[:, : 4 * 128] = torch.from_numpy(c.q.reshape(1, -1)).cuda()
    x = c.q[0, 0].astype(np.float64)
    k = 15 * np.sqrt(128.0) * x / (x @ x)                               # .. but the first: a score of 15
    codes, pairs = oc.quantise(k.astype(np.float32), 64)
    c.pool["k"][at], c.pool["ks"][at] = oc.pack(codes), pairs
    c.pool["vs"][at] = [2.0 ** -20, -2.0 ** -17]
    for name, p in c.pool.items():
        c.dev[name].copy_(torch.from_numpy(p))
    c.check(c.run(c.cache(q2)))


def test_shared_pages(q2):
    c = Case([100, 100], 2, 4, 64, 32, 16, 9)
    c.table[1, :3] = c.table[0, :3]
    c.dtable.copy_(torch.from_numpy(c.table))
    c.check(c.run(c.cache(q2)))


def test_outside_pages_and_lengths_are_errors(q2):
    c = Case([100, 60, 30, 10], 2, 4, 128, 64, 16, 10)
    c.dtable[0, 2] = c.pool["k"].shape[0]               # no such page
    c.dtable[1, 3] = -1
    c.dlens[2] = c.table.shape[1] * 16 + 1              # more than its table row can hold
    out = c.run(c.cache(q2))
    torch.cuda.synchronize()
    assert q2.device_errors() == q2.ERR_LENGTH | q2.ERR_PAGE and q2.device_errors() == 0
    assert torch.isnan(out[:3]).all()
    c.lens = [0, 0, 0, 10]
    c.check(torch.cat([torch.zeros_like(out[:3]), out[3:]]))
    c.dlens[3] = -1
    assert torch.isnan(c.run(c.cache(q2))[3]).all() and q2.device_errors() & q2.ERR_LENGTH


def test_nan_groups_show(q2):
    c = Case([50, 50, 50], 1, 4, 128, 32, 16, 11)
    c.dev["ks"][int(c.table[0, 1]), 3, 0, 2] = torch.tensor([0.0, float("nan")])
    c.dev["vs"][int(c.table[1, 1]), 3, 0, 1] = torch.tensor([0.0, float("nan")])
    out = c.run(c.cache(q2)).cpu().numpy()
    assert np.isnan(out[0]).all() and np.isnan(out[1, :, 32:64]).all()
    assert np.isfinite(np.delete(out[1], np.arange(32, 64), axis=1)).all() and np.isfinite(out[2]).all()


def test_stays_inside_its_buffers_and_shares_a_workspace(q2):
    a, b = Case([33, 5000], 2, 4, 128, 64, 16, 12), Case([900, 20, 4000], 4, 2, 256, page=16, seed=13, bits=16)
    need = max(x.cache(q2).ws.numel() for x in (a, b))
    ws = torch.full((256 + need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[256: 256 + need].zero_()
    buf = torch.full((512 + 2 * 1024 + 512,), 0x5A5A, dtype=torch.int16, device="cuda")
    out = buf[512: 512 + 2048].view(torch.float16).view(2, 8, 128)
    for _ in range(2):
        a.check(a.run(a.cache(q2, workspace=ws[256: 256 + need]), out=out))
        b.check(b.run(b.cache(q2, workspace=ws[256: 256 + need])))
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    assert (buf[:512] == 0x5A5A).all() and (buf[2560:] == 0x5A5A).all()
    with pytest.raises(q2.Q2Error):
        a.cache(q2, workspace=ws[:1024])


def test_captured_another_stream_and_no_sequences(q2):
    c = Case([90, 2000], 2, 4, 128, 32, 16, 14)
    cache = c.cache(q2)
    out = torch.empty((2, 8, 128), dtype=torch.float16, device="cuda")
    c.run(cache, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(cache, out=out)
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        c.check(out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(cache, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    empty = q2.PagedKV4(*(c.dev[n] for n in ("k", "ks", "v", "vs")), c.dtable[:0], 8)
    assert empty.attend(c.dq[:0], c.dlens[:0]).shape == (0, 8, 128)


# ---------------------------------------------------------------- over selected blocks


def _lists(c, n, seed):
    """Blocks in any order, some named twice, some that are none."""
    rng = np.random.default_rng(seed)
    return np.stack([np.stack([rng.integers(-2, max(1, -(-m // 64)) + 1, size=n) for _ in range(c.H)]) for m in c.lens]).astype(np.int32)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,q_group,page", [(128, 4, 16), (64, 5, 64), (256, 2, 100), (128, 12, 256), (128, 8, 24)])
@pytest.mark.parametrize("n", [1, 3, 17])
def test_selected_blocks(q2, bits, D, q_group, page, n):
    c = Case([70, 0, 1, 1333, 64, 640, 65], 2, q_group, D, 64, page, n + D, bits=bits, order="head" if n == 3 else "token")
    cache, lists = c.cache(q2), _lists(c, n, n)
    sel = torch.from_numpy(lists).cuda()
    out = c.run(cache, blocks=sel)
    c.check(out, lists)
    assert torch.equal(out, c.run(cache, blocks=sel)) and q2.device_errors() == 0


@pytest.mark.parametrize("bits", [16, 4])
def test_all_blocks_give_all_of_the_attention(q2, bits):
    c = Case([4000, 65, 700], 2, 4, 128, 64, 64, 21, bits=bits)
    lists = np.tile(np.arange(70, dtype=np.int32)[::-1].copy(), (3, 2, 1))
    for b, n in enumerate(c.lens):                      # in any order, those that are none behind
        m = -(-n // 64)
        lists[b, :, :] = -1
        lists[b, :, :m] = np.random.default_rng(b).permutation(m)
    c.check(c.run(c.cache(q2), blocks=torch.from_numpy(lists).cuda()))
    none = torch.full((3, 2, 5), -1, dtype=torch.int32, device="cuda")
    assert (c.run(c.cache(q2), blocks=none) == 0).all()


@pytest.mark.parametrize("bits", [16, 4])
def test_pages_of_other_blocks_are_not_looked_up(q2, bits):
    c = Case([640], 2, 4, 128, 64, 64, 22, bits=bits)
    lists = np.array([[[1, 9], [9, 4]]], dtype=np.int32)
    c.dtable[0, 2], c.dtable[0, 0] = -1, 1 << 30
    out = c.run(c.cache(q2), blocks=torch.from_numpy(lists).cuda())
    c.check(out, lists)
    assert q2.device_errors() == 0
    c.dtable[0, 4] = -5
    out = c.run(c.cache(q2), blocks=torch.from_numpy(lists).cuda())
    assert q2.device_errors() == q2.ERR_PAGE and torch.isnan(out[0, 4:]).all() and not torch.isnan(out[0, :4]).any()
    c.dlens[0] = 100000
    assert torch.isnan(c.run(c.cache(q2), blocks=torch.from_numpy(lists).cuda())).all() and q2.device_errors() == q2.ERR_LENGTH


def test_binding_refuses_what_it_would_misread(q2):
    for bits in (4, 16):
        c = Case([20, 30], 2, 4, 128, 64, 16, 23, bits=bits)
        cache = c.cache(q2)
        sel = torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda")
        for q, lens, kw in ((c.dq.float(), c.dlens, {}), (c.dq[:, :4], c.dlens, {}), (c.dq, c.dlens.long(), {}), (c.dq, c.dlens[:1], {}),
                            (c.dq.cpu(), c.dlens, {}), (c.dq, c.dlens, dict(scale=float("nan"))), (c.dq, c.dlens, dict(blocks=sel.long())),
                            (c.dq, c.dlens, dict(blocks=sel[:1])), (c.dq, c.dlens, dict(blocks=sel[:, :, :0])),
                            (c.dq, c.dlens, dict(blocks=sel[:, :, ::2])), (c.dq, c.dlens, dict(blocks=sel[0])),
                            (c.dq, c.dlens, dict(blocks=sel.cpu()))):
            with pytest.raises(q2.Q2Error):
                cache.attend(q, lens, **kw)
    with pytest.raises(q2.Q2Error):
        cache.attend(c.dq, c.dlens, new_k=c.dq[:, :2], new_v=c.dq[:, :2], blocks=sel)
