"""``q2_read`` and ``q2_read4`` of so many rows that a thread takes four pieces of them (four CTAs' per SM and more): rows of
ragged sequences out of random pools, bit for bit what the oracle says that they stand for."""
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


class Case:
    def __init__(self, bits, group, D, H, page, order, both):
        rng = np.random.default_rng(D + H + page)
        self.bits, self.group, self.D, self.H, self.page = bits, group, D, H, page
        pieces = 4 * 256 * 4 * torch.cuda.get_device_properties(0).multi_processor_count
        rows = -(-pieces // (H * D // 8 * (2 if both else 1)))
        # the last `counts` of `lens` tokens; a sequence without tokens, one that is read in part, one without rows
        self.counts = [1, rows // 3, 0, 777, 65, rows // 2, 0, rows // 6 + 40]
        self.lens = [1, rows // 3, 0, 1500, 65, rows // 2, 9, rows // 6 + 40]
        need = [-(-n // page) for n in self.lens]
        ids, at = rng.permutation(sum(need) + 1).astype(np.int32), 0
        self.table = np.full((8, max(need)), -7, dtype=np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at: at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        self.ntok = int(self.starts[-1]) + 5
        shape = (sum(need) + 1, page, H)
        if bits == 16:
            self.pools = {n: rng.normal(size=shape + (D,)).astype(np.float16) for n in "kv"}
        else:
            self.pools = {}
            for n in "kv":
                self.pools[n] = rng.integers(0, 256, size=shape + (D // 2,), dtype=np.uint8)
                self.pools[n + "s"] = rng.normal(size=shape + (D // group, 2)).astype(np.float16)
        ordered = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2) if order == "head" else t  # noqa: E731
        self.dev = {n: ordered(torch.from_numpy(p).cuda()) for n, p in self.pools.items()}
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dlens, self.dstarts = torch.tensor(self.lens, dtype=torch.int32, device="cuda"), torch.from_numpy(self.starts).cuda()

    def cache(self, q2):
        d = self.dev
        return q2.PagedKV(d["k"], d["v"], self.dtable, self.H) if self.bits == 16 else \
            q2.PagedKV4(d["k"], d["ks"], d["v"], d["vs"], self.dtable, self.H)

    def expect(self, name):
        out = np.full((self.ntok, self.H, self.D), 7, dtype=np.float16)
        for b, (n, c) in enumerate(zip(self.lens, self.counts)):
            pos = np.arange(n - c, n)
            at = self.table[b, pos // self.page], pos % self.page
            x = self.pools[name][at]
            out[self.starts[b]: self.starts[b + 1]] = x if self.bits == 16 else \
                oc.value_f64(x, self.pools[name + "s"][at]).astype(np.float32).astype(np.float16)
        return out


def _same(got, want):
    return np.array_equal(np.ascontiguousarray(got.cpu().numpy()).view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("bits,group", [(16, 32), (4, 32), (4, 64)])
@pytest.mark.parametrize("D,H,page,order", [(64, 8, 24, "token"), (128, 3, 64, "head"), (256, 2, 16, "token"), (128, 8, 256, "head")])
def test_rows_of_many_tokens(q2, bits, group, D, H, page, order):
    c = Case(bits, group, D, H, page, order, True)
    wide = torch.full((c.ntok, H * D + 16), 7.0, dtype=torch.float16, device="cuda")
    k, v = wide[:, : H * D].unflatten(1, (H, D)), torch.full((c.ntok, H, D), 7.0, dtype=torch.float16, device="cuda")
    c.cache(q2).read(c.dlens, starts=c.dstarts, k_out=k, v_out=v)
    want = c.expect("k"), c.expect("v")
    assert _same(k, want[0]) and _same(v, want[1]) and (wide[:, H * D:] == 7).all()
    assert q2.device_errors() == 0
    # a page that does not exist and a length that cannot be: their rows are NaN, the others as before
    c.dtable[5, 1], c.dlens[3] = -1, c.table.shape[1] * page + 1
    bad = np.zeros(c.ntok, dtype=bool)
    bad[c.starts[5] + page: min(c.starts[5] + 2 * page, c.starts[6])] = True
    bad[c.starts[3]: c.starts[4]] = True
    c.cache(q2).read(c.dlens, starts=c.dstarts, k_out=k, v_out=v)
    assert q2.device_errors() == q2.ERR_LENGTH | q2.ERR_PAGE
    for got, w in ((k, want[0]), (v, want[1])):
        assert torch.isnan(got[torch.from_numpy(bad).cuda()]).all() and _same(got[torch.from_numpy(~bad).cuda()], w[~bad])


@pytest.mark.parametrize("bits,group", [(16, 32), (4, 32), (4, 64)])
@pytest.mark.parametrize("name", ["k", "v"])
def test_keys_or_values_alone(q2, bits, group, name):
    c = Case(bits, group, 128, 5, 16, "token", False)
    out = torch.full((c.ntok, 5, 128), 7.0, dtype=torch.float16, device="cuda")
    c.cache(q2).read(c.dlens, starts=c.dstarts, **{name + "_out": out})
    assert _same(out, c.expect(name)) and q2.device_errors() == 0
