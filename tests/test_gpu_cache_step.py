"""The cache's operators together: prompts, then steps of one token each, appended, selected from and attended, against
f64 over what the cache then has to hold; and ``examples/decode_step.py`` on each kind of cache."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import cache as oc
from tests.test_gpu_attend4 import Case as Attention
from tests.test_gpu_select import Case as Selection

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as q2
    q2.load(build_if_missing=True)
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Sequences:
    """What the caches have to hold, in numpy."""

    def __init__(self, q2, bits, H, HQ, D, group, page, batch, room, seed):
        rng = self.rng = np.random.default_rng(seed)
        per = -(-room // page)
        self.bits, self.H, self.HQ, self.D, self.group, self.page, self.batch = bits, H, HQ, D, group, page, batch
        self.table = rng.permutation(batch * per).astype(np.int32).reshape(batch, per)
        dtable = torch.from_numpy(self.table).cuda()
        new = lambda tail, dtype=torch.float16: torch.zeros((batch * per, page, H) + tail, dtype=dtype, device="cuda")  # noqa: E731
        self.bounds = torch.full((batch * per, -(-page // 64), H, 2, D), float("nan"), dtype=torch.float16, device="cuda")
        if bits == 16:
            self.cache = q2.PagedKV(new((D,)), new((D,)), dtable, HQ, bounds=self.bounds)
        else:
            pools = [new((D // 2,), torch.uint8), new((D // group, 2)), new((D // 2,), torch.uint8), new((D // group, 2))]
            self.cache = q2.PagedKV4(*pools, dtable, HQ, bounds=self.bounds)
        self.angles = oc.angles_f32(D, room)
        self.rope = q2.Rope(torch.from_numpy(self.angles).cuda())
        self.keys, self.values = ([np.zeros((0, H, D), np.float32) for _ in range(batch)] for _ in range(2))
        self.lens = np.zeros(batch, dtype=np.int32)

    def append(self, counts):
        """New tokens; returns the turned queries of the last one of each sequence."""
        n, D = sum(counts), self.D
        q, k, v = (self.rng.normal(size=(n, h, D)).astype(np.float16) for h in (self.HQ, self.H, self.H))
        starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        for b, c in enumerate(counts):
            pos = np.arange(self.lens[b], self.lens[b] + c)
            rows = slice(starts[b], starts[b + 1])
            self.keys[b] = np.concatenate([self.keys[b], oc.turn_f64(k[rows], self.angles[pos], False)[0].astype(np.float32)])
            self.values[b] = np.concatenate([self.values[b], v[rows].astype(np.float32)])
        self.lens += np.array(counts, dtype=np.int32)
        dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        self.dlens = dev(self.lens)
        one = counts == [1] * self.batch
        turned = self.cache.append(dev(k), dev(v), self.dlens, starts=None if one else dev(starts), q=dev(q), rope=self.rope)
        return turned[torch.from_numpy(starts[1:].astype(np.int64) - 1).cuda()].contiguous()

    def check(self, q2, q, blocks):
        """The step's selection and attention."""
        sel = self.cache.select(q, self.dlens, blocks, first=1)
        out, some = self.cache.attend(q, self.dlens), self.cache.attend(q, self.dlens, blocks=sel)
        assert q2.device_errors() == 0
        s = Selection.__new__(Selection)
        s.lens, s.H, s.G, s.D, s.page, s.table, s.q = list(self.lens), self.H, self.HQ // self.H, self.D, self.page, self.table, q.cpu().numpy()
        s.bounds = self.bounds.cpu().numpy()
        for b in range(self.batch):                     # the bounds are those of the keys
            for i, want in enumerate(oc.bounds(self.keys[b].astype(np.float16))):
                assert np.array_equal(s.bounds[self.table[b, i * 64 // self.page], i * 64 % self.page // 64], want)
        assert np.array_equal(sel.cpu().numpy(), s.expect(blocks, 1, 1))
        a = Attention.__new__(Attention)
        a.lens, a.H, a.G, a.D, a.group, a.page, a.bits, a.table = s.lens, self.H, s.G, self.D, self.group, self.page, self.bits, self.table
        a.q, a.scale = s.q, self.D ** -0.5
        a.pool = {n: np.zeros(t.shape, np.uint8 if t.dtype == torch.uint8 else np.float16) for n, t in
                  [(n, getattr(self.cache, n)) for n in (("k", "v") if self.bits == 16 else ("k", "ks", "v", "vs"))]}
        for b in range(self.batch):
            pos = np.arange(self.lens[b])
            at = self.table[b, pos // self.page], pos % self.page
            for name, x in (("k", self.keys[b]), ("v", self.values[b])):
                if self.bits == 16:
                    a.pool[name][at] = x.astype(np.float16)
                else:
                    codes, pairs = oc.quantise(x, self.group)
                    a.pool[name][at], a.pool[name + "s"][at] = oc.pack(codes), pairs
        a.check(out)
        a.check(some, sel.cpu().numpy())


@pytest.mark.parametrize("bits,H,HQ,D,group,page", [(16, 2, 8, 128, 64, 64), (4, 2, 10, 128, 64, 16), (4, 1, 12, 64, 32, 256), (16, 3, 3, 64, 64, 32),
                                                    (4, 2, 8, 256, 32, 128)])
def test_prompts_and_steps(ex, bits, H, HQ, D, group, page):
    q2 = ex.q2
    s = Sequences(q2, bits, H, HQ, D, group, page, 4, 900, bits + D)
    s.check(q2, s.append([700, 3, 64, 333]), 4)
    for _ in range(3):
        s.check(q2, s.append([1, 1, 1, 1]), 4)
    s.check(q2, s.append([2, 61, 130, 1]), 6)


CFG = dict(layers=2, hidden=512, q_heads=8, kv_heads=2, dim=64, ffn=768, batch=3, room=400, seed=5)


def _steps(ex, graph, n=4, **kw):
    """Hidden states of n steps behind prompts of 250, 0 and 70 tokens."""
    d = ex.Decoder(**CFG, **kw)
    past = torch.tensor([250, 0, 70], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 250, 250, 320], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for cache in d.caches:
        k, v = (torch.randn(320, CFG["kv_heads"], CFG["dim"], device="cuda", generator=g).half() for _ in range(2))
        cache.append(k, v, past, starts=starts, rope=d.rope)
    d.lens.copy_(past)
    run = d.capture().replay if graph else d.step
    out = []
    for _ in range(n):
        d.h.copy_(torch.randn(3, CFG["hidden"], device="cuda", generator=g).half())
        run()
        out.append((d.h.double() + d.last.double()).cpu())
    assert ex.q2.device_errors() == 0 and d.lens.tolist() == [250 + n, n, 70 + n]
    return torch.stack(out)


@pytest.mark.parametrize("kw", [dict(), dict(bits=4), dict(blocks=2), dict(bits=4, blocks=2, page=64)])
def test_the_example_on_each_cache(ex, kw):
    """A captured step gives what an eager one does, and 4 bits and a few blocks what all of an fp16 cache does, roughly:
    a group of 64 spans 5 standard deviations, so a value in 4 bits is off by 5 / 15 / sqrt(12) = 10% of one (root mean
    square), which two layers add to hidden states of which attention is a part; two blocks of five keep the two that
    weigh the most of nearly even ones."""
    eager = _steps(ex, False, **kw)
    assert torch.isfinite(eager).all() and torch.equal(_steps(ex, True, **kw), eager)
    whole = _steps(ex, False)
    rel = ((eager - whole).square().sum(-1) / whole.square().sum(-1)).sqrt()
    assert (rel < (0.2 if "blocks" not in kw else 1.0)).all(), rel
    if kw == {}:
        assert torch.equal(eager, whole)


def test_all_blocks_are_all_of_the_cache(ex):
    """Selecting as many blocks as there are gives the same tokens: the outputs differ by the sums' splits alone."""
    for bits in (16, 4):
        rel = (_steps(ex, False, bits=bits, blocks=7) - _steps(ex, False, bits=bits)).abs().max()
        assert rel < 0.05, rel


@pytest.mark.parametrize("bits", [16, 4])
def test_capturing_leaves_the_state_alone(ex, bits):
    """Captured behind partly filled blocks with a live residual stream: nothing of the caches (their bounds among it), the
    lengths and the stream changes, and what comes behind is what eager steps alone give."""
    def start():
        d = ex.Decoder(**CFG, bits=bits, blocks=2, page=32)
        past = torch.tensor([250, 0, 70], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, 250, 250, 320], dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(2)
        for cache in d.caches:
            k, v = (torch.randn(320, CFG["kv_heads"], CFG["dim"], device="cuda", generator=g).half() for _ in range(2))
            cache.append(k, v, past, starts=starts, rope=d.rope)
        d.lens.copy_(past)
        hidden = [torch.randn(3, CFG["hidden"], device="cuda", generator=g).half() for _ in range(6)]
        return d, hidden

    def state(d):
        names = ("k", "v", "bounds") if bits == 16 else ("k", "ks", "v", "vs", "bounds")
        return [d.lens.clone(), d.h.clone(), d.last.clone()] + [getattr(c, n).clone() for c in d.caches for n in names]

    def run(d, hidden, captured):
        step, seen = d.step, []
        for i, h in enumerate(hidden):
            if captured and i == 3:
                before = state(d)
                step = d.capture().replay
                assert all(torch.equal(a, b) for a, b in zip(before, state(d)))
            d.h.copy_(h)
            step()
            seen.append(d.last.clone())
        return seen + state(d)

    assert all(torch.equal(a, b) for a, b in zip(run(*start(), True), run(*start(), False)))
    assert ex.q2.device_errors() == 0


@pytest.mark.parametrize("past", [0, 1, 100])
@pytest.mark.parametrize("more", [[], ["--cache-bits", "4", "--blocks", "2"]])
def test_the_example_from_the_command_line(ex, monkeypatch, capsys, past, more):
    sizes = dict(layers=1, hidden=512, q_heads=8, kv_heads=2, dim=64, ffn=768, batch=3, steps=2, past=past)
    args = [a for n, v in sizes.items() for a in ("--" + n.replace("_", "-"), str(v))]
    monkeypatch.setattr("sys.argv", ["decode_step.py"] + args + more)
    ex.main()
    assert f"lengths {[37 * b % max(past, 1) + 2 for b in range(3)]}" in capsys.readouterr().out


class _Checked:
    """A cache whose selections and outputs are compared with those of what it holds, call for call."""

    def __init__(self, cache, bits):
        self.cache, self.bits, self.calls = cache, bits, 0

    def append(self, *args, **kw):
        return self.cache.append(*args, **kw)

    def select(self, q, lens, blocks):
        self.sel = self.cache.select(q, lens, blocks)
        c = self.cache
        s = Selection.__new__(Selection)
        s.lens, s.H, s.G, s.D, s.page = lens.tolist(), c.kv_heads, c.q_heads // c.kv_heads, c.dim, c.k.shape[1]
        s.table, s.q, s.bounds = c.table.cpu().numpy(), q.cpu().numpy(), c.bounds.cpu().numpy()
        assert np.array_equal(self.sel.cpu().numpy(), s.expect(blocks, 0, 1))
        return self.sel

    def attend(self, q, lens, out, blocks):
        assert blocks is self.sel
        c = self.cache
        c.attend(q, lens, out=out, blocks=blocks)
        a = Attention.__new__(Attention)
        a.lens, a.H, a.G, a.D, a.group, a.page = lens.tolist(), c.kv_heads, c.q_heads // c.kv_heads, c.dim, 64, c.k.shape[1]
        a.bits, a.table, a.q, a.scale = self.bits, c.table.cpu().numpy(), q.cpu().numpy(), c.dim ** -0.5
        a.pool = {n: getattr(c, n).cpu().numpy() for n in (("k", "v") if self.bits == 16 else ("k", "ks", "v", "vs"))}
        a.check(out, blocks.cpu().numpy())
        assert (out != 0).any(-1).all()
        self.calls += 1


@pytest.mark.parametrize("bits,page", [(16, 16), (4, 64), (4, 16)])
def test_the_example_attends_the_blocks_that_promise_the_most(ex, bits, page):
    """Every layer's selection and attention of eager steps against f64 over the blocks that the bounds name."""
    d = ex.Decoder(**CFG, bits=bits, blocks=2, page=page)
    past = torch.tensor([250, 0, 70], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 250, 250, 320], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for cache in d.caches:
        k, v = (torch.randn(320, CFG["kv_heads"], CFG["dim"], device="cuda", generator=g).half() for _ in range(2))
        cache.append(k, v, past, starts=starts, rope=d.rope)
    d.lens.copy_(past)
    d.caches = [_Checked(c, bits) for c in d.caches]
    for _ in range(4):
        d.h.copy_(torch.randn(3, CFG["hidden"], device="cuda", generator=g).half())
        d.step()
    assert [c.calls for c in d.caches] == [4, 4] and ex.q2.device_errors() == 0
