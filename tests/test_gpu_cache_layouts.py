"""Caches laid out in other ways than one tensor per pool, places far into them, scales of either sign, selections whose
shared memory leaves no room for stages, and what several calls in a row leave."""
import numpy as np
import pytest

from oracle import cache as oc
from tests.test_gpu_append import Case as Append
from tests.test_gpu_attend4 import Case as Attention
from tests.test_gpu_select import Case as Selection

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _apart(t, gap):
    """The same values in a tensor whose pages, tokens and heads lie further apart, marks in between."""
    P, page, H = t.shape[:3]
    n = t[0, 0, 0].numel()
    wide = torch.full((P, page + 1, H + 1, n + gap), 77, dtype=t.dtype, device=t.device)
    view = wide[:, :page, :H, :n].unflatten(3, t.shape[3:])
    view.copy_(t)
    return view, wide


@pytest.mark.parametrize("bits,group,D", [(16, 32, 128), (4, 32, 128), (4, 64, 64), (4, 64, 256), (4, 32, 256)])
def test_pools_with_gaps(q2, bits, group, D):
    """Strides that are multiples of 16 bytes (of the pairs of a head) and nothing more."""
    c = Append([70, 3, 130], [70, 1, 40], 2, 8, D, bits, group, page=16, seed=D + group)
    gap = {"k": 8, "v": 8, "ks": min(8, 2 * D // group), "vs": min(8, 2 * D // group)} if bits == 16 else \
        {"k": 16, "v": 16, "ks": min(8, 2 * D // group), "vs": min(8, 2 * D // group)}
    wides = {}
    for n in c.dev:
        c.dev[n], wides[n] = _apart(c.dev[n], gap[n])
    before = {n: w.clone() for n, w in wides.items()}
    cache = c.cache(q2)
    c.check_q(c.run(q2, cache=cache))
    c.check_pools()
    for n, w in wides.items():                          # nothing between the rows
        P, page, H = c.dev[n].shape[:3]
        row = c.dev[n][0, 0, 0].numel()
        for a, b in ((w[:, page:], before[n][:, page:]), (w[:, :, H:], before[n][:, :, H:]), (w[..., row:], before[n][..., row:])):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    # and what the other calls read is what is there
    want, _ = c.expect()
    k, v = cache.read(c.dlens, starts=c.dstarts, ntok=c.ntok)
    lens, q = list(c.lens), torch.randn((3, 8, D), device="cuda").half()
    a = Attention.__new__(Attention)
    a.lens, a.H, a.G, a.D, a.group, a.page, a.bits, a.table, a.q, a.scale = lens, 2, 4, D, group, 16, bits, c.table, q.cpu().numpy(), 0.3
    a.pool = want
    # tokens before the new ones hold marks: make them tokens
    for b, (n, m) in enumerate(zip(c.lens, c.counts)):
        pos = np.arange(n - m)
        at = c.table[b, pos // 16], pos % 16
        rng = np.random.default_rng(b)
        for name in want:
            x = want[name][at]
            want[name][at] = rng.integers(0, 256, size=x.shape) if x.dtype == np.uint8 else np.abs(rng.normal(size=x.shape)) * 0.1
        for name in want:
            c.dev[name].copy_(torch.from_numpy(want[name]))
    for blocks in (None, torch.tensor([[[0, 1]] * 2, [[0, -1]] * 2, [[2, 0]] * 2], dtype=torch.int32, device="cuda")):
        a.check(cache.attend(q, c.dlens, scale=0.3, blocks=blocks), None if blocks is None else blocks.cpu().numpy())
    assert q2.device_errors() == 0


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("q_group", [2, 7, 11])
def test_scales_of_either_sign(q2, bits, scale, q_group):
    c = Attention([300, 33], 2, q_group, 128, 64, 16, 31, bits=bits)
    c.scale = scale
    c.check(c.run(c.cache(q2)))
    lists = np.array([[[4, 1]] * 2, [[0, -1]] * 2], dtype=np.int32)
    c.check(c.run(c.cache(q2), blocks=torch.from_numpy(lists).cuda()), lists)


def test_queries_far_apart(q2):
    """One column of the queries far above the rest, heads of zeros, and heads whose sizes differ by 2^20."""
    c = Attention([200, 17], 2, 4, 128, 64, 16, 32)
    q = c.q.copy()
    q[:, 0, 5], q[:, 1] = 300.0, 0
    q[:, 2] *= np.float16(2.0 ** -12)
    q[:, 3] *= 200
    c.q = q
    c.dwide[:, : 8 * 128] = torch.from_numpy(q.reshape(2, -1)).cuda()
    c.check(c.run(c.cache(q2)))


def test_places_beyond_four_gigabytes(q2):
    """Pools of five pages a gigabyte and more apart: token by token, into the last page and back."""
    P, page, H, D, group = 5, 64, 2, 128, 64
    far = {"k": (1 << 30) + 4096, "ks": (1 << 28) + 64}                         # bytes; pairs
    flat = {n: torch.zeros(4 * far["k"] + page * H * D // 2, dtype=torch.uint8, device="cuda") for n in ("k", "v")}
    flat |= {n: torch.zeros(2 * (4 * far["ks"] + page * H * D // group), dtype=torch.float16, device="cuda") for n in ("ks", "vs")}
    pool = {n: flat[n].as_strided((P, page, H, D // 2), (far["k"], H * D // 2, D // 2, 1)) for n in ("k", "v")}
    pool |= {n: flat[n].as_strided((P, page, H, D // group, 2), (2 * far["ks"], 2 * H * D // group, 2 * D // group, 2, 1)) for n in ("ks", "vs")}
    table = torch.tensor([[4, 2, 3]], dtype=torch.int32, device="cuda")
    bounds = torch.zeros((P, 1, H, 2, D), dtype=torch.float16, device="cuda")
    cache = q2.PagedKV4(pool["k"], pool["ks"], pool["v"], pool["vs"], table, 8, bounds=bounds)
    rng = np.random.default_rng(33)
    k, v = (rng.normal(size=(150, H, D)).astype(np.float16) for _ in range(2))
    lens, starts = torch.tensor([150], dtype=torch.int32, device="cuda"), torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    cache.append(torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), lens, starts=starts)
    values = [oc.value_f64(oc.pack(oc.quantise(x.astype(np.float32), group)[0]), oc.quantise(x.astype(np.float32), group)[1]) for x in (k, v)]
    for got, want in zip(cache.read(lens, starts=starts, ntok=150), values):
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32).astype(np.float16))
    a = Attention([150], H, 4, D, group, page, 34)
    a.table = table.cpu().numpy()
    a.pool = {n: np.zeros(t.shape, np.uint8 if t.dtype == torch.uint8 else np.float16) for n, t in pool.items()}
    pos = np.arange(150)
    for n, x in (("k", k), ("v", v)):
        codes, pairs = oc.quantise(x.astype(np.float32), group)
        a.pool[n][a.table[0, pos // 64], pos % 64], a.pool[n + "s"][a.table[0, pos // 64], pos % 64] = oc.pack(codes), pairs
    a.check(cache.attend(a.dq, lens))
    sel = cache.select(a.dq, lens, 2)
    a.check(cache.attend(a.dq, lens, blocks=sel), sel.cpu().numpy())
    assert q2.device_errors() == 0


@pytest.mark.parametrize("D,q_group,pages", [(256, 64, 512), (256, 8, 512), (128, 64, 512), (64, 64, 512), (128, 4, 256)])
def test_selections_of_caches_with_room_for_millions_of_tokens(q2, D, q_group, pages):
    """Pages of 4096 tokens, so that a table row reaches 2^21 tokens: shared memory for all of their scores."""
    c = Selection([9000, 130, 64 * 77], 1, q_group, D, 4096, D + q_group)
    c.table = np.concatenate([c.table, np.full((3, pages - c.table.shape[1]), -7, dtype=np.int32)], axis=1)
    c.check(q2, 5, 1, 1)
    assert q2.device_errors() == 0


def test_angles_whose_tile_takes_nearly_all_of_the_plain_shared_memory(q2):
    """Turned columns from 16 to 256 of heads of 256: 4 to 64 KB of angles."""
    for rot in (16, 112, 128, 144, 160, 176, 192, 208, 256):
        for bits in (16, 4):
            c = Append([64, 100], [64, 70], 2, 6, 256, bits, 64, page=64, rot=rot, bounds=True, seed=rot)
            c.check_q(c.run(q2))
            c.check_pools()


def test_several_calls_in_a_row_without_waiting(q2):
    """Appends, reads and attentions on one stream, each on what the one before it left, as one captured graph would run them."""
    c = Append([200, 90], [200, 90], bits=4, group=64, page=64, order="head", bounds=True, seed=35)
    cache, rope = c.cache(q2), c.rope(q2)
    lens = [torch.tensor([a, b], dtype=torch.int32, device="cuda") for a, b in ((100, 1), (150, 45), (200, 90))]
    outs = []
    q = torch.randn((2, c.HQ, c.D), device="cuda").half()
    for n, prev in zip(lens, [torch.zeros_like(lens[0])] + lens[:-1]):
        count = (n - prev).tolist()
        starts = torch.tensor([0, count[0], count[0] + count[1]], dtype=torch.int32, device="cuda")
        rows = torch.cat([torch.arange(int(prev[0]), int(n[0])), 200 + torch.arange(int(prev[1]), int(n[1]))]).cuda()
        cache.append(c.dk[rows], c.dv[rows], n, starts=starts, rope=rope)
        outs.append((cache.attend(q, n), cache.select(q, n, 2), cache.read(n)[0]))
    c.check_pools()
    for n, (o, s, k) in zip(lens, outs):                # the same again, now that all is there
        assert torch.equal(o, cache.attend(q, n)) and torch.equal(k, cache.read(n)[0])
    assert torch.equal(outs[-1][1], cache.select(q, lens[-1], 2)) and q2.device_errors() == 0


def test_what_the_caches_refuse(q2):
    c = Append([20, 30], [1, 1], bits=16, page=16, seed=36, starts=False, bounds=True)
    cache, q = c.cache(q2), torch.zeros((2, c.HQ, c.D), dtype=torch.float16, device="cuda")
    with pytest.raises(q2.Q2Error):                     # the new tokens would not be in the bounds
        cache.attend(q, c.dlens, c.dk, c.dv)
    cache.attend(q, c.dlens)
    c = Append([20, 30], [1, 1], bits=4, page=16, seed=37, starts=False)
    d = c.dev
    for n in (1, 3, 8, 16):                             # 128 columns in 1, 3, 8, 16 groups
        bad = [torch.zeros(d["k"].shape[:3] + (n, 2), dtype=torch.float16, device="cuda") for _ in range(2)]
        with pytest.raises(q2.Q2Error):
            q2.PagedKV4(d["k"], bad[0], d["v"], bad[1], c.dtable, c.HQ)
    assert q2.device_errors() == 0


def _held_block(nbytes):
    """Give back a block that the current stream will still write, some 20 ms from now."""
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(40_000_000)
    block.fill_(0x5A)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("which", ["attend", "blocks", "select", "read"])
def test_outputs_made_by_calls_on_another_stream(q2, bits, which):
    """They do not lie in memory that the current stream may still write."""
    c = Append([200, 90], [200, 90], bits=bits, group=64, page=64, bounds=True, seed=38)
    cache = c.cache(q2)
    c.run(q2, cache=cache)
    q, lens = torch.randn((2, c.HQ, c.D), device="cuda").half(), c.dlens
    sel = cache.select(q, lens, 2)
    call = {"attend": lambda s: (cache.attend(q, lens, stream=s),), "blocks": lambda s: (cache.attend(q, lens, blocks=sel, stream=s),),
            "select": lambda s: (cache.select(q, lens, 2, stream=s),),
            "read": lambda s: cache.read(lens, starts=c.dstarts, ntok=c.ntok, stream=s)}[which]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        for t in want:
            _held_block(t.numel() * t.element_size())
        got = call(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bits", [16, 4])
def test_two_captured_graphs_on_one_workspace(q2, bits):
    """A step of a long sequence and one of a few short ones, replayed by turns."""
    long, short = (Attention(lens, 2, 4, 128, 64, 16, 40 + i, bits=bits) for i, lens in enumerate(([9000], [70, 1, 300])))
    caches = [c.cache(q2) for c in (long, short)]
    ws = max((k.ws for k in caches), key=lambda w: w.numel())
    caches = [type(k)(*(getattr(k, n) for n in (("k", "v") if bits == 16 else ("k", "ks", "v", "vs"))), k.table, k.q_heads, workspace=ws)
              for k in caches]
    side, graphs, outs = torch.cuda.Stream(), [], []
    for c, k in zip((long, short), caches):
        out = torch.zeros((len(c.lens), 8, 128), dtype=torch.float16, device="cuda")
        k.attend(c.dq, c.dlens, scale=c.scale, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            k.attend(c.dq, c.dlens, scale=c.scale, out=out)
        graphs.append(graph)
        outs.append(out)
    for out in outs:
        out.zero_()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for c, out in zip((long, short), outs):
        c.check(out)
    assert q2.device_errors() == 0


@pytest.mark.parametrize("D,q_group,lens", [(128, 4, [64 * 2000]), (64, 3, [64 * 1500, 64 * 700]), (256, 12, [64 * 900, 5000])])
def test_one_block_far_above_the_rest(q2, D, q_group, lens):
    """Its magnitudes say that any of the others' sums may be off by more than they are apart: all are taken exactly."""
    c = Selection(lens, 2, q_group, D, 64, D + 1)
    pages = c.table[0]
    c.bounds[pages[100], 0, 0] = [[-65504.0], [65504.0]]
    c.bounds[pages[200], 0, 1, 1, 7] = np.inf
    c.check(q2, 40, 1, 1)
    c.check(q2, 1, 0, 0)
    c.q[:, :, :3] *= 1000                               # and some columns of the queries far above the others
    c.check(q2, 40, 0, 1)
    assert q2.device_errors() == 0


def test_a_cache_without_bounds_keeps_no_room_for_them(q2):
    pages, page, H, D = 512, 16, 8, 128
    table = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    least = 2 * pages * page * H * (D // 2 + 4 * D // 64)
    for bounds in (False, True):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        c = q2.PagedKV4.empty(pages, page, H, D, 64, table, 16, bounds=bounds)
        kept = c.bounds.numel() * 2 if bounds else 0
        room = least + c.ws.numel() + kept
        assert room <= torch.cuda.max_memory_allocated() - before < room + (1 << 20) and (c.bounds is None) == (not bounds)
        del c
