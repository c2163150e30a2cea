"""Calls on a stream that is not the current one: outputs made by the call do not lie in memory that the current stream
may still write, and a workspace made by a constructor is zero before any stream's first call.

The current stream is held up by a short sleep with a write behind it, to a block which is then given back.
"""
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
MS = 2_000_000                                                  # about a millisecond of clock cycles


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _held_block(nbytes):
    """Give back a block that the current stream will still write, 20 ms from now."""
    block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(20 * MS)
    block.fill_(0x5A)


def _operators(q2):
    d, e = synth.int4(640, 512, 64, 970, True), synth.bpdq(640, 512, 971)
    four = q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], 64))
    two = q2.Packed(q2.q2_pack_bpdq(e["plane0"], e["plane1"], e["coef"]))
    x = torch.from_numpy(synth.activations(4, 512, 972)).cuda()
    x8, xs = (torch.from_numpy(a).cuda() for a in synth.activations8(4, 512, 973))
    norm = q2.RmsNorm(torch.ones(512, dtype=torch.float16, device="cuda"))
    inp = synth.rotation(1024, 1024, 974)
    rot, xr = q2.Rotation(inp["signs"], inp["q"], 1024, 1024), torch.from_numpy(synth.activations(4, 1024, 975)).cuda()
    k = torch.randn((8, 16, 2, 64), device="cuda").half()
    kv = q2.PagedKV(k, k.clone(), torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4), 8)
    q, lens = torch.randn((2, 8, 64), device="cuda").half(), torch.tensor([50, 9], dtype=torch.int32, device="cuda")
    return [("gemv, 2 bits", lambda s: two.gemv(x, stream=s)), ("gemv, 4 bits", lambda s: four.gemv(x, stream=s)),
            ("gemv_x8", lambda s: four.gemv_x8(x8, xs, stream=s)), ("decode", lambda s: four.decode(stream=s)),
            ("norm", lambda s: norm.apply(x, stream=s)), ("rotation", lambda s: rot.apply(xr, stream=s)),
            ("attention", lambda s: kv.attend(q, lens, stream=s))]


@pytest.mark.parametrize("which", range(7))
def test_outputs_made_by_the_call(q2, which):
    name, call = _operators(q2)[which]
    want = call(None).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        _held_block(want.numel() * want.element_size())
        got = call(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name


def test_workspaces_made_by_constructors(q2):
    k = torch.randn((400, 16, 2, 64), device="cuda").half()
    table, lens = torch.arange(400, dtype=torch.int32, device="cuda").view(1, 400), torch.tensor([6400], dtype=torch.int32, device="cuda")
    q, d = torch.randn((1, 8, 64), device="cuda").half(), synth.bpdq(640, 512, 976)
    blob, x = q2.q2_pack_bpdq(d["plane0"], d["plane1"], d["coef"]), torch.from_numpy(synth.activations(1, 512, 977)).cuda()
    kv, pk = (lambda: q2.PagedKV(k, k, table, 8)), (lambda: q2.Packed(blob, ntok_max=1))
    want = kv().attend(q, lens).clone(), pk().gemv(x).clone()
    side = torch.cuda.Stream()
    for make, call, w in ((kv, lambda h: h.attend(q, lens, stream=side), want[0]), (pk, lambda h: h.gemv(x, stream=side), want[1])):
        n = make().ws.numel()
        torch.cuda.synchronize()
        _held_block(n)
        got = call(make())
        torch.cuda.synchronize()
        assert torch.equal(got, w)
