"""Workspaces that a caller brings: one run of GPU memory, counted in bytes; anything else is refused on the host."""
import pytest

import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    return m


def _bad(need):
    return [torch.zeros(need, dtype=torch.uint8), torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]]


def test_attention(q2):
    k = torch.randn((8, 16, 2, 64), device="cuda").half()
    table, lens = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4), torch.tensor([50, 9], dtype=torch.int32, device="cuda")
    q = torch.randn((2, 8, 64), device="cuda").half()
    make = lambda ws=None: q2.PagedKV(k, k.clone(), table, 8, workspace=ws)
    want, need = make().attend(q, lens), make().ws.numel()
    for ws in _bad(need) + [torch.zeros(need // 4 - 64, dtype=torch.int32, device="cuda")]:
        with pytest.raises(q2.Q2Error):
            make(ws)
    assert torch.equal(make(torch.zeros(need // 4 + 1, dtype=torch.int32, device="cuda")).attend(q, lens), want)


def test_products(q2):
    d = synth.bpdq(256, 512, 960)
    pk = q2.Packed(q2.q2_pack_bpdq(d["plane0"], d["plane1"], d["coef"]), ntok_max=2)
    x = torch.from_numpy(synth.activations(2, 512, 961)).cuda()
    want, own, need = pk.gemv(x), pk.ws, pk.workspace_bytes(2)
    for ws in _bad(need):
        with pytest.raises(q2.Q2Error):
            pk.set_workspace(ws)
        assert pk.ws is own and torch.equal(pk.gemv(x), want)       # the one before stays
    pk.set_workspace(torch.zeros(need // 8, dtype=torch.int64, device="cuda"))
    assert torch.equal(pk.gemv(x), want)


def test_attention_needs_no_more_than_its_parts(q2):
    """Two parts to a CTA, of as many rows of D numbers, a maximum and a denominator as a unit has heads (two CTAs per SM of 16
    heads of 128 are the most), then a counter per (sequence, key-value head): a workspace of this size serves every call."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    parts = 2 * 2 * sms * 16 * (128 * 4 + 8)
    g = torch.Generator(device="cuda").manual_seed(5)
    table = torch.arange(1024, dtype=torch.int32, device="cuda").view(2, 512)
    lens = torch.tensor([32768, 9001], dtype=torch.int32, device="cuda")
    for D, heads in ((64, 2), (64, 32), (128, 2), (128, 32), (256, 2), (256, 32)):
        need = -(-parts // 256) * 256 + 2 * 2 * -(-(heads // 2) // (16 if D < 256 else 8)) * 4
        ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        ws[:need] = 0
        rows = lambda *shape: torch.randn(shape, device="cuda", generator=g).half()
        q = rows(2, heads, D)
        k, v = rows(1024, 64, 2, D), rows(1024, 64, 2, D)
        full = q2.PagedKV(k, v, table, heads)
        c4 = q2.PagedKV4.empty(1024, 64, 2, D, 64, table, heads)
        c4.ks[..., 0], c4.vs[..., 0] = 0.1, 0.1
        c4.k.random_(0, 256, generator=g)
        c4.v.random_(0, 256, generator=g)
        want = full.attend(q, lens), c4.attend(q, lens)
        full = q2.PagedKV(k, v, table, heads, workspace=ws[:need])
        c4 = q2.PagedKV4(c4.k, c4.ks, c4.v, c4.vs, table, heads, workspace=ws[:need])
        assert torch.equal(full.attend(q, lens), want[0]) and torch.equal(c4.attend(q, lens), want[1])
        assert (ws[need:] == 0xA5).all() and (ws[need - 16:need] == 0).all()
    assert q2.device_errors() == 0
