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
