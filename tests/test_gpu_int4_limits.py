"""``Q2_INT4`` products where they could go wrong: every token count of the tensor-core
path, few columns, rows of weights that are all zero, and waits that run out.

Tolerances.  For fp16 x and up to 16 tokens a group's sum is formed as
sum q x - z sum x: both are sums of exact products in fp32 of at most
2^-23 of their magnitudes per addition, so with M = sum s (q + z) |x| the
bound is 2^-11 |ref| + 2^-25 + (2 group + C / group + 16) 2^-24 M; above 16
tokens M = sum |w x| takes its place.  (For a typical row M is about three
times sum |w x|.)  8-bit x: the group sums are exact, without the term
2 group; and sum q x8 = z sum x8 exactly where q = z.
"""
import numpy as np
import pytest

import synth
from oracle import int4 as oint4, matvec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as m
    m.load(build_if_missing=True)
    m.debug_wait_limit(0)
    m.device_errors()                          # start from a clear error word
    yield m
    m.debug_wait_limit(0)


def _check(y, d, x, exact_groups=False):
    group, C = d["group"], d["C"]
    w = oint4.decode_f64(d["code"], d["scale"], d["zero"], group)
    M = matvec.abs_bound(w, x)
    if x.shape[0] <= 16:
        q = np.stack([d["code"] & 15, d["code"] >> 4], axis=-1).reshape(w.shape).astype(np.float64)
        z = 8.0 if d["zero"] is None else np.repeat(d["zero"].astype(np.float64), group, axis=1)
        M = matvec.abs_bound(np.repeat(d["scale"].astype(np.float64), group, axis=1) * (q + z), x)
    ref = matvec.gemv(w, x)
    k = C // group + 16 + (0 if exact_groups else 2 * group)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + k * 2.0 ** -24 * M
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} outside; worst {(err / tol).max():.2f}x"


def _both(q2, d, ntok, seed):
    pk = q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], d["group"]))
    x = synth.activations(ntok, d["C"], seed)
    _check(pk.gemv(torch.from_numpy(x).cuda()), d, x)
    x8, xs = synth.activations8(ntok, d["C"], seed)
    _check(pk.gemv_x8(torch.from_numpy(x8).cuda(), torch.from_numpy(xs).cuda()), d, x8 * xs.astype(np.float64)[:, None], True)


@pytest.mark.parametrize("ntok", range(1, 65))
def test_every_token_count(q2, ntok):
    _both(q2, synth.int4(145, 416 if ntok % 2 else 384, 32 if ntok % 2 else 64, 700 + ntok, ntok % 3 > 0), ntok, 701)


@pytest.mark.parametrize("C,group", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 32), (128, 128), (160, 32), (256, 128)])
@pytest.mark.parametrize("ntok", [1, 16, 17, 40, 64])
def test_few_columns(q2, C, group, ntok):
    _both(q2, synth.int4(300, C, group, 710, True), ntok, 711)


@pytest.mark.parametrize("ntok", [1, 2, 6, 16, 20, 64])
def test_weights_that_are_zero(q2, ntok):
    """Every other row has q = z throughout: exactly zero from 8-bit x, and within the bound from fp16."""
    R, C, group = 96, 2048, 128
    d = synth.int4(R, C, group, 720, True)
    z = np.repeat(d["zero"], group // 2, axis=1)
    d["code"][::2] = (z | z << 4)[::2]
    _both(q2, d, ntok, 721)
    pk = q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], group))
    x8, xs = synth.activations8(ntok, C, 722)
    y = pk.gemv_x8(torch.from_numpy(x8).cuda(), torch.from_numpy(xs).cuda())
    assert (y[:, ::2] == 0).all() and (y[:, 1::2] != 0).any()


@pytest.mark.parametrize("ntok", [3, 16, 64])
def test_captured_in_a_graph(q2, ntok):
    d = synth.int4(640, 1024, 64, 730, False)
    pk = q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], 64))
    xd = torch.zeros((ntok, 1024), dtype=torch.float16, device="cuda")
    y = torch.empty((ntok, 640), dtype=torch.float16, device="cuda")
    pk.gemv(xd, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.gemv(xd, y)
        pk.gemv(xd, y)
    x = synth.activations(ntok, 1024, 731)
    xd.copy_(torch.from_numpy(x))
    graph.replay()
    _check(y, d, x)


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("R,C,ntok", [(128, 4096, 64), (4096, 1024, 33)])
def test_waits_that_run_out_report_and_recover(q2, x8, R, C, ntok):
    """The issuing warps' waits for a block are cut to one poll: rows come out NaN, the error word says so, and the
    next call is right again.  A CTA of 128 x 4096 sums its tile over a cluster, one of 4096 x 1024 on its own."""
    d = synth.int4(R, C, 128, 740, True)
    pk = q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], 128))
    if x8:
        xn, xs = synth.activations8(ntok, C, 741)
        args, x = (torch.from_numpy(xn).cuda(), torch.from_numpy(xs).cuda()), xn * xs.astype(np.float64)[:, None]
    else:
        x = synth.activations(ntok, C, 741)
        args = (torch.from_numpy(x).cuda(),)
    call = pk.gemv_x8 if x8 else pk.gemv
    q2.debug_wait_limit(1)
    try:
        y = call(*args)
        torch.cuda.synchronize()
    finally:
        q2.debug_wait_limit(0)
    assert q2.device_errors() != 0
    assert torch.isnan(y).any()
    y = call(*args)
    torch.cuda.synchronize()
    assert q2.device_errors() == 0
    _check(y, d, x, x8)
