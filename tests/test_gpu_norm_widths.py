"""``q2_rmsnorm`` of wide rows that begin anywhere, each as the first call of its process: the outputs' images take
44 to 48 KB of shared memory at these widths, and what a wider call has asked for before must not matter.

Tolerances as in test_gpu_norm.py.
"""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CODE = """
import numpy as np, torch
import dequant_gemv_q2_gb300 as q2
from oracle import norm as onorm
C, gap, residual, fp16, int8 = {C}, {gap}, {residual}, {fp16}, {int8}
rng = np.random.default_rng(C)
x, r = (rng.normal(size=(3, C)).astype(np.float16) for _ in range(2))
w = (1 + 0.3 * rng.normal(size=C)).astype(np.float16)
wide = torch.zeros((3, C + gap), dtype=torch.float16, device="cuda")
xd = wide[:, :C]
xd.copy_(torch.from_numpy(x))
rd = torch.from_numpy(r).cuda() if residual else None
out = torch.empty((3, C), dtype=torch.float16, device="cuda") if fp16 else None
q8 = torch.empty((3, C), dtype=torch.int8, device="cuda") if int8 else None
s8 = torch.empty(3, device="cuda") if int8 else None
q2.RmsNorm(w).apply(xd, residual=rd, out=out, out8=q8, scale8=s8)
h, y = onorm.rmsnorm_f64(x, w, 1e-6, r if residual else None)
f64 = lambda t: t.cpu().numpy().astype(np.float64)
if residual: assert (np.abs(f64(rd) - h) <= (2.0 ** -11 + 2.0 ** -18) * np.abs(h) + 2.0 ** -25).all()
if fp16: assert (np.abs(f64(out) - y) <= (2.0 ** -11 + 2.0 ** -18) * np.abs(y) + 2.0 ** -25).all()
if int8: assert (np.abs(f64(q8) * f64(s8)[:, None] - y) <= (0.5 + 127 * 2.0 ** -17) * f64(s8)[:, None]).all()
"""


@pytest.mark.parametrize("C,gap,residual,fp16,int8", [
    (9737, 0, True, True, True), (9824, 1, True, True, True), (12288, 1, True, True, False), (12167, 0, True, True, False),
    (16383, 0, True, False, True), (16384, 3, False, True, True), (24575, 0, False, True, False), (24321, 0, False, True, False)])
def test_first_call_of_a_process(C, gap, residual, fp16, int8):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = CODE.format(C=C, gap=gap, residual=residual, fp16=fp16, int8=int8)
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
