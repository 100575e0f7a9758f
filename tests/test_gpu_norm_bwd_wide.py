"""The norm's backward at row widths around the borders of its shared-memory use, each as the
first launch of a fresh process: a kernel's shared-memory limit, once raised, stays raised, so a
wider row that ran before would hide a launch that is refused."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# every type and both access forms are kernels of their own, so one process runs them all; widths
# ascend, as a wider one would raise the limit for those after it
SCRIPT = """
import sys
import torch
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import fp8_ref as R
import hybrid_masked_attention_b200 as M
from fp8_ref import HALF, U
F32, BF16 = torch.float32, torch.bfloat16
g = torch.Generator(device="cuda").manual_seed(3)
rnd = lambda t, *s: torch.randn(*s, generator=g, device="cuda").to(t)
for dim in {dims}:
    for xt, yt, rt in ((F32, F32, F32), (F32, BF16, None), (BF16, BF16, BF16), (BF16, F32, None)):
        for pitch in (dim, dim + 1):
            rows = 5
            mat = lambda t: rnd(t, rows, pitch)[:, :dim]
            x, dy, w = mat(xt), mat(yt), 1 + 0.3 * rnd(F32, dim)
            dres = None if rt is None else mat(rt)
            rstd = torch.rsqrt(x.float().square().mean(1) + 1e-6)
            dx, dw = mat(xt), torch.full((dim,), 7.0, device="cuda")
            ws = torch.empty(M.rmsnorm_bwd_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda")
            M.rmsnorm_bwd(x, w, rstd, dy, dres, dx, dw, ws)
            rx, rw = R.rmsnorm_bwd(x, w, rstd, dy, dres)
            X, G, r = x.double().abs(), (dy.double() * w.double()).abs(), rstd.double()[:, None]
            res = 0 if dres is None else dres.double().abs()
            # a lane adds at most 32 terms, then 5 shuffles and up to 16 warps; 8 for the factors
            tol = r * (4 * U * G + X * r * r * (G * X).mean(1, keepdim=True) * 61 * U) + 3 * U * (res + rx.abs())
            assert ((dx.double() - rx).abs() <= tol + HALF[xt] * rx.abs()).all(), (dim, xt, yt, rt, pitch)
            assert ((dw.double() - rw).abs() <= (rows + 40) * U * (dy.double().abs() * X * r).sum(0)).all(), (dim, xt, yt, rt)
print("done")
"""


@pytest.mark.parametrize("dims", [[6128, 6129, 6144, 6145], [12256, 12257, 12288, 12289, 16384], [4096, 4097, 8192, 8193]], ids=str)
def test_first_launch_at_a_border(dims, cuda_ok):
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, dims=dims)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "done" in r.stdout, (r.stdout + r.stderr)[-2000:]
