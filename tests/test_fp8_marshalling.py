"""The 8-bit operators' Python wrappers with and without the marshalling in C (csrc/fastcall.c)."""
import os
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "hybrid_masked_attention_b200")

WITHOUT = "import sys; sys.path.insert(0, {root!r}); sys.modules['hybrid_masked_attention_b200._fastcall'] = None\n"


def run(code, timeout=300):
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=timeout)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    return r.stdout


def test_package_without_the_c_marshalling():
    """The package imports, and its wrappers make their checks, without the extension and without
    torch's internal names."""
    out = run(WITHOUT.format(root=ROOT) + """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import hybrid_masked_attention_b200 as M
x = torch.zeros(4, 64)
q, s = x.to(torch.float8_e4m3fn), torch.zeros(4, 1)
for call in (lambda: M.fp8_quant(x, q, s), lambda: M.add_rmsnorm_fp8(x, None, torch.ones(64), None, q, s),
             lambda: M.fp8_gemm(q, s, q, s, x, torch.zeros(1, dtype=torch.int32))):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("not refused")
print("ok")
""")
    assert "ok" in out


def test_extension_is_named_for_its_interpreter():
    """Another interpreter must not load it: the file carries the ABI tag, and none without is left."""
    sys.path.insert(0, PKG)
    try:
        import build
    finally:
        sys.path.remove(PKG)
    build.build_fastcall()
    assert build.FASTCALL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.exists(build.FASTCALL)
    assert not os.path.exists(os.path.join(PKG, "_fastcall.so"))


def test_other_threads_run_while_an_entry_point_blocks():
    """An entry point that blocks (libc's sleep in the place of the quantiser: its first argument
    is the number of rows) does not hold the interpreter's lock."""
    out = run("""
import ctypes
import sys
import threading
import time
sys.path.insert(0, {pkg!r})
import _fastcall
f32, bf16, f8, u8, i32 = object(), object(), object(), object(), object()
class Matrix:   # as much of a tensor on device 0 as the marshalling reads
    def __init__(self, dtype, rows, cols):
        self.dtype, self.shape = dtype, (rows, cols)
    def get_device(self):
        return 0
    def stride(self):
        return self.shape[1], 1
    def data_ptr(self):
        return 4096
sleep = ctypes.cast(ctypes.CDLL(None).sleep, ctypes.c_void_p).value
_fastcall.setup(f32, bf16, f8, u8, i32, lambda: 0, lambda dev: 0, *[sleep] * 5)
ticks, end = [], threading.Event()
def count():
    while not end.is_set():
        ticks.append(time.perf_counter())
        time.sleep(0.01)
t = threading.Thread(target=count)
t.start()
t0 = time.perf_counter()
status = _fastcall.fp8_quant(Matrix(f32, 1, 128), Matrix(f8, 1, 128), Matrix(f32, 1, 1), 1)
t1 = time.perf_counter()
end.set()
t.join()
assert status == 0 and t1 - t0 > 0.9, (status, t1 - t0)
print(sum(t0 + 0.2 < v < t1 - 0.2 for v in ticks))
""".format(pkg=PKG))
    assert int(out) >= 5


@pytest.mark.gpu
def test_same_results_without_the_c_marshalling(cuda_ok):
    code = """
import hashlib
import torch
import hybrid_masked_attention_b200 as M
F8 = torch.float8_e4m3fn
g = torch.Generator(device="cuda").manual_seed(1)
x, w = torch.randn(300, 256, generator=g, device="cuda"), torch.randn(256, generator=g, device="cuda")
new = lambda r, c, t: torch.empty(r, c, dtype=t, device="cuda")
q, s, rstd = new(300, 256, F8), new(300, 2, torch.float32), torch.empty(300, device="cuda")
b, bs = new(256, 256, F8), new(2, 2, torch.float32)
out, status = new(300, 256, torch.float32), torch.zeros(1, dtype=torch.int32, device="cuda")
dx, dw = torch.empty_like(x), torch.empty_like(w)
M.add_rmsnorm_fp8(x, None, w, None, q, s, rstd)
M.fp8_quant(x[:256].contiguous(), b, bs, 128)
M.fp8_gemm(q, s, b, bs, out, status, "silu")
M.rmsnorm_bwd(x, w, rstd, out, None, dx, dw, torch.empty(M.rmsnorm_bwd_workspace_bytes(300, 256), dtype=torch.uint8, device="cuda"))
M.fp8_check(status)
print(hashlib.sha256(b"".join(t.cpu().contiguous().view(torch.uint8).numpy().tobytes() for t in (q, s, out, dx, dw))).hexdigest())
"""
    path = "import sys; sys.path.insert(0, {root!r})\n"
    assert run(path.format(root=ROOT) + code) == run(WITHOUT.format(root=ROOT) + code)
