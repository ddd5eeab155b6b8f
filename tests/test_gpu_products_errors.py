"""A launch that fails is reported by its own call and by no later one."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import ctypes, torch
import fine_grained_moe_gemm_b200 as moe
t = lambda *s, d=torch.bfloat16: torch.ones(s, dtype=d, device="cuda")
x, w, y = t(20, 64), t(1, 48, 64), t(20, 48)
xl, wl, yl = t(6000, 64), t(2, 4096, 64), t(6000, 4096)
off = torch.tensor([0, 3000, 6000], dtype=torch.int32, device="cuda")
dw, none = t(1, 48, 64, d=torch.float32), t(0, 64)
rt = ctypes.CDLL("libcudart.so.12")
torch.cuda.synchronize()
calls = [lambda s: moe.moe_grouped_mm(x, w, None, y, stream=s), lambda s: moe.moe_grouped_mm(xl, wl, off, yl, stream=s),
         lambda s: moe.moe_grouped_wgrad(none[:, :48], none, None, dw, stream=s)]
for call in calls:
    call(None)          # kernels loaded, attributes set
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h = ctypes.c_void_p(s.cuda_stream)
    # a capture that a synchronisation ended: every launch into it is refused by the runtime
    assert rt.cudaStreamBeginCapture(h, 2) == 0
    assert rt.cudaStreamSynchronize(h) != 0
    rt.cudaGetLastError()
    try:
        call(s)
        raise SystemExit("the launch was not refused")
    except moe.MoeError as e:
        assert e.status == moe.MOE_ERR_CUDA
    left = rt.cudaPeekAtLastError()
    g = ctypes.c_void_p()
    rt.cudaStreamEndCapture(h, ctypes.byref(g))
    rt.cudaGetLastError()
    assert left == 0, left
    call(None)
    moe.moe_swiglu(y, y, t(20, 48))
    torch.cuda.synchronize()
assert moe.device_error() == 0
print("fine")
"""


def test_failed_launch_leaves_no_error_behind():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr[-2000:]
