"""A launch that CUDA refuses is an error of that call alone: nothing of it is left for the program's next call."""

import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

# The launches are refused because the stream's capture has been invalidated (by a host call that a capture does not
# allow): an error of the runtime, nothing reaches the GPU.
CODE = """
import ctypes, re, torch
from weight_linear_attention_gb300 import falcon as F

B, H, T, d = 2, 3, 700, 64
x, g, z, o, dx, dz = (torch.randn(B, H, T, d, device="cuda").bfloat16() for _ in range(6))
h, w, dw, db = torch.zeros(B, H, d, device="cuda"), *(torch.ones(H, d, device="cuda") for _ in range(3))
dims, one = F.make_seq_dims(B, H, T, d), F.make_seq_dims(B, H, 1, d)
ws = torch.empty(F.falcon_gn_bwd_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
q = torch.randn(B, H, 128, d, device="cuda").bfloat16()
b = torch.rand(B, H, 128, device="cuda")
calls = {
    "glr_fwd": lambda s: F.falcon_glr_fwd(2, x, g, h, None, o, None, dims, stream=s),
    "glr_fwd T=1": lambda s: F.falcon_glr_fwd(2, x, g, h, None, o, None, one, stream=s),
    "glr_bwd": lambda s: F.falcon_glr_bwd(2, x, g, z, h, None, o, None, dx, dz, None, dims, stream=s),
    "glr_bwd T=1": lambda s: F.falcon_glr_bwd(2, x, g, z, h, None, o, None, dx, dz, None, one, stream=s),
    "glr_bwd T=0": lambda s: F.falcon_glr_bwd(2, None, None, None, None, None, None, None, None, None, h,
                                              F.make_seq_dims(B, H, 0, d), stream=s),
    "gn_fwd": lambda s: F.falcon_gn_fwd(1, x, z, w, None, None, o, dims, stream=s),
    "gn_bwd": lambda s: F.falcon_gn_bwd(1, x, z, w, None, None, g, dx, dz, dw, db, dims, workspace=ws, stream=s),
    "gn_bwd T=0": lambda s: F.falcon_gn_bwd(1, None, None, w, None, None, None, None, None, dw, db,
                                            F.make_seq_dims(B, H, 0, d), stream=s),
}
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
for name, call in calls.items():
    assert call(s.cuda_stream) == F.FALCON_OK, name
torch.cuda.synchronize()
path = [l.split()[-1] for l in open("/proc/self/maps") if re.search(r"/libcudart\\.so", l)]
assert len(set(path)) == 1, path  # the library and torch share one runtime, and so its last error
rt = ctypes.CDLL(path[0])
handle, graph = ctypes.c_void_p(s.cuda_stream), ctypes.c_void_p()
left = {}
for name, call in calls.items():
    assert rt.cudaStreamBeginCapture(handle, 2) == 0
    assert rt.cudaStreamSynchronize(handle) != 0
    rt.cudaGetLastError()
    assert call(s.cuda_stream) == F.FALCON_ERR_CUDA, name
    left[name] = rt.cudaGetLastError()
    assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
    rt.cudaGetLastError()
    assert call(s.cuda_stream) == F.FALCON_OK, name
torch.cuda.synchronize()
assert F.falcon_device_status() == F.FALCON_OK
bad = {k: v for k, v in left.items() if v}
assert not bad, bad
F.forward("falcon1", q, q, q, b, b)
torch.cuda.synchronize()
print("clean")
"""


def test_a_refused_launch_leaves_no_error_behind():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "clean" in r.stdout, r.stderr[-2000:]
