"""The binding loads on a torch without GPU support, which lacks private functions of the others."""
import os
import subprocess
import sys
import types

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    del torch._C._cuda_getCurrentRawStream
from combine_ep_route_topk_amd import ep
assert ep.ep_abi_version() > 0
try:
    ep.ep_quantize_fp8(torch.zeros((4, 32), dtype=torch.bfloat16))
except ValueError as e:
    assert "GPU" in str(e)
else:
    raise AssertionError("a host tensor was taken")
"""


def test_import_without_gpu_support():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


def test_current_stream_without_the_short_way(monkeypatch):
    import torch
    from combine_ep_route_topk_amd import ep
    monkeypatch.setattr(ep, "_current_handle", None)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device: types.SimpleNamespace(cuda_stream=4096 + device.index))
    assert ep._stream(None, torch.device("cuda", 3)) == 4099
    assert ep._stream(7, torch.device("cuda", 3)) == 7
