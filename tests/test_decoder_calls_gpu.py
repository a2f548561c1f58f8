"""The decoder operators' calls: arguments that end in an exception, and leave the process and the GPU usable."""
import subprocess
import sys

import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

WITHOUT_MEMORY = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from differentiable_gaussian_splatting_gs_gb300 import _abi, api
x, q = torch.randn(4, 8, device="cuda"), torch.randn(1, 5, 2, 16, device="cuda")
y, mean, rstd = api.gs_layer_norm_fwd(x)
out, lse = api.gs_cross_attention_fwd(q, q, q)
with FakeTensorMode():
    fx, fq = torch.empty(4, 8, device="cuda"), torch.empty(1, 5, 2, 16, device="cuda")
raised = 0
for call in (lambda: api.gs_layer_norm_fwd(fx), lambda: api.gs_layer_norm_bwd(fx, x, mean, rstd),
             lambda: api.gs_cross_attention_fwd(q, fq, q), lambda: api.gs_cross_attention_bwd(q, q, q, fq, out, lse)):
    try:
        call()
    except (RuntimeError, ValueError, TypeError):
        raised += 1
assert raised == 4, raised
assert torch.equal(api.gs_layer_norm_fwd(x)[0], y) and torch.equal(api.gs_cross_attention_fwd(q, q, q)[0], out)
assert api.gs_device_error() == _abi.GS_OK
print("usable")
"""


def test_tensors_without_memory_raise():
    # in a process of its own: an exception that leaves the interpreter without its lock ends it
    r = subprocess.run([sys.executable, "-c", WITHOUT_MEMORY], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("usable"), (r.returncode, r.stderr[-2000:])
