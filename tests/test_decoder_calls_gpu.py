"""The decoder operators' calls: arguments that end in an exception, and leave the process and the GPU usable."""
import subprocess
import sys

import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

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


def test_outputs_on_inputs_on_one_another_or_on_themselves_are_refused():
    q, k, v = (torch.randn(2, n, h, 64, device=DEV) for n, h in ((40, 4), (90, 2), (90, 2)))
    out, lse = api.gs_cross_attention_fwd(q, k, v)
    dout = torch.randn_like(q)
    fresh = lambda: [torch.empty_like(t) for t in (q, k, v)]  # noqa: E731
    dq, dk, dv = fresh()
    bad = [lambda: api.gs_cross_attention_fwd(q, k, v, out=(q, lse)),
           lambda: api.gs_cross_attention_fwd(q, k, v, out=(torch.empty(2, 40, 1, 64, device=DEV).expand(-1, -1, 4, -1), lse)),
           lambda: api.gs_cross_attention_fwd(q, k, v, out=(torch.empty(1, 40, 4, 64, device=DEV).expand(2, -1, -1, -1), lse))]
    for grads in ((q, dk, dv), (dout, dk, dv), (out, dk, dv), (dq, k, dv), (dq, dk, v), (dq, v, dv), (dq, dk, dk),
                  (dq, dk, torch.empty(2, 1, 2, 64, device=DEV).expand(-1, 90, -1, -1))):
        bad.append(lambda g=grads: api.gs_cross_attention_bwd(dout, q, k, v, out, lse, grads=g))
    x = torch.randn(50, 128, device=DEV)
    over = x.as_strided((30, 64), (128, 1))
    stats = [torch.empty(30, device=DEV) for _ in range(2)]
    bad.append(lambda: api.gs_layer_norm_fwd(over, out=(x.as_strided((30, 64), (100, 1)), *stats)))
    for call in bad:
        with pytest.raises(_abi.GsError, match="lies on|share memory"):
            call()
    # interleaved in one buffer, elements of their own
    both = torch.empty(2, 90, 4, 64, device=DEV)
    grads = api.gs_cross_attention_bwd(dout, q, k, v, out, lse, grads=(dq, both[:, :, :2], both[:, :, 2:]))
    want = api.gs_cross_attention_bwd(dout, q, k, v, out, lse)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("scale", [1e-50, 1e-46, 1e39, float("inf"), float("nan"), -1.0, 0.0])
def test_scales_that_are_none_in_float32_are_refused(scale):
    q = torch.randn(1, 5, 2, 16, device=DEV)
    with pytest.raises(ValueError, match="scale"):
        api.gs_cross_attention_fwd(q, q.clone(), q.clone(), scale=scale)


def test_a_scene_without_tokens_has_the_gaussians_of_the_queries_alone():
    from differentiable_gaussian_splatting_gs_gb300 import decoder

    n = 20
    base = {"mean3d": torch.zeros(n, 3, device=DEV), "log_scale": torch.zeros(n, 3, device=DEV), "quat": torch.ones(n, 4, device=DEV),
            "opacity_logit": torch.zeros(n, device=DEV), "sh": torch.zeros(n, 1, 3, device=DEV)}
    d = decoder.GaussianDecoder(base, 24, channels=16, heads=2, head_dim=8)
    none = d.forward(torch.zeros(1, 0, 24, device=DEV))
    masked = d.forward(torch.randn(1, 30, 24, device=DEV), k_len=torch.zeros(1, dtype=torch.int32, device=DEV))
    assert all(torch.equal(none[k], masked[k]) for k in none)
    grads = {k: torch.randn_like(v) for k, v in none.items()}
    d.backward(grads)
    want = {k: v.clone() for k, v in d.grads.items()}
    d.forward(torch.zeros(1, 0, 24, device=DEV))
    assert d.backward(grads).shape == (1, 0, 24)
    assert all(torch.equal(d.grads[k], want[k]) for k in want)
