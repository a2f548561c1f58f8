"""Which products the Gaussian decoder runs in 8 bits, and of which weights."""
import numpy as np
import pytest
import torch

import gs_scenes

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import api, decoder  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
PROJECTIONS = ("wq", "wk", "wv", "wo")


def _decoder(n, **kw):
    scene = gs_scenes.make_scene(0)
    base = {k: torch.from_numpy(np.ascontiguousarray(getattr(scene, k)[:n])).to(DEV) for k in ("mean3d", "log_scale", "quat", "opacity_logit")}
    base["sh"] = torch.zeros(n, 1, 3, device=DEV)
    d = decoder.GaussianDecoder(base, 96, channels=200, heads=4, kv_heads=2, head_dim=40, **kw)
    gen = torch.Generator(device=DEV).manual_seed(3)
    return d, torch.randn(1, 150, 96, device=DEV, generator=gen), {k: torch.randn(v.shape, device=DEV, generator=gen) for k, v in base.items()}


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_backwards_8_bit_weights_are_the_forwards(norm, dtype):
    d, tokens, grads = _decoder(77, norm=norm, fp8=True, dtype=dtype)
    d.forward(tokens)
    dtokens = d.backward(grads)
    want = {k: v.clone() for k, v in d.grads.items()}
    d.forward(tokens)
    for name in PROJECTIONS:
        d.weights[name].mul_(-3).add_(1)
    got = d.backward(grads)
    assert torch.equal(got, dtokens) and all(torch.equal(d.grads[k], want[k]) for k in want)

