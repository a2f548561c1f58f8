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



def _counted(monkeypatch, product):
    """The operands' shapes of the 8-bit products that the decoder asks for, each answered by `product`."""
    calls = []

    def count(a, a_scale, b, b_scale, dtype=None, out=None):
        calls.append((tuple(a.shape), tuple(b.shape)))
        return product(a, a_scale, b, b_scale, dtype=dtype, out=out)

    monkeypatch.setattr(decoder.api, "gs_matmul_fp8", count)
    return calls


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_every_projection_and_both_of_its_gradients_are_8_bit_products(norm, monkeypatch):
    n, length, tokens_c, c, inner, inner_kv = 77, 150, 96, 200, 160, 80
    d, tokens, grads = _decoder(n, norm=norm, fp8=True, dtype=torch.bfloat16)
    calls = _counted(monkeypatch, api.gs_matmul_fp8)
    d.forward(tokens)
    forward = [((n, c), (inner, c)), ((length, tokens_c), (inner_kv, tokens_c)), ((length, tokens_c), (inner_kv, tokens_c)), ((n, inner), (c, inner))]
    assert sorted(calls) == sorted(forward)
    calls.clear()
    d.backward(grads)
    back = []
    for (rows, inputs), (outputs, _) in forward:
        back += [((inputs, rows), (outputs, rows)), ((rows, outputs), (inputs, outputs))]
    assert sorted(calls) == sorted(back)
    calls.clear()
    state = d.serving()
    assert calls == forward[:1]
    calls.clear()
    d.serve(tokens, state)
    assert sorted(calls) == sorted(forward[1:])


def test_without_fp8_there_are_none(monkeypatch):
    d, tokens, grads = _decoder(77, norm="rms", dtype=torch.bfloat16)
    calls = _counted(monkeypatch, api.gs_matmul_fp8)
    d.forward(tokens)
    d.backward(grads)
    assert calls == []


def test_results_are_the_products(monkeypatch):
    # every product's result reaches the outputs: answered by zeros, the Gaussians and gradients change
    d, tokens, grads = _decoder(77, norm="rms", fp8=True)
    params = d.forward(tokens)
    d.backward(grads)
    want = {k: v.clone() for k, v in d.grads.items()}
    calls = _counted(monkeypatch, lambda a, sa, b, sb, dtype=None, out=None: out.zero_() if out is not None else torch.zeros(len(a), len(b), device=DEV, dtype=dtype))
    other = d.forward(tokens)
    d.backward(grads)
    assert len(calls) == 12 and all((d.grads[k] == 0).all() and (want[k] != 0).any() for k in PROJECTIONS)
    assert all(not torch.equal(other[k], params[k]) for k in params)
