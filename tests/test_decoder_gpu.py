"""The Gaussian decoder on the GPU: its gradients against torch's autograd of the same model in float64, and training
through the rasterizer.

Tolerance of the gradients: each is a chain of a dozen float32 operators, the worst of them sums of up to 400 products
in float32 (relative error of the sum's magnitude 2^-20); the bound is 2e-4 of the tensor's largest magnitude, as the
rasterizer's end-to-end gradients are compared.
"""
import numpy as np
import pytest
import torch

import gs_scenes

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import api, decoder, step  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _base(scene, n):
    names = ("mean3d", "log_scale", "quat", "opacity_logit")
    base = {k: torch.from_numpy(np.ascontiguousarray(getattr(scene, k)[:n])).to(DEV) for k in names}
    base["sh"] = torch.zeros(n, 1, 3, device=DEV)
    return base


def _reference(d, tokens, valid, grads):
    """Gradients of sum(parameters * grads) by autograd of the model's definition in float64."""
    w = {k: v.double().requires_grad_() for k, v in d.weights.items()}
    tok = tokens[0].double().requires_grad_()

    def norm(x, name):
        return torch.nn.functional.layer_norm(x, x.shape[-1:], w[f"norm_{name}_weight"], w[f"norm_{name}_bias"], 1e-5)

    t = norm(tok, "t")
    heads = lambda x, n: x.view(x.shape[0], n, d.head_dim).repeat_interleave(d.heads // n, 1)  # noqa: E731
    q = heads(norm(w["queries"], "q") @ w["wq"], d.heads)
    k, v = heads(t @ w["wk"], d.kv_heads), heads(t @ w["wv"], d.kv_heads)
    s = torch.einsum("ihd,jhd->hij", q, k) * d.head_dim ** -0.5
    p = torch.softmax(s.masked_fill(~valid[0][None, None], -float("inf")), 2)
    a = torch.einsum("hij,jhd->ihd", p, v).reshape(d.n, -1)
    out = norm(w["queries"] + a @ w["wo"], "x") @ w["wh"] + w["bh"]
    dout = torch.cat([grads[name].reshape(d.n, -1) for name in decoder.PARTS], 1).double()
    (out * dout).sum().backward()
    return {k: v.grad for k, v in w.items()}, tok.grad, out


@pytest.mark.parametrize("n,length,heads,kv_heads,head_dim", [(300, 400, 4, 4, 32), (77, 101, 6, 2, 40), (1, 64, 2, 2, 64)])
def test_gradients_against_autograd_in_64_bits(n, length, heads, kv_heads, head_dim):
    d = decoder.GaussianDecoder(_base(gs_scenes.make_scene(0), n), 96, channels=80, heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    gen = torch.Generator(device=DEV).manual_seed(3)
    tokens = torch.randn(1, length, 96, device=DEV, generator=gen)
    mask = torch.rand(1, length, device=DEV, generator=gen) < 0.8
    params = d.forward(tokens, key_mask=mask)
    grads = {k: torch.randn(v.shape, device=DEV, generator=gen) for k, v in params.items()}
    dtokens = d.backward(grads)
    want, dtok, out = _reference(d, tokens, mask, grads)
    got = torch.cat([(params[k] - d.base[k]).reshape(n, -1) for k in decoder.PARTS], 1)
    scale = torch.cat([d.base[k].abs().reshape(n, -1) for k in decoder.PARTS], 1)  # rounding of base + offset
    assert ((got - out).abs() <= 2e-4 * out.abs().max() + 2.0 ** -23 * scale).all()
    for name, g in want.items():
        assert (d.grads[name] - g).abs().max() <= 2e-4 * g.abs().max(), name
    assert (dtokens[0] - dtok).abs().max() <= 2e-4 * dtok.abs().max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_through_the_rasterizer_lowers_the_loss(dtype):
    scene = gs_scenes.make_scene(0)
    n = 1000
    params = {k: torch.from_numpy(np.ascontiguousarray(getattr(scene, k)[:n])).to(DEV)
              for k in ("mean3d", "log_scale", "quat", "opacity_logit", "sh")}
    opt, cam = api.make_options(scene.sh_degree), scene.cameras[0]
    buffers = step.StepBuffers(n, DEV)
    proj = api.gs_preprocess(params, cam, opt, out=buffers.proj)
    b = api.gs_bin_and_sort(proj, cam, opt, buffers=buffers.sort)
    target = api.gs_render_fwd(proj, b.vals, b.ranges, cam, opt)[0].clone()
    d = decoder.GaussianDecoder(_base(scene, n), 64, channels=64, heads=2, head_dim=32, dtype=dtype)
    tokens = torch.randn(1, 64, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    k_len = torch.tensor([60], dtype=torch.int32, device=DEV)
    trainer = decoder.DecoderTrainer(d)
    losses = []
    for _ in range(40):
        image = trainer.step(tokens, [cam], [target], k_len=k_len)
        losses.append(float((image - target).square().sum()))
    assert np.isfinite(losses).all() and losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])
    assert api.gs_device_error() == 0
