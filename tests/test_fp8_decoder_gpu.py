"""The Gaussian decoder with the root-mean-square norm, 8-bit products and clipping: its gradients against torch's autograd in
float64, its 8-bit products against those of the values that their operands stand for.

Tolerances. Gradients with float32 products: as the layer norm's decoder, a chain of a dozen float32 operators, 2e-4 of the
tensor's largest magnitude. 8-bit products against products in float64 of the same 8-bit operands: the operands' inputs differ
by float32 roundings, so that a value next to a border may round the other way, by 2^-3 of itself. That happens to one in a
hundred thousand of them, and each is one of 64 or more terms of similar size: 2^-3 / 8 of the largest sum.
"""
import numpy as np
import pytest
import torch

import gs_scenes

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import api, decoder  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _base(n):
    scene = gs_scenes.make_scene(0)
    names = ("mean3d", "log_scale", "quat", "opacity_logit")
    base = {k: torch.from_numpy(np.ascontiguousarray(getattr(scene, k)[:n])).to(DEV) for k in names}
    base["sh"] = torch.zeros(n, 1, 3, device=DEV)
    return base


def _inputs(d, length, channels, masked=True):
    gen = torch.Generator(device=DEV).manual_seed(3)
    tokens = torch.randn(1, length, channels, device=DEV, generator=gen)
    mask = torch.rand(1, length, device=DEV, generator=gen) < 0.8 if masked else None
    grads = {k: torch.randn(v.shape, device=DEV, generator=gen) for k, v in d.base.items()}
    return tokens, mask, grads


def _run(d, tokens, mask, grads):
    params = d.forward(tokens, key_mask=mask)
    dtokens = d.backward(grads)
    return params, {**{k: v.clone() for k, v in d.grads.items()}, "tokens": dtokens}


@pytest.mark.parametrize("n,length,heads,kv_heads,head_dim", [(300, 400, 4, 4, 32), (77, 101, 6, 2, 40), (1, 64, 2, 2, 64)])
def test_rms_gradients_against_autograd_in_64_bits(n, length, heads, kv_heads, head_dim):
    d = decoder.GaussianDecoder(_base(n), 96, channels=80, heads=heads, kv_heads=kv_heads, head_dim=head_dim, norm="rms")
    assert not any("bias" in k for k in d.weights)
    for name in ("norm_q_weight", "norm_t_weight", "norm_x_weight"):
        d.weights[name].add_(0.3 * torch.randn_like(d.weights[name]))
    tokens, mask, grads = _inputs(d, length, 96)
    params, got = _run(d, tokens, mask, grads)
    w = {k: v.double().requires_grad_() for k, v in d.weights.items()}
    tok = tokens[0].double().requires_grad_()
    norm = lambda x, name: x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w[f"norm_{name}_weight"]  # noqa: E731
    spread = lambda x, m: x.view(x.shape[0], m, head_dim).repeat_interleave(heads // m, 1)  # noqa: E731
    t = norm(tok, "t")
    q, k, v = spread(norm(w["queries"], "q") @ w["wq"], heads), spread(t @ w["wk"], kv_heads), spread(t @ w["wv"], kv_heads)
    s = torch.einsum("ihd,jhd->hij", q, k) * head_dim ** -0.5
    a = torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(~mask[0][None, None], -float("inf")), 2), v).reshape(n, -1)
    out = norm(w["queries"] + a @ w["wo"], "x") @ w["wh"] + w["bh"]
    (out * torch.cat([grads[name].reshape(n, -1) for name in decoder.PARTS], 1).double()).sum().backward()
    offsets = torch.cat([(params[k] - d.base[k]).reshape(n, -1) for k in decoder.PARTS], 1)
    size = torch.cat([d.base[k].abs().reshape(n, -1) for k in decoder.PARTS], 1)  # rounding of base + offset
    assert ((offsets - out).abs() <= 2e-4 * out.abs().max() + 2.0 ** -23 * size).all()
    for name, g in {**{k: x.grad for k, x in w.items()}, "tokens": tok.grad}.items():
        assert (got[name].view_as(g) - g).abs().max() <= 2e-4 * g.abs().max(), name


def _values(q, scale):
    block = 1 if scale.shape[0] == q.shape[0] else 128
    return q.double() * scale.double().repeat_interleave(block, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def _product(a, a_scale, b, b_scale, dtype=None, out=None):
    got = _values(a, a_scale) @ _values(b, b_scale).t()
    return got.to(dtype) if out is None else out.copy_(got)


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("n,length,dtype", [(300, 400, torch.float32), (33, 129, torch.float32), (200, 300, torch.bfloat16)])
def test_8_bit_products_forward_and_backward(norm, n, length, dtype, monkeypatch):
    d = decoder.GaussianDecoder(_base(n), 96, channels=128, heads=4, kv_heads=2, head_dim=32, norm=norm, fp8=True, dtype=dtype)
    tokens, mask, grads = _inputs(d, length, 96)
    before = api.gs_kernel_launches()
    params, got = _run(d, tokens, mask, grads)
    assert api.gs_kernel_launches() - before >= 12  # twelve products among them
    served = d.serve(tokens, d.serving(), key_mask=mask)
    monkeypatch.setattr(decoder.api, "gs_matmul_fp8", _product)
    want_params, want = _run(d, tokens, mask, grads)
    # bfloat16 activations round the other way too, by 2^-8 of themselves
    bound = 2.0 ** -6 if dtype == torch.float32 else 2.0 ** -6 + 8 * 2.0 ** -8
    for name in want:
        assert (got[name] - want[name]).abs().max() <= bound * want[name].abs().max(), name
    for name in params:
        offset = (want_params[name] - d.base[name]).abs().max()
        assert (params[name] - want_params[name]).abs().max() <= bound * offset, name
        assert (served[name] - params[name]).abs().max() <= (bound + 2.0 ** -6) * offset, name
    assert api.gs_device_error() == 0


def test_without_tokens_and_with_one_gaussian():
    d = decoder.GaussianDecoder(_base(1), 96, channels=64, heads=2, head_dim=32, norm="rms", fp8=True)
    tokens, _, grads = _inputs(d, 0, 96, False)
    params, got = _run(d, tokens, None, grads)
    assert got["tokens"].shape == (1, 0, 96) and (got["wk"] == 0).all() and (got["wq"] == 0).all()
    served = d.serve(tokens, d.serving())
    assert all(torch.equal(served[k], params[k]) for k in params)


@pytest.mark.parametrize("kw", [dict(), dict(norm="rms"), dict(norm="rms", fp8=True, dtype=torch.bfloat16)])
def test_training_steps_with_clipping(kw):
    scene = gs_scenes.make_scene(0)
    n = 300
    d = decoder.GaussianDecoder(_base(n), 64, channels=64, heads=2, head_dim=32, **kw)
    tokens, _, _ = _inputs(d, 70, 64, False)
    target = torch.rand(3, scene.cameras[0].height, scene.cameras[0].width, device=DEV)
    plain, clipped = decoder.DecoderTrainer(d), decoder.DecoderTrainer(d, max_norm=1e-3)
    plain.step(tokens, [scene.cameras[0]], [target])
    assert plain.grad_norm is None
    for _ in range(3):
        clipped.step(tokens, [scene.cameras[0]], [target])
        after = torch.stack([g.double().square().sum() for g in d.grads.values()]).sum().sqrt()
        norm = float(clipped.grad_norm)
        assert norm > 1e-3 and abs(float(after) / (1e-3 * norm / (norm + 1e-6)) - 1) <= 1e-6
    assert all(torch.isfinite(w).all() for w in d.weights.values()) and api.gs_device_error() == 0


def test_serving_captured_into_a_graph():
    d = decoder.GaussianDecoder(_base(200), 96, channels=128, heads=4, head_dim=32, norm="rms", fp8=True, dtype=torch.bfloat16)
    tokens, _, _ = _inputs(d, 300, 96, False)
    state = d.serving()
    want = d.serve(tokens, state)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = d.serve(tokens, state)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    other = torch.randn_like(tokens)
    want = d.serve(other, state)
    tokens.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_norms_that_there_are_not():
    with pytest.raises(ValueError, match="norm"):
        decoder.GaussianDecoder(_base(4), 24, norm="batch")
