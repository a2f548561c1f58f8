"""The float64 layer norm and cross attention that the GPU tests compare with, pinned by torch's autograd of
the definition, by differences, and by closed forms (CPU)."""
import numpy as np
import pytest
import torch

from oracle import decoder


def _case(seed, b=2, lq=5, lk=7, h=4, hk=2, d=6):
    g = np.random.default_rng(seed)
    q, do = g.standard_normal((b, lq, h, d)), g.standard_normal((b, lq, h, d))
    k, v = g.standard_normal((b, lk, hk, d)), g.standard_normal((b, lk, hk, d))
    valid = g.random((b, lk)) < 0.7
    valid[0, 0] = True
    return q, k, v, do, valid


def test_layer_norm_gradient_is_the_derivative():
    g = np.random.default_rng(0)
    x, dy, w, b = g.standard_normal((4, 9)) + 3, g.standard_normal((4, 9)), g.standard_normal(9), g.standard_normal(9)
    t = [torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (9,), t[1], t[2], 1e-5)
    assert np.allclose(decoder.layer_norm_fwd(x, w, b, 1e-5)[0], y.detach().numpy(), rtol=0, atol=1e-13)
    y.backward(torch.tensor(dy))
    for got, want in zip(decoder.layer_norm_bwd(dy, x, w, 1e-5), t):
        assert np.allclose(got, want.grad.numpy(), rtol=0, atol=1e-12)


@pytest.mark.parametrize("seed", [1, 2])
def test_attention_gradient_is_the_derivative(seed):
    q, k, v, do, valid = _case(seed)
    r = decoder.attention_bwd(do, q, k, v, valid, 0.4)
    g = np.random.default_rng(seed + 10)

    def loss(q, k, v):
        return (decoder.attention_fwd(q, k, v, valid, 0.4)["out"] * do).sum()

    for i, name in enumerate(("dq", "dk", "dv")):
        at = [q, k, v]
        u = g.standard_normal(at[i].shape)
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + 1e-5 * u, at[i] - 1e-5 * u
        assert abs((loss(*hi) - loss(*lo)) / 2e-5 - (r[name] * u).sum()) < 1e-8


def test_attention_against_torch_softmax_and_autograd():
    q, k, v, do, valid = _case(3, h=3, hk=3)
    t = [torch.tensor(a, requires_grad=True) for a in (q, k, v)]
    s = 0.4 * torch.einsum("bihd,bjhd->bhij", t[0], t[1])
    p = torch.softmax(s.masked_fill(~torch.tensor(valid)[:, None, None], -1e300), 3)
    out = torch.einsum("bhij,bjhd->bihd", p, t[2])
    out.backward(torch.tensor(do))
    r = decoder.attention_bwd(do, q, k, v, valid, 0.4)
    assert np.allclose(r["out"], out.detach().numpy(), rtol=0, atol=1e-13)
    for name, a in zip(("dq", "dk", "dv"), t):
        assert np.allclose(r[name], a.grad.numpy(), rtol=0, atol=1e-12)


def test_rows_without_keys_and_equal_scores():
    q, k, v, do, valid = _case(4)
    valid[1] = False
    k[1], v[1] = np.nan, np.inf
    r = decoder.attention_bwd(do, q, k, v, valid, 0.4)
    f = decoder.attention_fwd(q, k, v, valid, 0.4)
    assert (f["out"][1] == 0).all() and (f["lse"][1] == -np.inf).all()
    assert all(np.isfinite(r[n]).all() for n in ("dq", "dk", "dv")) and (r["dk"][1] == 0).all()
    # equal keys: the mean of the values, lse = score + log n
    f = decoder.attention_fwd(q[:1], np.ones_like(k[:1]), v[:1], np.ones((1, 7), bool), 0.5)
    assert np.allclose(f["out"][0, :, 0], v[0, :, 0].mean(0))
    assert np.allclose(f["lse"][0], 0.5 * q[0].sum(2).T + np.log(7))
