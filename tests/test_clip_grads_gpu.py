"""The global gradient norm and clipping on the GPU against float64.

Tolerances: a thread adds 64 squares in four chains of float32 (17 roundings of 2^-24 of positive terms), the rest is
float64; the root halves that: the norm is off by 9 x 2^-24 and its own rounding. The factor is off by as much, a gradient by
that, the factor's and its own rounding.
"""
import numpy as np
import pytest
import torch

from oracle import fp8

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F32: 2.0 ** -150, F16: 2.0 ** -25, BF16: 2.0 ** -134}  # half the spacing of subnormals (2^-149, 2^-24, 2^-133)
NORM = 11 * 2.0 ** -24


def _np(t):
    return t.double().cpu().numpy()


def _grads(sizes, dtypes, seed=0, factor=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, device=DEV, generator=g) * factor * (1 + i % 3)).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def _check(grads, most, eps=1e-6):
    want, clipped = fp8.clip([_np(g) for g in grads], most, eps)
    before = [g.clone() for g in grads]
    out = [torch.full_like(g, 3) for g in grads]
    norms = [api.gs_grad_norm(grads), api.gs_clip_grads(grads, most, eps, out=out)]
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    norms.append(api.gs_clip_grads(grads, most, eps))
    for n in norms:
        assert n.shape == () and n.dtype == F32 and abs(n.item() - want) <= NORM * want
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
    for g, c in zip(grads, clipped):
        tol = np.abs(c) * (NORM + 2.0 ** -23 + U[g.dtype]) + TINY[g.dtype]
        assert (np.abs(_np(g) - c) <= tol).all()
    return norms[0]


@pytest.mark.parametrize("dtypes", [(F32,), (F16,), (BF16,), (F32, BF16, F16)])
@pytest.mark.parametrize("sizes", [(1,), (7,), (16384,), (16385, 3), (0, 5, 0, 40000), (100, 1, 77, 16384 * 3 + 9, 512, 2, 4096), (1000003,)])
@pytest.mark.parametrize("most", [0.5, 1e9])
def test_clip(sizes, dtypes, most):
    _check(_grads(sizes, dtypes, len(sizes)), most)


@pytest.mark.parametrize("count", [31, 32, 33, 512, 513, 1100])
def test_many_tensors(count):
    _check(_grads([1 + 37 * i % 901 for i in range(count)], (F32, BF16), count), 2.0)


def test_misaligned_and_shaped_gradients():
    base = _grads([100000], (BF16,))[0]
    grads = [base[1:1000], base[1002:2001], base[3000:23000].view(100, 200).t(), base[40008:90008].view(10, 50, 100)]
    _check(grads, 1.0)
    a, b = base.clone(), base.clone()  # (the check left a small norm: a bound below it whatever it is)
    api.gs_clip_grads([a[1:100]], 0.0)
    assert torch.equal(a[:1], b[:1]) and torch.equal(a[100:], b[100:]) and (a[1:100] == 0).all()


def test_squares_outside_float32():
    for factor in (1e-30, 1e-20, 1e25):
        _check([g.clamp(-3e38, 3e38) for g in _grads([70000, 9], (F32,), 2, factor)], factor)
    # large and tiny tensors together
    _check(_grads([20000], (F32,), 1, 1e-25) + _grads([20000], (F32,), 2, 1e22) + _grads([20000], (BF16,), 2, 1.0), 1.0)


def test_norms_that_are_not_finite_and_zeros():
    g = torch.ones(50, device=DEV)
    g[7] = float("nan")
    h = torch.ones(20, device=DEV, dtype=BF16)
    assert api.gs_clip_grads([g, h], 1.0).isnan() and g.isnan().all() and h.isnan().all()
    g = torch.ones(50, device=DEV)
    g[7] = -float("inf")
    assert api.gs_clip_grads([g], 1.0).isinf() and g[7].isnan() and (g[:7] == 0).all()
    z = torch.zeros(50, device=DEV)
    for most, eps in ((1.0, 1e-6), (0.0, 0.0), (0.0, 1e-6), (float("inf"), 0.0)):
        assert api.gs_clip_grads([z], most, eps) == 0 and (z == 0).all()
    g = torch.ones(50, device=DEV)
    assert (api.gs_clip_grads([g], float("inf")) - 50 ** 0.5).abs() < 1e-5 and (g == 1).all()
    api.gs_clip_grads([g], 0.0)
    assert (g == 0).all()
    assert api.gs_grad_norm([torch.empty(0, device=DEV)]) == 0
    assert api.gs_clip_grads([torch.empty(0, device=DEV)], 1.0) == 0


def test_a_large_set_against_torch():
    grads = _grads([3_000_000, 4_800_000, 1_000_000], (F32,), 5, 1e-3)
    want = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
    expected = [(g.double() * (0.1 / (want + 1e-6))) for g in grads]
    norm = api.gs_clip_grads(grads, 0.1)
    assert (norm.double() - want).abs() <= NORM * want
    for g, e in zip(grads, expected):
        assert ((g.double() - e).abs() <= e.abs() * (NORM + 2.0 ** -22)).all()


def test_same_bits_kept_workspace_streams_and_capture():
    grads = _grads([100000, 33, 70000], (F32, BF16))
    out = [torch.empty_like(g) for g in grads]
    want_norm = api.gs_clip_grads(grads, 0.1, out=out)
    want = [o.clone() for o in out]
    kept, norm = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV), torch.empty((), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert api.gs_clip_grads(grads, 0.1, out=out, norm=norm, workspace=kept, stream=side) is norm
    side.synchronize()
    assert torch.equal(norm, want_norm) and all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = api.gs_clip_grads(grads, 0.1, out=out)
        api.gs_clip_grads(grads, 0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want_norm) and all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(grads, want))
    assert api.gs_device_error() == _abi.GS_OK


def test_refusals():
    g, h = torch.ones(50, device=DEV), torch.ones(50, device=DEV)
    for bad in (lambda: api.gs_clip_grads([], 1.0), lambda: api.gs_clip_grads([g.double()], 1.0), lambda: api.gs_clip_grads([g[::2]], 1.0),
                lambda: api.gs_clip_grads([g.expand(3, 50)], 1.0), lambda: api.gs_clip_grads([g, g.cpu()], 1.0), lambda: api.gs_clip_grads([g], 1.0, out=[]),
                lambda: api.gs_clip_grads([g], 1.0, out=[h.half()]), lambda: api.gs_clip_grads([g], 1.0, out=[h[:20]]),
                lambda: api.gs_clip_grads([g], None, out=[h]), lambda: api.gs_clip_grads([g], 1.0, norm=torch.empty(2, device=DEV)),
                lambda: api.gs_clip_grads([g.view(5, 10)], 1.0, out=[h.view(10, 5).t()]), lambda: api.gs_clip_grads([3.0], 1.0),
                lambda: api.gs_clip_grads([g], 1.0, workspace=torch.empty(100, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        api.gs_clip_grads([g], "one")
    for bad in (lambda: api.gs_clip_grads([g], -1.0), lambda: api.gs_clip_grads([g], float("nan")), lambda: api.gs_clip_grads([g, g], 1.0),
                lambda: api.gs_clip_grads([g, g[10:20]], 1.0), lambda: api.gs_clip_grads([g, h], 1.0, out=[h, g]),
                lambda: api.gs_clip_grads([g[:40]], 1.0, out=[g[10:]])):
        with pytest.raises(_abi.GsError):
            bad()
    assert (g == 1).all() and (h == 1).all()
