"""GPU layer norm against the float64 one.

Tolerances, from float32 arithmetic and one rounding to the element type (unit roundoff u): the mean is a sum
of C terms, off by at most 2^-22 of the mean magnitude of the row for the pairwise orders used; centred values
are off by that and half an ulp, so xhat is off by 2^-21 (|x| + mean|x|) rstd plus 2^-21 |xhat|; the weight and
bias add 2^-23 of their terms; the result is rounded once. dx is a chain of such terms, dweight and dbias are
sums over R rows of float32 terms in a fixed order of short chains: 2^-20 of the sum of the magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import decoder

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half the spacing of subnormals
EPS = 1e-5


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _rand(shape, dtype, seed, factor=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device=DEV, generator=g) * factor + shift).to(dtype)


def _check(x, w, b, dy):
    u, tiny = U[x.dtype], TINY[x.dtype]
    y, mean, rstd = api.gs_layer_norm_fwd(x, w, b, eps=EPS)
    X, W, B = _np(x), _np(w), _np(b)
    ry, rm, rr = decoder.layer_norm_fwd(X, W, B, EPS)
    row = np.abs(X).mean(1)
    xhat = (X - rm[:, None]) * rr[:, None]
    exh = 2.0 ** -21 * ((np.abs(X) + row[:, None]) * rr[:, None] + np.abs(xhat))
    aw = 1.0 if w is None else np.abs(W)
    assert (np.abs(_np(mean) - rm) <= 2.0 ** -22 * row + 1e-37).all()
    # var is off by 2 |c| ec averaged; rstd by half of that relative to var + eps
    assert (np.abs(_np(rstd) / rr - 1) <= 2.0 ** -21 + (np.abs(xhat) * exh).mean(1)).all()
    rel = (2.0 ** -21 + (np.abs(xhat) * exh).mean(1))[:, None]
    ab = 0.0 if b is None else np.abs(B)
    tol = exh * aw + np.abs(xhat) * aw * rel + 2.0 ** -22 * ab + u * np.abs(ry) + tiny
    assert (np.abs(_np(y) - ry) <= tol).all(), np.max(np.abs(_np(y) - ry) / tol)

    dx, dw, db = api.gs_layer_norm_bwd(dy, x, mean, rstd, w)
    DY = _np(dy)
    rdx, rdw, rdb = decoder.layer_norm_bwd(DY, X, W, EPS)
    g = np.abs(DY) * aw
    ex = exh + np.abs(xhat) * rel
    c1 = (np.abs(DY * (1.0 if w is None else W) * xhat)).mean(1, keepdims=True)
    tol = rr[:, None] * (2.0 ** -20 * (g + g.mean(1, keepdims=True) + np.abs(xhat) * c1) + ex * c1 +
                         np.abs(xhat) * (g * ex).mean(1, keepdims=True)) + rel * np.abs(rdx) + u * np.abs(rdx) + tiny
    assert (np.abs(_np(dx) - rdx) <= tol).all(), np.max(np.abs(_np(dx) - rdx) / tol)
    if w is None:
        assert dw is None and db is None
        return
    uw, tw = U[w.dtype], TINY[w.dtype]
    tol = 2.0 ** -20 * np.abs(DY * xhat).sum(0) + (np.abs(DY) * ex).sum(0) + uw * np.abs(rdw) + tw
    assert (np.abs(_np(dw) - rdw) <= tol).all(), np.max(np.abs(_np(dw) - rdw) / tol)
    tol = 2.0 ** -20 * np.abs(DY).sum(0) + uw * np.abs(rdb) + tw
    assert (np.abs(_np(db) - rdb) <= tol).all(), np.max(np.abs(_np(db) - rdb) / tol)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (70, 31), (513, 64), (257, 100), (200, 128), (65, 256), (33, 333),
                                       (129, 384), (40, 512), (700, 768), (37, 1000), (64, 1024), (9, 1023), (12, 2048),
                                       (11, 4095), (5, 4096), (7, 8192), (3, 8193), (2, 20000)])
def test_layer_norm(dtype, rows, cols):
    x = _rand((rows, cols), dtype, rows + cols, 2.0, 0.5)
    _check(x, _rand((cols,), dtype, 1, 0.3, 1.0), _rand((cols,), dtype, 2), _rand((rows, cols), dtype, 3))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_float32_weights_of_16_bit_rows(dtype):
    x = _rand((77, 192), dtype, 5)
    _check(x, _rand((192,), torch.float32, 1, 0.3, 1.0), _rand((192,), torch.float32, 2), _rand((77, 192), dtype, 3))


def test_without_weight_with_offset_rows_and_many_rows():
    x = _rand((100, 96), torch.float32, 5, 0.01, 100.0)  # mean 10^4 times the spread
    _check(x, None, None, _rand((100, 96), torch.float32, 6))
    x = _rand((30011, 40), torch.bfloat16, 7)
    _check(x, _rand((40,), torch.bfloat16, 1), _rand((40,), torch.bfloat16, 2), _rand((30011, 40), torch.bfloat16, 8))


@pytest.mark.parametrize("offset,width", [(0, 80), (1, 80), (8, 72), (8, 80)])
def test_strided_and_misaligned_rows(offset, width):
    base = _rand((50, 100), torch.bfloat16, 3)
    x = base[:, offset:offset + width]
    dyb = _rand((50, 120), torch.bfloat16, 4)
    _check(x, _rand((width,), torch.bfloat16, 1), _rand((width,), torch.bfloat16, 2), dyb[:, 3:3 + width])
    out = torch.zeros(50, 128, dtype=torch.bfloat16, device=DEV)
    stats = torch.empty(50, device=DEV), torch.empty(50, device=DEV)
    y, _, _ = api.gs_layer_norm_fwd(x, out=(out[:, 5:5 + width],) + stats)
    assert torch.equal(y, api.gs_layer_norm_fwd(x.contiguous())[0])
    assert (out[:, :5] == 0).all() and (out[:, 5 + width:] == 0).all()  # nothing beside the rows


def test_leading_dimensions_in_place_and_another_stream():
    x = _rand((3, 17, 64), torch.float32, 9)
    y, mean, rstd = api.gs_layer_norm_fwd(x)
    assert y.shape == x.shape and mean.shape == (51,)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z, _, _ = api.gs_layer_norm_fwd(x, stream=side)
    side.synchronize()
    assert torch.equal(y, z)
    inplace = x.clone()
    api.gs_layer_norm_fwd(inplace, out=(inplace, mean, rstd))
    assert torch.equal(inplace, y)


def test_constant_rows_non_finite_rows_and_empty():
    x = torch.full((4, 40), 3.0, device=DEV)
    x[1, 7], x[2, 3] = float("nan"), float("inf")
    y, mean, rstd = api.gs_layer_norm_fwd(x)
    assert (y[0] == 0).all() and (y[3] == 0).all() and abs(rstd[0].item() * EPS ** 0.5 - 1) < 1e-6
    assert y[1].isnan().all() and y[2].isnan().any()
    e = torch.empty(0, 40, device=DEV)
    w = torch.ones(40, device=DEV)
    y, mean, rstd = api.gs_layer_norm_fwd(e, w, w)
    dx, dw, db = api.gs_layer_norm_bwd(e, e, mean, rstd, w)
    assert y.shape == (0, 40) and (dw == 0).all() and (db == 0).all()


def test_gradient_against_differences():
    x, w, dy = _rand((6, 50), torch.float32, 1), _rand((50,), torch.float32, 2), _rand((6, 50), torch.float32, 3)
    _, mean, rstd = api.gs_layer_norm_fwd(x, w, None)
    dx, dw, _ = api.gs_layer_norm_bwd(dy, x, mean, rstd, w)
    g = np.random.default_rng(0)
    for got, at in ((dx, 0), (dw, 1)):
        u = g.standard_normal(tuple(got.shape))
        args = [_np(x), _np(w)]

        def loss(t):
            a = list(args)
            a[at] = a[at] + t * u
            return (decoder.layer_norm_fwd(a[0], a[1], None, EPS)[0] * _np(dy)).sum()

        want, terms = (loss(1e-5) - loss(-1e-5)) / 2e-5, np.abs(_np(got) * u).sum()
        assert abs((_np(got) * u).sum() - want) <= 1e-6 * terms + 1e-8


def test_same_bits_twice_and_graph_capture():
    x, w, dy = _rand((5000, 256), torch.float32, 1), _rand((256,), torch.float32, 2), _rand((5000, 256), torch.float32, 3)
    _, mean, rstd = api.gs_layer_norm_fwd(x, w, w)
    a, b = (api.gs_layer_norm_bwd(dy, x, mean, rstd, w) for _ in range(2))
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c = api.gs_layer_norm_bwd(dy, x, mean, rstd, w)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, c))


def test_refusals():
    x = torch.zeros(4, 40, device=DEV)
    for bad in (lambda: api.gs_layer_norm_fwd(x.double()), lambda: api.gs_layer_norm_fwd(x.t()),
                lambda: api.gs_layer_norm_fwd(x, torch.zeros(39, device=DEV)),
                lambda: api.gs_layer_norm_fwd(x, torch.zeros(40, device=DEV, dtype=torch.float16)),
                lambda: api.gs_layer_norm_fwd(x.half(), torch.zeros(40, device=DEV, dtype=torch.bfloat16)),
                lambda: api.gs_layer_norm_fwd(x, out=(x.half(), x[:, 0], x[:, 1])),
                lambda: api.gs_layer_norm_bwd(x[:2], x, x[:, 0].contiguous(), x[:, 0].contiguous())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_abi.GsError, match="eps"):
        api.gs_layer_norm_fwd(x, eps=-1.0)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("rows,cols", [(1000, 8), (999, 16), (517, 32), (301, 24), (130, 48), (61, 34), (41, 70), (33, 126), (29, 250),
                                       (23, 382), (19, 510), (17, 1022), (9, 2046), (7, 4094), (3, 6002)])
def test_narrow_rows_and_rows_of_odd_pairs(dtype, rows, cols):
    x = _rand((rows, cols), dtype, rows + cols, 2.0, 0.5)
    _check(x, _rand((cols,), dtype, 1, 0.3, 1.0), _rand((cols,), dtype, 2), _rand((rows, cols), dtype, 3))


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("rows,cols", [(300, 64), (2000, 256), (900, 333), (400, 1024), (70, 4096), (40, 8193), (200, 9000)])
def test_gradient_written_over_an_input(dtype, rows, cols):
    x, dy = _rand((rows, cols), dtype, 1), _rand((rows, cols), dtype, 2)
    w = _rand((cols,), dtype, 3, 0.3, 1.0)
    _, mean, rstd = api.gs_layer_norm_fwd(x, w, None)
    want = api.gs_layer_norm_bwd(dy, x, mean, rstd, w)
    for over in (0, 1):
        a, b = x.clone(), dy.clone()
        got = api.gs_layer_norm_bwd(b, a, mean, rstd, w, out=((a, b)[over], torch.empty_like(w), torch.empty_like(w)))
        for g, t in zip(got, want):
            assert torch.equal(g, t)
    y = x.clone()
    api.gs_layer_norm_fwd(y, w, w, out=(y, torch.empty_like(mean), torch.empty_like(rstd)))
    assert torch.equal(y, api.gs_layer_norm_fwd(x, w, w)[0])
