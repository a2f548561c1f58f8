"""GPU root-mean-square norm against the float64 one.

Tolerances, from float32 arithmetic and one rounding to the element type (unit roundoff u): the mean square is a sum of
positive terms; a thread adds at most 32 of them in a chain (cols / 256 in rows above 8,192), the lanes and warps at most 13
more: relative error (45 + cols / 256) 2^-24 =: e. rstd is off by e / 2 and three roundings, y by two more. With 8 bits a
value is off by half a step beside that: 2^-4 of itself, or 2^-10 of its scale below the normal values; the scale by the
relative error of the block's largest value and two roundings. dx and dweight are chains of such terms: the error of rstd,
six roundings of each term's magnitude, and the row's (column's) sum, whose chain has at most 45 + cols / 256 links (rows
in blocks of up to 1,024 shares: rows / 152 + 64).
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
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}  # half the spacing of subnormals
EPS = 1e-6
SIZES = [(1, 1), (3, 5), (1, 1024), (70, 31), (513, 64), (257, 100), (200, 128), (65, 256), (33, 333), (129, 384), (40, 512), (700, 768),
         (37, 1000), (64, 1024), (9, 1023), (12, 2048), (11, 4095), (5, 4096), (7, 8192), (3, 8193), (2, 20000)]


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _rand(shape, dtype, seed, factor=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device=DEV, generator=g) * factor + shift).to(dtype)


def _sum(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def _check_fwd(x, w, r, **kw):
    u, tiny, cols = U[x.dtype], TINY[x.dtype], x.shape[1]
    e = (45 + cols / 256) * 2.0 ** -24
    want_h = _sum(x, r)
    y, h, rstd = api.gs_rms_norm_fwd(x, w, r, eps=EPS, **kw)
    ry, rr = fp8.rms_norm_fwd(_np(want_h), None, _np(w), EPS)
    assert torch.equal(h, want_h) and (r is not None or h is x)
    assert (np.abs(_np(rstd) / rr - 1) <= e / 2 + 3 * 2.0 ** -24).all()
    tol = np.abs(ry) * (e / 2 + 5 * 2.0 ** -24 + u) + tiny
    assert (np.abs(_np(y) - ry) <= tol).all(), np.max(np.abs(_np(y) - ry) / (tol + 1e-300))
    return y, h, rstd


def _check_fp8(x, w, r, **kw):
    cols = x.shape[1]
    e = (45 + cols / 256) * 2.0 ** -25 + 5 * 2.0 ** -24
    want_h = _sum(x, r)
    q, s, h, rstd = api.gs_rms_norm_fp8(x, w, r, eps=EPS, **kw)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and q.stride(0) % 16 == 0 and s.shape == (len(x), -(-cols // 128))
    ry, rr = fp8.rms_norm_fwd(_np(want_h), None, _np(w), EPS)
    assert torch.equal(h, want_h) and (kw or torch.equal(rstd, api.gs_rms_norm_fwd(x, w, r, eps=EPS)[2]))
    rs = fp8.scales(ry, 1)
    assert (np.abs(_np(s) / rs - 1) <= e + 2 * 2.0 ** -24).all()
    each = fp8.spread(_np(s), ry.shape)
    tol = np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * each) * (1 + 2.0 ** -18) + (e + 4 * 2.0 ** -24) * np.abs(ry)
    assert (np.abs(_np(q) * each - ry) <= tol).all()
    assert np.abs(_np(q)).max() == 448
    return q, s


def _check_bwd(dy, h, w, dh, **kw):
    u, tiny, (rows, cols) = U[h.dtype], TINY[h.dtype], h.shape
    rstd = api.gs_rms_norm_fwd(h, w, eps=EPS)[2]
    dx, dw = api.gs_rms_norm_bwd(dy, h, rstd, w, dh, **kw)
    DY, H, W, DH = _np(dy), _np(h), _np(w), _np(dh)
    rdx, rdw = fp8.rms_norm_bwd(DY, H, W, DH, EPS)
    rr = 1 / np.sqrt((H * H).mean(1, keepdims=True) + EPS)
    e = (45 + cols / 256) * 2.0 ** -24
    g, hhat = np.abs(DY * (1.0 if W is None else W)), np.abs(H) * rr
    size = rr * (g + hhat * (g * hhat).mean(1, keepdims=True))
    tol = size * (2 * e + 8 * 2.0 ** -24) + (u + 2.0 ** -24) * np.abs(rdx) + (0 if dh is None else 2.0 ** -24 * np.abs(DH)) + tiny
    assert (np.abs(_np(dx) - rdx) <= tol).all(), np.max(np.abs(_np(dx) - rdx) / (tol + 1e-300))
    if w is None:
        assert dw is None
        return dx, dw
    tol = (np.abs(DY) * hhat).sum(0) * ((rows / 152 + 64 + 8) * 2.0 ** -24 + e / 2) + U[w.dtype] * np.abs(rdw) + TINY[w.dtype]
    assert (np.abs(_np(dw) - rdw) <= tol).all(), np.max(np.abs(_np(dw) - rdw) / tol)
    return dx, dw


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_rms_norm(dtype, rows, cols, residual):
    x, w = _rand((rows, cols), dtype, rows + cols, 2.0, 0.5), _rand((cols,), dtype, 1, 0.3, 1.0)
    r = _rand((rows, cols), dtype, 2, 0.7) if residual else None
    _check_fwd(x, w, r)
    _check_fp8(x, w, r)
    _check_bwd(_rand((rows, cols), dtype, 3), _sum(x, r), w, _rand((rows, cols), dtype, 4) if residual else None)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("rows,cols", [(1000, 8), (999, 16), (517, 32), (301, 24), (130, 48), (61, 34), (41, 70), (33, 126), (29, 250), (23, 382),
                                       (19, 510), (17, 1022), (9, 2046), (7, 4094), (3, 6002), (5, 129), (6, 160), (4, 1032), (2, 8136)])
def test_narrow_rows_and_ends_inside_a_block(dtype, rows, cols):
    x, w = _rand((rows, cols), dtype, rows + cols, 2.0, 0.5), _rand((cols,), dtype, 1, 0.3, 1.0)
    r = _rand((rows, cols), dtype, 2)
    _check_fwd(x, w, r)
    _check_fp8(x, w, None)
    _check_bwd(_rand((rows, cols), dtype, 3), x, w, r)


def test_float32_weights_without_weights_and_many_rows():
    for dtype in (torch.float16, torch.bfloat16):
        x, w = _rand((77, 192), dtype, 5), _rand((192,), torch.float32, 1, 0.3, 1.0)
        _check_fwd(x, w, x.flip(0))
        _check_fp8(x, w, None)
        _check_bwd(_rand((77, 192), dtype, 3), x, w, None)
    x = _rand((30011, 40), torch.bfloat16, 7)
    _check_fwd(x, None, None)
    _check_fp8(x, None, x)
    _check_bwd(_rand((30011, 40), torch.bfloat16, 8), x, None, x)
    _check_bwd(_rand((30011, 40), torch.bfloat16, 8), x, _rand((40,), torch.bfloat16, 9), None)


@pytest.mark.parametrize("offset,width", [(0, 80), (1, 80), (8, 72), (8, 80)])
def test_strided_and_misaligned_rows(offset, width):
    base, rb = _rand((50, 100), torch.bfloat16, 3), _rand((50, 130), torch.bfloat16, 4)
    x, r, w = base[:, offset:offset + width], rb[:, 2:2 + width], _rand((width,), torch.bfloat16, 1)
    _check_fwd(x, w, r)
    _check_fp8(x, w, r)
    _check_bwd(r, x, w, rb[:, 7:7 + width])
    room = torch.zeros(50, 256, dtype=torch.bfloat16, device=DEV)
    # (rows of another alignment are added in another order: within the tolerances, not the same bits)
    _check_fwd(x, w, r, out=(room[:, 3:3 + width], room[:, 120:120 + width], torch.empty(50, device=DEV)))
    room[:, 3:3 + width] = 0
    room[:, 120:120 + width] = 0
    assert (room == 0).all()  # nothing beside the rows
    q = torch.zeros(50, 128, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    s = torch.zeros(50, 4, device=DEV)
    _check_fp8(x, w, r, out=(q[:, 16:16 + width], s[:, 1:2], room[:, 120:120 + width], torch.empty(50, device=DEV)))
    q.view(torch.uint8)[:, 16:16 + width] = 0
    assert (q.view(torch.uint8) == 0).all() and (s[:, 0] == 0).all() and (s[:, 2:] == 0).all()


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("rows,cols", [(300, 64), (2000, 256), (900, 333), (400, 1024), (70, 4096), (40, 8193), (200, 9000)])
def test_results_written_over_an_input(dtype, rows, cols):
    x, r, dy = (_rand((rows, cols), dtype, i) for i in range(3))
    w = _rand((cols,), dtype, 3, 0.3, 1.0)
    y, h, rstd = api.gs_rms_norm_fwd(x, w, r)
    for over in ((0, None), (1, None), (None, 0), (None, 1), (0, 1), (1, 0)):
        both = [x.clone(), r.clone()]
        to = [torch.empty_like(x) if i is None else both[i] for i in over]
        api.gs_rms_norm_fwd(both[0], w, both[1], out=(to[0], to[1], torch.empty_like(rstd)))
        assert torch.equal(to[0], y) and torch.equal(to[1], h), over
    same = x.clone()
    api.gs_rms_norm_fwd(same, w, out=(same, None, torch.empty_like(rstd)))
    assert torch.equal(same, api.gs_rms_norm_fwd(x, w)[0])
    want = api.gs_rms_norm_bwd(dy, h, rstd, w, r)
    for over in range(3):
        a = [dy.clone(), h.clone(), r.clone()]
        got = api.gs_rms_norm_bwd(a[0], a[1], rstd, w, a[2], out=(a[over], torch.empty_like(w)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), over


def test_leading_dimensions_and_another_stream():
    x = _rand((3, 17, 80), torch.float32, 9)
    y, h, rstd = api.gs_rms_norm_fwd(x)
    q, s, _, _ = api.gs_rms_norm_fp8(x)
    assert y.shape == x.shape and h is x and rstd.shape == (51,) and q.shape == x.shape and s.shape == (51, 1)
    flat = api.gs_rms_norm_fp8(x.view(51, 80))
    assert torch.equal(flat[0].view(torch.uint8), q.view(torch.uint8).view(51, 80)) and torch.equal(flat[1], s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = api.gs_rms_norm_fwd(x, stream=side)[0]
    p = api.gs_rms_norm_fp8(x, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, z) and torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_zeros_non_finite_values_and_no_rows():
    x = torch.zeros(6, 300, device=DEV)
    x[1, 7], x[2, 3], x[3, 200], x[4, 5] = float("nan"), float("inf"), 1e-30, 1e30
    y, _, rstd = api.gs_rms_norm_fwd(x)
    q, s, _, _ = api.gs_rms_norm_fp8(x)
    assert (y[0] == 0).all() and (q[0].float() == 0).all() and (s[0] == 1).all() and abs(rstd[0].item() * EPS ** 0.5 - 1) < 1e-6
    assert y[1].isnan().all() and s[1].isnan().all() and q[1].float().isnan().all()
    assert y[2, 3].isnan() and (y[2, :3] == 0).all()  # inf x 0
    assert s[2, 0].isnan() and (s[2, 1:] == 1).all()
    assert rstd[4].item() == 0 and (y[4] == 0).all()  # the square is no float32
    assert y[3, 200].item() == pytest.approx(1e-27, rel=1e-6)
    e, w = torch.empty(0, 40, device=DEV), torch.ones(40, device=DEV)
    y, h, rstd = api.gs_rms_norm_fwd(e, w, e)
    dx, dw = api.gs_rms_norm_bwd(e, e, rstd, w, e)
    q, s, _, _ = api.gs_rms_norm_fp8(e, w)
    assert y.shape == h.shape == dx.shape == q.shape == (0, 40) and s.shape == (0, 1) and (dw == 0).all()


def test_gradient_against_differences():
    h, w, dy, dh = _rand((6, 50), torch.float32, 1), _rand((50,), torch.float32, 2), _rand((6, 50), torch.float32, 3), _rand((6, 50), torch.float32, 4)
    dx, dw = api.gs_rms_norm_bwd(dy, h, api.gs_rms_norm_fwd(h, w)[2], w, dh)
    g = np.random.default_rng(0)
    for got, at in ((dx, 0), (dw, 1)):
        u = g.standard_normal(tuple(got.shape))

        def loss(t):
            a = [_np(h), _np(w)]
            a[at] = a[at] + t * u
            return (fp8.rms_norm_fwd(a[0], None, a[1], EPS)[0] * _np(dy)).sum() + (a[0] * _np(dh)).sum()

        want, terms = (loss(1e-5) - loss(-1e-5)) / 2e-5, np.abs(_np(got) * u).sum()
        assert abs((_np(got) * u).sum() - want) <= 1e-6 * terms + 1e-8


def test_same_bits_twice_kept_workspace_and_capture():
    x, w, dy = _rand((5000, 256), torch.float32, 1), _rand((256,), torch.float32, 2), _rand((5000, 256), torch.float32, 3)
    rstd = api.gs_rms_norm_fwd(x, w)[2]
    want = api.gs_rms_norm_bwd(dy, x, rstd, w, dy) + api.gs_rms_norm_fp8(x, w, dy)[:3]
    kept = torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV)
    again = api.gs_rms_norm_bwd(dy, x, rstd, w, dy, workspace=kept) + api.gs_rms_norm_fp8(x, w, dy)[:3]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = api.gs_rms_norm_bwd(dy, x, rstd, w, dy) + api.gs_rms_norm_fp8(x, w, dy)[:3]
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, again, captured):
        assert torch.equal(a.float(), b.float()) and torch.equal(a.float(), c.float())
    assert api.gs_device_error() == _abi.GS_OK


def test_refusals():
    x, v = torch.zeros(4, 40, device=DEV), torch.zeros(4, device=DEV)
    q = torch.zeros(4, 48, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[:, :40]
    s = torch.zeros(4, 1, device=DEV)
    for bad in (lambda: api.gs_rms_norm_fwd(x.double()), lambda: api.gs_rms_norm_fwd(x.t()), lambda: api.gs_rms_norm_fwd(x, torch.zeros(39, device=DEV)),
                lambda: api.gs_rms_norm_fwd(x, torch.zeros(40, device=DEV, dtype=torch.float16)), lambda: api.gs_rms_norm_fwd(x, None, x[:2]),
                lambda: api.gs_rms_norm_fwd(x, None, x.half()), lambda: api.gs_rms_norm_fwd(x, out=(x.half(), None, v)),
                lambda: api.gs_rms_norm_fwd(x, out=(x, v)), lambda: api.gs_rms_norm_fp8(x, out=(x, s, None, v)),
                lambda: api.gs_rms_norm_fp8(x, out=(q, s[:2], None, v)), lambda: api.gs_rms_norm_fp8(x, out=(q[:, :32], s, None, v)),
                lambda: api.gs_rms_norm_bwd(x[:2], x, v), lambda: api.gs_rms_norm_bwd(x, x, v[:2]),
                lambda: api.gs_rms_norm_bwd(x, x, v, workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_abi.GsError, match="eps"):
        api.gs_rms_norm_fwd(x, eps=-1.0)
    with pytest.raises(_abi.GsError, match="lies on"):
        api.gs_rms_norm_fwd(x, None, x.clone(), out=(y := torch.empty_like(x), y, v))
    with pytest.raises(_abi.GsError, match="aligned"):
        api.gs_rms_norm_fp8(x, out=(torch.zeros(4, 48, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[:, 8:], s, None, v))


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("cols", [8200, 9992, 16384, 16385, 24600])
def test_rows_longer_than_a_blocks_registers(dtype, cols):
    rows = 6
    x, r, dy, dh = (_rand((rows, cols), dtype, cols + i, 1.5, 0.2) for i in range(4))
    wide = _rand((cols + 8,), dtype, 9, 0.3, 1.0)
    for w in (wide[:cols], wide[1:cols + 1], wide[:cols].float(), None):  # on 16 bytes, not, float32, none
        _check_fwd(x, w, r)
        _check_fp8(x, w, r)
        _check_fp8(x, w, None)
        _check_bwd(dy, _sum(x, r), w, dh)
        _check_bwd(dy, x, w, None)
    # rows apart that start on 16 bytes, or do not; results over the inputs
    for start, apart in ((0, cols + 8 - cols % 8), (1, cols + 1)):
        room = torch.full((3, rows * apart + 8), 7.0, device=DEV, dtype=dtype)
        a, b, c = (room[i, start:start + rows * apart].view(rows, apart)[:, :cols] for i in range(3))
        a.copy_(x), b.copy_(r)
        want = api.gs_rms_norm_fwd(x, wide[:cols], r, eps=EPS)
        y, h, _ = api.gs_rms_norm_fwd(a, wide[:cols], b, eps=EPS, out=(b, a, torch.empty(rows, device=DEV)))
        assert torch.equal(h, want[1]) and y.data_ptr() == b.data_ptr()
        assert ((y.double() - want[0].double()).abs() <= 2 * U[dtype] * want[0].double().abs() + 2.0 ** -18 * want[0].double().abs() + TINY[dtype] * 2).all()
        c.copy_(dy)
        one = api.gs_rms_norm_bwd(dy, want[1], want[2], wide[:cols], dh)
        two = api.gs_rms_norm_bwd(c, a, want[2], wide[:cols], dh, out=(c, torch.empty_like(wide[:cols])))
        near = one[0].double().abs() * 2 * U[dtype] + 2.0 ** -16 * (dy.double().abs() + dh.double().abs() + 1) * (1 + want[2].double().max())
        assert ((two[0].double() - one[0].double()).abs() <= near).all()
        for i in range(2):
            rest = room[i, start:start + rows * apart].view(rows, apart)[:, cols:]
            assert (rest == 7).all() and (room[i, :start] == 7).all()
