"""Refusals of the 8-bit decoder's entry points: host checks before any device work (CPU, addresses that are never read)."""
import ctypes as C

import pytest
import torch

import __graft_entry__
from differentiable_gaussian_splatting_gs_gb300 import _abi, api

if torch.cuda.is_available():
    pytest.skip("made-up addresses: only where no device could follow them", allow_module_level=True)

ARG, OK = _abi.GS_ERR_ARG, _abi.GS_OK
ROOM = 1 << 32  # the addresses below are further apart than the tensors' sizes


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _abi.load()


def _fp8(data=8 * ROOM, stride=64, scale=9 * ROOM, row=1, block=64, rows=1):
    return _abi.gs_fp8(data=data, stride=stride, scale=scale, scale_row=row, scale_block=block, block_rows=rows)


def _ref(x):
    return None if x is None else C.byref(x)


def test_rms_norm_refusals(lib):
    def fwd(x=ROOM, xs=64, r=2 * ROOM, rs=64, rows=4, cols=64, dt=0, w=256, wdt=0, eps=1e-6, h=3 * ROOM, hs=64, y=4 * ROOM, ys=64, q=None, rstd=256):
        return lib.gs_rms_norm_fwd(x, xs, r, rs, rows, cols, dt, w, wdt, eps, h, hs, y, ys, _ref(q), rstd, None)

    assert fwd(rows=0) == OK and fwd(rows=0, y=None, q=_fp8()) == OK
    for bad in (dict(x=None), dict(x=ROOM + 2), dict(xs=63), dict(rows=-1), dict(cols=0), dict(cols=1 << 30), dict(dt=3), dict(wdt=1),
                dict(dt=1, wdt=2), dict(w=257), dict(eps=-1.0), dict(eps=float("inf")), dict(r=2 * ROOM + 1), dict(rs=63), dict(h=None),
                dict(hs=10), dict(y=None), dict(ys=63), dict(rstd=None), dict(rstd=258), dict(q=_fp8()),
                dict(y=None, q=_fp8(data=None)), dict(y=None, q=_fp8(data=8 * ROOM + 8)), dict(y=None, q=_fp8(stride=72)),
                dict(y=None, q=_fp8(stride=48)), dict(y=None, q=_fp8(scale=None)), dict(y=None, q=_fp8(rows=128)), dict(y=None, q=_fp8(rows=2)),
                dict(y=None, q=_fp8(row=0)), dict(y=None, q=_fp8(block=0), cols=192, xs=192, rs=192, hs=192)):
        assert fwd(**bad) == ARG, bad
        assert lib.gs_last_error_message()
    for bad in (dict(h=ROOM, hs=72), dict(h=ROOM + 64 * 4), dict(y=3 * ROOM), dict(y=ROOM + 4 * 8), dict(y=2 * ROOM, ys=128), dict(y=None, q=_fp8(data=ROOM))):
        assert fwd(**bad) == ARG and b"lies on" in lib.gs_last_error_message(), bad
    # over an input, beside one in its rows: refused for the missing statistics alone
    for fine in (dict(h=ROOM), dict(h=2 * ROOM), dict(y=ROOM), dict(y=2 * ROOM), dict(h=ROOM, y=2 * ROOM),
                 dict(xs=256, rs=256, hs=256, ys=256, r=ROOM + 256, h=ROOM + 512, y=ROOM + 768)):
        assert fwd(rstd=None, **fine) == ARG and b"rstd" in lib.gs_last_error_message(), fine

    def bwd(dy=ROOM, h=2 * ROOM, dh=3 * ROOM, rows=4, cols=64, dt=0, rstd=256, w=256, wdt=0, dx=4 * ROOM, dxs=64, dw=256, ws=256, n=1 << 20):
        return lib.gs_rms_norm_bwd(dy, cols, h, cols, dh, cols, rows, cols, dt, rstd, w, wdt, dx, dxs, dw, ws, n, None)

    for bad in (dict(dy=None), dict(h=None), dict(dh=3 * ROOM + 2), dict(rstd=None), dict(dx=None), dict(dw=257), dict(ws=None), dict(ws=264),
                dict(n=16), dict(wdt=2), dict(dx=ROOM, dxs=72), dict(dx=ROOM + 4)):
        assert bwd(**bad) == ARG, bad
    assert lib.gs_rms_norm_workspace_bytes(4, 64) == 4 * 64 * 4
    assert lib.gs_rms_norm_workspace_bytes(-1, 64) == 0


def test_quantize_refusals(lib):
    def call(x=ROOM, xr=64, xc=1, rows=4, cols=64, dt=0, q=_fp8()):
        return lib.gs_quantize_fp8(x, xr, xc, rows, cols, dt, _ref(q), None)

    assert call(rows=0) == OK and call(cols=0) == OK
    for bad in (dict(x=None), dict(x=ROOM + 1), dict(xr=2, xc=2), dict(xr=-64), dict(rows=-1), dict(cols=-1), dict(dt=7), dict(q=None),
                dict(q=_fp8(rows=64)), dict(q=_fp8(stride=60)), dict(q=_fp8(data=8 * ROOM + 4)), dict(q=_fp8(scale=9 * ROOM + 2)),
                dict(q=_fp8(row=0)), dict(q=_fp8(data=ROOM)), dict(q=_fp8(data=ROOM + 32))):
        assert call(**bad) == ARG, bad


def test_matmul_refusals(lib):
    def call(a=_fp8(), b=_fp8(data=10 * ROOM, rows=128), m=4, n=4, k=64, dt=2, out=ROOM, stride=4):
        return lib.gs_matmul_fp8(_ref(a), _ref(b), m, n, k, dt, out, stride, None)

    assert call(m=0) == OK and call(n=0) == OK
    for bad in (dict(a=None), dict(b=None), dict(m=-1), dict(n=-1), dict(k=-1), dict(k=(1 << 30) + 1), dict(dt=3), dict(out=None), dict(out=ROOM + 1),
                dict(stride=3), dict(a=_fp8(rows=128)), dict(b=_fp8(rows=3)), dict(a=_fp8(stride=65)), dict(a=_fp8(stride=48)),
                dict(b=_fp8(data=8)), dict(a=_fp8(scale=None)), dict(out=8 * ROOM), dict(out=10 * ROOM + 2)):
        assert call(**bad) == ARG, bad


def test_clip_refusals(lib):
    def grads(*rows):
        return (_abi.gs_gradient * max(1, len(rows)))(*[_abi.gs_gradient(grad=g, out=o, n=n, dtype=d) for g, o, n, d in rows])

    def call(g, count, clip=1, most=1.0, eps=1e-6, norm=256, ws=256, n=1 << 20):
        return lib.gs_clip_grads(g, count, clip, most, eps, norm, ws, n, None)

    two = grads((ROOM, None, 10, 0), (2 * ROOM, None, 10, 2))
    for bad in (dict(norm=None), dict(norm=258), dict(ws=None), dict(ws=264), dict(n=4), dict(most=-1.0), dict(most=float("nan")), dict(eps=-1.0),
                dict(eps=float("nan"))):
        assert call(two, 2, **bad) == ARG, bad
    assert call(None, 2) == ARG and call(two, -1) == ARG
    for rows in ([(None, None, 3, 0)], [(ROOM + 2, None, 3, 0)], [(ROOM, None, -1, 0)], [(ROOM, None, 3, 4)], [(ROOM, 2 * ROOM + 1, 3, 2)]):
        assert call(grads(*rows), 1) == ARG, rows
    # written twice, or written where another is read
    for rows in ([(ROOM, None, 10, 0), (ROOM, None, 10, 0)], [(ROOM, None, 10, 0), (ROOM + 36, None, 10, 0)],
                 [(ROOM, 2 * ROOM, 10, 0), (3 * ROOM, 2 * ROOM + 4, 10, 0)], [(ROOM, 2 * ROOM, 10, 0), (2 * ROOM + 36, 3 * ROOM, 10, 0)],
                 [(ROOM, ROOM + 4, 10, 0)], [(ROOM, 5 * ROOM, 100, 0), (3 * ROOM, ROOM + 200, 4, 0), (ROOM + 20, 7 * ROOM, 2, 0)]):
        assert call(grads(*rows), len(rows)) == ARG and b"lies on" in lib.gs_last_error_message(), rows
    # read twice, written side by side: refused for the missing norm alone
    for rows in ([(ROOM, 2 * ROOM, 10, 0), (ROOM, 3 * ROOM, 10, 0)], [(ROOM, None, 10, 0), (ROOM + 40, None, 10, 0)]):
        assert call(grads(*rows), 2, norm=None) == ARG and b"norm is" in lib.gs_last_error_message(), rows
    assert lib.gs_clip_workspace_bytes(two, 2) >= 2 * 8


def test_bindings_refuse_host_tensors():
    x = torch.zeros(4, 16)
    q, s = x.to(torch.float8_e4m3fn), torch.ones(4, 1)
    for call in (lambda: api.gs_rms_norm_fwd(x), lambda: api.gs_rms_norm_fp8(x), lambda: api.gs_rms_norm_bwd(x, x, s[:, 0]),
                 lambda: api.gs_quantize_fp8(x), lambda: api.gs_matmul_fp8(q, s, q, s), lambda: api.gs_clip_grads([x], 1.0),
                 lambda: api.gs_grad_norm([x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        api.gs_grad_norm([])
    with pytest.raises(ValueError, match="float32"):
        api.gs_matmul_fp8(q, s, q, s, dtype=torch.float64)


def _accepted(lib, status):
    """Past the checks of the arguments (there is no device to go on with)."""
    return status == _abi.GS_ERR_CUDA


def test_rows_that_repeat_take_only_their_memory(lib):
    def call(x, xr, xc, rows=1000, cols=128, q=_fp8(data=ROOM + 4096, stride=128, block=1000)):
        return lib.gs_quantize_fp8(x, xr, xc, rows, cols, 0, _ref(q), None)

    # a row, a column, windows one element apart: 512, 4,000 and 4,508 bytes
    assert _accepted(lib, call(ROOM, 0, 1))
    assert _accepted(lib, call(ROOM, 1, 0))
    assert _accepted(lib, call(ROOM - 512, 1, 1))
    for bad in ((ROOM + 4096, 0, 1), (ROOM + 3600, 0, 1), (ROOM + 100, 1, 0), (ROOM, 1, 1)):
        assert call(*bad) == ARG and b"lies on" in lib.gs_last_error_message(), bad


def test_scales_have_memory_of_their_own(lib):
    def quantize(q, rows=256, cols=512):
        return lib.gs_quantize_fp8(ROOM, 512, 1, rows, cols, 0, _ref(q), None)

    def q(**kw):
        return _fp8(**{"stride": 512, "block": 256, **kw})

    assert _accepted(lib, quantize(q())) and _accepted(lib, quantize(q(row=4, block=1))) and _accepted(lib, quantize(q(row=8, block=2)))
    for bad in (q(block=255), q(row=3, block=1), q(row=1, block=1), q(row=2, block=2), q(row=-1), q(block=-256), q(row=0), q(block=0)):
        assert quantize(bad) == ARG and b"share memory" in lib.gs_last_error_message(), (bad.scale_row, bad.scale_block)
    for bad in (q(scale=ROOM), q(scale=ROOM + 512 * 1024 - 4), q(scale=8 * ROOM + 512), q(scale=8 * ROOM - 4)):
        assert quantize(bad) == ARG and b"lies on" in lib.gs_last_error_message(), bad.scale

    def norm(t, y=None):
        return lib.gs_rms_norm_fwd(ROOM, 512, 2 * ROOM, 512, 256, 512, 0, None, 0, 1e-6, 3 * ROOM, 512, y, 512, _ref(t), 4 * ROOM, None)

    assert _accepted(lib, norm(q()))
    for bad in (q(scale=ROOM), q(scale=2 * ROOM + 4), q(scale=3 * ROOM + 8), q(scale=8 * ROOM)):
        assert norm(bad) == ARG and b"lies on" in lib.gs_last_error_message(), bad.scale
    assert norm(q(block=255)) == ARG

    def product(a, b, out=ROOM):
        return lib.gs_matmul_fp8(_ref(a), _ref(b), 256, 256, 512, 2, out, 256, None)

    b = _fp8(data=10 * ROOM, stride=512, scale=11 * ROOM, rows=128, row=4, block=1)
    assert _accepted(lib, product(q(), b))
    # scales that are read may repeat, or run backwards
    for fine in (q(row=0), q(block=0), q(row=0, block=0), q(row=-1), q(block=-256), q(row=1, block=1)):
        assert _accepted(lib, product(fine, b)), (fine.scale_row, fine.scale_block)
    for bad in (9 * ROOM, 9 * ROOM + 4 * 1022, 11 * ROOM + 16):
        assert product(q(), b, bad) == ARG and b"lies on" in lib.gs_last_error_message(), bad


def test_sizes_without_an_end(lib):
    """Rows and strides at their limits: refused or passed on, never a wrapped address."""
    top = 1 << 40
    assert _accepted(lib, lib.gs_quantize_fp8(ROOM, 0, 1, top, 128, 0, _ref(_fp8(data=1 << 44, scale=1 << 43, stride=128)), None))
    assert lib.gs_quantize_fp8(ROOM, top, 1, top, 128, 0, _ref(_fp8(stride=1 << 39, block=0)), None) == ARG
    assert lib.gs_quantize_fp8(ROOM, 1, top, top, (1 << 30) - 1, 0, _ref(_fp8(stride=1 << 39, block=top)), None) == ARG
