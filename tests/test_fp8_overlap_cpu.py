"""Overlaps of strided tensors: the calls refuse those in which a byte that is written is one that is read or written besides, and
no others (CPU, addresses that are never read)."""
import ctypes as C
import random

import pytest
import torch

import __graft_entry__
from differentiable_gaussian_splatting_gs_gb300 import _abi

if torch.cuda.is_available():
    pytest.skip("made-up addresses: only where no device could follow them", allow_module_level=True)

ARG = _abi.GS_ERR_ARG
ROOM = 1 << 32


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _abi.load()


def _fp8(data, stride, scale, row, block, rows=1):
    return _abi.gs_fp8(data=data, stride=stride, scale=scale, scale_row=row, scale_block=block, block_rows=rows)


def _lies_on(lib, status):
    """Refused for an overlap; past the checks otherwise (there is no device to go on with)."""
    if status == ARG:
        assert b"lies on" in lib.gs_last_error_message(), lib.gs_last_error_message()
        return True
    assert status == _abi.GS_ERR_CUDA
    return False


def _bytes(start, rows, length, stride):
    return {start + r * stride + i for r in range(rows) for i in range(length)}


def test_values_and_x_of_other_strides(lib):
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(4000):
        rows, cols, wide = rng.randint(1, 9), rng.randint(1, 40), rng.choice([0, 1, 2])
        size = 4 if wide == 0 else 2
        xs, qs = cols + rng.randint(0, 60), (cols + 15) // 16 * 16 + 16 * rng.randint(0, 12)
        x, q = ROOM + size * rng.randint(0, 700 // size), ROOM + 16 * rng.randint(0, 60)
        want = bool(_bytes(x, rows, cols * size, xs * size) & _bytes(q, rows, cols, qs))
        t = _fp8(q, qs, 2 * ROOM, 1, rows)
        assert _lies_on(lib, lib.gs_quantize_fp8(x, xs, 1, rows, cols, wide, C.byref(t), None)) == want, (x - ROOM, xs, q - ROOM, qs, rows, cols, size)
        seen[want] += 1
    assert min(seen) > 500, seen


def test_results_between_rows_of_operands(lib):
    rng = random.Random(2)
    seen = [0, 0]
    for _ in range(4000):
        m, n, k = rng.randint(1, 7), rng.randint(1, 12), rng.randint(1, 30)
        at, os = ROOM + 16 * rng.randint(0, 20), n + rng.randint(0, 40)
        out, a_stride = ROOM + 4 * rng.randint(0, 120), 16 * rng.randint((k + 15) // 16, 9)
        a, b = _fp8(at, a_stride, 3 * ROOM, 1, m), _fp8(4 * ROOM, 128, 5 * ROOM, 1, n)
        want = bool(_bytes(out, m, 4 * n, 4 * os) & _bytes(at, m, k, a_stride))
        assert _lies_on(lib, lib.gs_matmul_fp8(C.byref(a), C.byref(b), m, n, k, 0, out, os, None)) == want, (out - ROOM, os, at - ROOM, a_stride, m, n, k)
        seen[want] += 1
    assert min(seen) > 500, seen


def test_many_rows_whose_gaps_hold_the_others(lib):
    # rows of 16 bytes 4096 apart and values of 16 bytes 8192 apart: in the gaps, or in one of a million rows
    rows = 1 << 20
    for start, want in ((2048, False), (4080, False), (4096 * 5, True), (8192 - 48, False), (8192 * 3 + 16, False), (8192 * 3, True)):
        t = _fp8(ROOM + start, 8192, 4 * ROOM * 64, 1, rows)
        assert _lies_on(lib, lib.gs_quantize_fp8(ROOM, 1024, 1, rows, 4, 0, C.byref(t), None)) == want, start
    # strides without a common factor of the rows' length: the first that meet are far in
    t = _fp8(ROOM + 64, 4112, 1 << 50, 1, rows)
    assert _lies_on(lib, lib.gs_quantize_fp8(ROOM, 1024, 1, rows, 4, 0, C.byref(t), None))
    assert not _lies_on(lib, lib.gs_quantize_fp8(ROOM, 1024, 1, 200, 4, 0, C.byref(t), None))  # row 252 is the first (64 + 252 x 16 = 4096)
    assert _lies_on(lib, lib.gs_quantize_fp8(ROOM, 1024, 1, 260, 4, 0, C.byref(t), None))


def test_scales_that_run_backwards_are_where_they_are(lib):
    def product(a, out):
        b = _fp8(10 * ROOM, 512, 11 * ROOM, 4, 1, 128)
        return _lies_on(lib, lib.gs_matmul_fp8(C.byref(a), C.byref(b), 256, 256, 512, 2, out, 256, None))

    a = _fp8(8 * ROOM, 512, 9 * ROOM, -4, 1)
    assert product(a, 9 * ROOM - 4096 * 2) and not product(a, 9 * ROOM + 16) and not product(a, 9 * ROOM - 4 * 4 * 255 - 131072)
    a = _fp8(8 * ROOM, 512, 9 * ROOM, 1, -256)
    assert product(a, 9 * ROOM - 4 * 256 * 3) and not product(a, 9 * ROOM + 4 * 256)


def test_strides_whose_products_pass_64_bits(lib):
    # 2^32 + 1 rows of blocks whose scales are 2^32 apart reach past the next column's, 2^36 away: 2^32 x 2^32 is not 0
    t = _fp8(8 * ROOM, 1 << 31, 1 << 50, 1 << 32, 1 << 36, 128)
    assert lib.gs_quantize_fp8(ROOM, 1 << 31, 1, 128 * ((1 << 32) + 1), 256, 0, C.byref(t), None) == ARG
    assert b"share memory" in lib.gs_last_error_message()


@pytest.mark.parametrize("dt,size", [(0, 4), (2, 2)])
def test_norms_outputs_on_weights_statistics_and_one_another(lib, dt, size):
    rows, cols = 64, 512

    def fwd(x=ROOM, r=2 * ROOM, w=3 * ROOM, h=4 * ROOM, y=5 * ROOM, rstd=6 * ROOM, q=None):
        return _lies_on(lib, lib.gs_rms_norm_fwd(x, cols, r, cols, rows, cols, dt, w, 0, 1e-6, h, cols, None if q else y, cols, q and C.byref(q), rstd, None))

    end = rows * cols * size
    assert not fwd() and not fwd(q=_fp8(7 * ROOM, cols, 8 * ROOM, 1, rows)) and not fwd(w=None)
    assert not fwd(rstd=ROOM + end) and not fwd(rstd=3 * ROOM + 4 * cols) and not fwd(h=3 * ROOM - end)
    for bad in (dict(h=3 * ROOM), dict(y=3 * ROOM + 4 * cols - 16), dict(rstd=3 * ROOM - 4), dict(rstd=ROOM + end - 4), dict(rstd=2 * ROOM), dict(rstd=4 * ROOM + 16),
                dict(rstd=5 * ROOM + 8)):
        assert fwd(**bad), bad
    t = _fp8(7 * ROOM, cols, 8 * ROOM, 1, rows)
    for bad in (dict(rstd=7 * ROOM + 16), dict(rstd=8 * ROOM + 4), dict(w=7 * ROOM), dict(w=8 * ROOM - 4)):
        assert fwd(q=t, **bad), bad
    assert not fwd(q=t, rstd=8 * ROOM + 4 * rows * 4)  # behind the scales

    def bwd(dy=ROOM, h=2 * ROOM, dh=3 * ROOM, rstd=4 * ROOM, w=5 * ROOM, dx=6 * ROOM, dw=7 * ROOM, ws=8 * ROOM):
        return _lies_on(lib, lib.gs_rms_norm_bwd(dy, cols, h, cols, dh, cols, rows, cols, dt, rstd, w, 0, dx, cols, dw, ws, 1 << 20, None))

    need = lib.gs_rms_norm_workspace_bytes(rows, cols)
    assert not bwd() and not bwd(dx=ROOM) and not bwd(dx=3 * ROOM) and not bwd(ws=ROOM - need) and not bwd(w=None, dw=None, ws=ROOM)
    assert not bwd(dw=5 * ROOM)  # written when the weights are read
    for bad in (dict(dx=4 * ROOM), dict(dx=5 * ROOM + 16), dict(dw=6 * ROOM + 8), dict(ws=7 * ROOM), dict(ws=6 * ROOM), dict(ws=5 * ROOM), dict(ws=4 * ROOM), dict(ws=3 * ROOM),
                dict(ws=2 * ROOM + end - 16), dict(ws=ROOM + 16 - need)):
        assert bwd(**bad), bad


def test_the_norm_and_the_workspace_of_clipping(lib):
    def clip(g=ROOM, out=None, n=1000, norm=2 * ROOM, ws=3 * ROOM, clip=1):
        t = (_abi.gs_gradient * 2)(_abi.gs_gradient(grad=4 * ROOM, out=None, n=10, dtype=2), _abi.gs_gradient(grad=g, out=out, n=n, dtype=0))
        return _lies_on(lib, lib.gs_clip_grads(t, 2, clip, 1.0, 1e-6, norm, ws, 1 << 20, None))

    assert not clip() and not clip(norm=ROOM + 4000) and not clip(out=5 * ROOM) and not clip(norm=ROOM + 16, clip=0) and not clip(norm=3 * ROOM - 4)
    for bad in (dict(norm=ROOM + 3996), dict(norm=4 * ROOM + 16), dict(out=5 * ROOM, norm=5 * ROOM), dict(out=5 * ROOM, norm=ROOM), dict(ws=ROOM + 3984), dict(ws=2 * ROOM),
                dict(out=5 * ROOM, ws=5 * ROOM), dict(ws=ROOM, clip=0), dict(ws=4 * ROOM)):
        assert clip(**bad), bad


def test_the_workspace_of_gradients_that_clipping_refuses(lib):
    def need(n):
        t = (_abi.gs_gradient * 2)(_abi.gs_gradient(grad=ROOM, out=None, n=10, dtype=0), _abi.gs_gradient(grad=4 * ROOM, out=None, n=n, dtype=0))
        return lib.gs_clip_workspace_bytes(t, 2)

    assert need(0) > 0 and need(1 << 40) > 0
    assert [need(n) for n in (-1, (1 << 40) + 1, (1 << 63) - 1)] == [0, 0, 0]
