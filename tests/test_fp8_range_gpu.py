"""8-bit products whose scales reach the ends of float32's range: what the values and their scales give is a float32 number,
although the scales' product, or a value times one scale, is not.

Tolerance: as in test_fp8_gpu.py, 2^-15 of the sum of the block's magnitudes for the tensor cores, three roundings of 2^-24 for
a block's scales and one for each addition; below the normal numbers each of these is half of 2^-149 instead.
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
# rows along the lanes or the columns, alone, in clusters that share the inner dimension, tiles of 64 to 256 columns, pairs
FORMS = [(1, 300, 1100, 128), (20, 333, 700, 1), (60, 500, 260, 128), (70, 130, 900, 128), (300, 200, 500, 1), (1300, 1000, 300, 128), (1300, 1000, 300, 1),
         (2500, 1280, 260, 128), (2500, 1280, 260, 1)]


def _tensors(m, n, k, block, seed, exponent_a, exponent_b, q=None):
    """8-bit values and scales 2^exponent times 1 to 2: exponents of [rows, blocks]."""
    g = np.random.default_rng(seed)
    got = []
    for rows, blk, exponent in ((m, 1, exponent_a), (n, block, exponent_b)):
        values = q(rows, k, len(got) // 2) if q else fp8.round_e4m3(g.standard_normal((rows, k)) * 60)
        scale = np.ldexp(1 + g.random((-(-rows // blk), -(-k // 128))), exponent(g, (-(-rows // blk), -(-k // 128)))).astype(np.float32)
        pad = torch.zeros(rows, (k + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device=DEV)[:, :k]
        pad.copy_(torch.from_numpy(values).to(DEV).float())
        got += [pad, torch.from_numpy(scale).to(DEV)]
    return got


def _wanted(qa, sa, qb, sb):
    a, s, b, t = (x.double().cpu().numpy() for x in (qa, sa, qb, sb))
    return fp8.matmul(a, s, b, t if t.shape[0] == len(b) else np.repeat(t, 128, 0)[:len(b)])


def _check(qa, sa, qb, sb):
    got = api.gs_matmul_fp8(qa, sa, qb, sb, dtype=torch.float32)
    want, size = _wanted(qa, sa, qb, sb)
    assert np.abs(want).max() < 2.0 ** 127
    blocks = sa.shape[1]
    tol = size * (2.0 ** -15 + (3 + blocks) * 2.0 ** -24) + 2.0 ** -24 * np.abs(want) + (4 + blocks) * 2.0 ** -149
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), np.nanmax(err / tol)
    assert torch.equal(api.gs_matmul_fp8(qa, sa, qb, sb, dtype=torch.bfloat16), got.to(torch.bfloat16))
    assert api.gs_device_error() == _abi.GS_OK
    return got


def _level(e):
    return lambda g, shape: np.full(shape, e)


@pytest.mark.parametrize("m,n,k,block", FORMS)
@pytest.mark.parametrize("ea,eb", [(-75, -60), (-60, -75), (-70, -56), (-126, -20), (-90, -90), (110, -110), (-110, 110), (119, -126), (-126, 119), (80, -100), (-149, 100),
                                   (60, 40)])
def test_scales_that_leave_float32_alone_or_together(m, n, k, block, ea, eb):
    _check(*_tensors(m, n, k, block, 1, _level(ea), _level(eb)))


@pytest.mark.parametrize("m,n,k,block", FORMS)
def test_large_values_that_do_not_meet(m, n, k, block):
    # blocks whose large elements stand beside zeros of the other operand: sums of 0, and not 0 times an infinity
    def apart(rows, k, which):
        q = np.zeros((rows, k))
        q[:, which::2] = 448
        return q

    for ea, eb in ((75, 75), (119, 119), (75, 119)):
        out = api.gs_matmul_fp8(*_tensors(m, n, k, block, 2, _level(ea), _level(eb), apart), dtype=torch.float32)
        assert (out == 0).all(), (ea, eb)
    big = 1e25
    x, w = torch.zeros(m, k, device=DEV), torch.zeros(n, k, device=DEV)
    x[:, ::2], w[:, 1::2] = big, big
    assert (api.gs_matmul_fp8(*api.gs_quantize_fp8(x), *api.gs_quantize_fp8(w, block), dtype=torch.float32) == 0).all()


@pytest.mark.parametrize("m,n,k,block", FORMS)
def test_exponents_of_every_row_and_block(m, n, k, block):
    for low, high in ((-126, 30), (-100, 50), (-149, -10)):
        _check(*_tensors(m, n, k, block, low + 200, lambda g, shape: g.integers(low, high, shape), lambda g, shape: g.integers(low, high, shape)))


@pytest.mark.parametrize("m,n,k,block", FORMS)
def test_small_maxima(m, n, k, block):
    # maxima of 1e-18 on both sides: results around 1e-34
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w = (torch.randn(r, k, device=DEV, generator=g) * 3e-19 for r in (m, n))
    out = _check(*api.gs_quantize_fp8(x), *api.gs_quantize_fp8(w, block))
    exact = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    assert ((out.double() - exact).abs() <= (2 * 2.0 ** -4 + 2.0 ** -8 + 2.0 ** -14) * size + 300 * 2.0 ** -9 * size.max()).all()


@pytest.mark.parametrize("m,n,k,block", FORMS)
def test_rows_and_columns_beside_extreme_ones_keep_their_bits(m, n, k, block):
    qa, sa, qb, sb = _tensors(m, n, k, block, 5, _level(-3), _level(2))
    want = api.gs_matmul_fp8(qa, sa, qb, sb, dtype=torch.float32)
    a, b = sa.clone(), sb.clone()
    a[::3, 0] *= 2.0 ** -120
    b[1::2, -1] *= 2.0 ** 100
    got = _check(qa, a, qb, b)
    rows = torch.arange(m, device=DEV) % 3 != 0
    columns = (torch.arange(n, device=DEV) // block) % 2 == 0
    assert torch.equal(got[rows][:, columns], want[rows][:, columns])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k,block", FORMS)
def test_inside_larger_buffers_and_captured(m, n, k, block, dtype):
    # every third row outside (by column: every second column), what lies behind the rows is NaN
    qa, sa, qb, sb = _tensors(m, n, k, block, 6, _level(-3), _level(-1))
    sa[::3] *= 2.0 ** -122
    if block == 1:
        sb[::2] *= 2.0 ** 111
    want = api.gs_matmul_fp8(qa, sa, qb, sb, dtype=torch.float32)
    wide = [torch.full((2 * r, (k + 15) // 16 * 16 + 32), 0x7F, dtype=torch.uint8, device=DEV) for r in (m, n)]  # NaN
    a, b = (w[::2, 16:16 + k] for w in wide)
    a.copy_(qa.view(torch.uint8)), b.copy_(qb.view(torch.uint8))
    a, b = a.view(torch.float8_e4m3fn), b.view(torch.float8_e4m3fn)
    room = torch.full((m + 2, n + 19), 5.0, device=DEV, dtype=dtype)
    out = room[1:m + 1, 3:3 + n]
    api.gs_matmul_fp8(a, sa.t().contiguous().t(), b, sb.t().contiguous().t(), out=out)
    assert torch.equal(out, want.to(dtype))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        api.gs_matmul_fp8(a, sa, b, sb, out=out)
    out.fill_(0)
    sa.mul_(2)  # new scales of a replay
    graph.replay()
    torch.cuda.synchronize()
    again = api.gs_matmul_fp8(qa, sa, qb, sb, dtype=torch.float32)
    assert torch.equal(out, again.to(dtype))
    out.fill_(5)
    assert (room == 5).all() and api.gs_device_error() == _abi.GS_OK


def test_several_at_once_with_ordinary_ones():
    cases = []
    for i, (m, n, k, block) in enumerate(FORMS):
        for ea, eb in ((-70, -70), (-2, 1)):
            t = _tensors(m, n, k, block, i, _level(ea), _level(eb if block == 128 or eb > 0 else -115))
            cases.append((t, api.gs_matmul_fp8(*t, dtype=torch.float32)))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [(api.gs_matmul_fp8(*t, dtype=torch.float32, stream=streams[(i + j) % 4]), want) for j in range(3) for i, (t, want) in enumerate(cases)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got) and api.gs_device_error() == _abi.GS_OK
