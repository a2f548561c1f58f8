"""8-bit values and their matrix product on the GPU against the float64 ones.

Tolerances. Scales: one division, and the comparison of magnitudes is exact: 2^-23. A value is the nearest one to its quotient
(half a step) but for the rounding of the reciprocal and of the product with it (2^-23 of the quotient each). The product:
the tensor cores add 32 terms and the sum so far, aligned to the largest and cut below its float32 significand: at most 33
units of 2^-23 of the largest per addition, four additions a block, so 132 x 2^-23 < 2^-15 of the sum of the block's magnitudes
in the worst case, all errors of one sign; the blocks' sums are multiplied by scales (2 x 2^-24) and added in float32 (2^-24
for each block); the result is rounded once.
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
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


def _np(t):
    return t.double().cpu().numpy()


def _rand(shape, dtype, seed, factor=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    spread = torch.rand(shape[-1], device=DEV, generator=g) * 2
    return (torch.randn(shape, device=DEV, generator=g) * spread * factor).to(dtype)


def _bits(*ts):
    return [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in ts]


def _check_quantize(x, block, **kw):
    q, s = api.gs_quantize_fp8(x, block, **kw)
    X = _np(x)
    rs = fp8.scales(X, block)
    assert q.shape == x.shape and s.shape == rs.shape
    assert (np.abs(_np(s) - rs) <= 2.0 ** -23 * rs).all()
    each = fp8.spread(_np(s), X.shape) if block == 1 or x.shape[0] > 1 else np.repeat(_np(s), 128, 1)[:, :X.shape[1]]
    v = X / each
    assert (np.abs(_np(q) - v) <= fp8.step(np.abs(v) * (1 + 2.0 ** -22)) / 2 + 2.0 ** -22 * np.abs(v)).all()
    assert (np.abs(_np(q)) <= 448).all()
    return q, s


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 130), (128, 128), (129, 127), (130, 257), (70, 4), (9, 1000), (1000, 9), (511, 384), (256, 1030)])
def test_quantize(rows, cols, dtype, block, transposed):
    x = _rand((cols, rows), dtype, rows + cols).t() if transposed else _rand((rows, cols), dtype, rows + cols)
    _check_quantize(x, block)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("cols", [1, 96, 100, 128, 129, 200, 256, 257, 384, 500, 512, 520, 1024, 1032])
def test_quantize_few_columns(cols, dtype):
    for rows in (1, 5, 31, 33, 1000):  # warps beside one another, or below
        room = torch.full((rows + 1, (cols + 15) // 16 * 16 + 16), 0x55, dtype=torch.uint8, device=DEV)
        scales = torch.full((rows + 2, -(-cols // 128)), 3.0, device=DEV)
        _check_quantize(_rand((rows, cols), dtype, rows + cols), 1, out=(room[:rows, :cols].view(torch.float8_e4m3fn), scales[1:-1]))
        assert (room[rows:] == 0x55).all() and (room[:, cols:] == 0x55).all() and (scales[0] == 3).all() and (scales[-1] == 3).all()


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_strides_offsets_and_the_callers_tensors(block):
    base = _rand((300, 400), torch.bfloat16, 3)
    for x in (base[:, 3:203], base[:, 4:204], base[7:, 8:136], base[1:260:2, :130], base.t()[3:203], base.t()[4:204, ::2], base.t()[:, 1:131],
              base[:1], base[:, :1], base.t()[:, :1], base.t()[:1]):
        q, s = _check_quantize(x, block)
        wide = torch.full((x.shape[0], 512), 77, dtype=torch.uint8, device=DEV)
        room = torch.full((2 * s.shape[0], 2 * s.shape[1]), 5.0, device=DEV)
        got = api.gs_quantize_fp8(x, block, out=(wide.view(torch.float8_e4m3fn)[:, 16:16 + x.shape[1]], room[::2, ::2]))
        assert all(torch.equal(a, b) for a, b in zip(_bits(*got), _bits(q, s)))
        wide[:, 16:16 + x.shape[1]] = 77
        room[::2, ::2] = 5
        assert (wide == 77).all() and (room == 5).all()  # nothing beside them


def test_quantize_zeros_tiny_and_non_finite_blocks():
    x = torch.zeros(256, 512, device=DEV)
    x[0, 0], x[1, 1], x[2, 130] = float("nan"), float("inf"), -float("inf")
    x[3, 5], x[4, 260], x[5, 390], x[6, 400] = 1e-38, 1e-36, 3e38, 448 * 2.0 ** -126
    q, s = api.gs_quantize_fp8(x)
    assert s[0, 0].isnan() and q[0, :128].float().isnan().all() and (s[0, 1:] == 1).all() and (q[0, 128:].float() == 0).all()
    for r, c in ((1, 1), (2, 130)):
        b = c // 128
        assert s[r, b].isinf() and q[r, c].float().isnan() and (q[r, b * 128:c].float() == 0).all()
    assert s[3, 0] == 1 and q[3, 5].float() == 0 and s[6, 3] == 2.0 ** -126 and q[6, 400].float() == 448
    assert s[4, 2] == 1 and q[4, 260].float() == 0  # 1e-36 / 448 is below 2^-126 = 1.2e-38
    assert (q[5, 390].float() * s[5, 3] / x[5, 390] - 1).abs() < 1e-6 and q[5, 390].float() == 448
    for block in (1, 128):
        for t in (x, x.t()):
            a, b = api.gs_quantize_fp8(t, block)
            c, d = api.gs_quantize_fp8(t.contiguous(), block)
            assert torch.equal(a.float().nan_to_num(-1), c.float().nan_to_num(-1)) and torch.equal(b.nan_to_num(-1), d.nan_to_num(-1))


def _check_matmul(qa, sa, qb, sb, dtype, out=None):
    got = api.gs_matmul_fp8(qa, sa, qb, sb, dtype=dtype, out=out)
    want, size = fp8.matmul(_np(qa), _np(sa), _np(qb), np.repeat(_np(sb), 128, 0)[:len(qb)] if sb.shape[0] != len(qb) else _np(sb))
    tol = size * (2.0 ** -15 + (2 + sa.shape[1]) * 2.0 ** -24) + U[dtype] * np.abs(want) + TINY[dtype]
    assert got.dtype == dtype and got.shape == want.shape
    assert (np.abs(_np(got) - want) <= tol).all(), np.max(np.abs(_np(got) - want) / tol)
    return got


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 14, 128), (1, 4096, 1024), (2, 130, 100), (16, 256, 384), (17, 128, 129), (33, 333, 1000), (64, 64, 2048),
                                   (65, 14, 128), (128, 128, 128), (129, 127, 130), (300, 260, 96), (500, 1000, 515), (2000, 256, 1024)])
def test_matmul(m, n, k, dtype, block):
    qa, sa = api.gs_quantize_fp8(_rand((m, k), torch.float32, m + n + k))
    qb, sb = api.gs_quantize_fp8(_rand((n, k), torch.float32, m + n + k + 1), block)
    _check_matmul(qa, sa, qb, sb, dtype)


@pytest.mark.parametrize("m,n,k,block", [(4346, 1024, 1024, 128), (2200, 2304, 640, 128), (5000, 2100, 300, 1), (8, 14000, 4096, 128), (1024, 1024, 8700, 1),
                                         (20000, 1030, 128, 128), (20001, 2049, 260, 128)])
def test_matmul_large(m, n, k, block):
    qa, sa = api.gs_quantize_fp8(_rand((m, k), torch.bfloat16, 1))
    qb, sb = api.gs_quantize_fp8(_rand((n, k), torch.bfloat16, 2), block)
    got = api.gs_matmul_fp8(qa, sa, qb, sb, dtype=torch.float32)
    a = (qa.double().cpu() * sa.cpu().double().repeat_interleave(128, 1)[:, :k])
    b = (qb.double().cpu() * sb.cpu().double().repeat_interleave(block, 0)[:n].repeat_interleave(128, 1)[:, :k])
    at = torch.randperm(m, generator=torch.Generator().manual_seed(0))[:300]
    want, size = a[at] @ b.t(), a[at].abs() @ b.t().abs()
    tol = size * (2.0 ** -15 + (2 + sa.shape[1]) * 2.0 ** -24) + 2.0 ** -24 * want.abs()
    assert ((got.cpu()[at].double() - want).abs() <= tol).all()
    for dtype in (torch.bfloat16, torch.float16):  # the same sums, rounded
        assert torch.equal(api.gs_matmul_fp8(qa, sa, qb, sb, dtype=dtype), got.to(dtype))


def test_matmul_strides_offsets_and_the_callers_result():
    base = _rand((150, 600), torch.bfloat16, 5)
    qa, sa = api.gs_quantize_fp8(base)
    qb, sb = api.gs_quantize_fp8(_rand((90, 600), torch.bfloat16, 6), 128)
    # rows and columns of larger tensors; scales in another order
    for m in (150, 40, 1):
        rows = slice(3, 3 + 2 * m, 2) if m < 150 else slice(None)
        a, b = qa[rows, 128:400], qb[:, 128:400]
        s, t = sa[rows, 1:4].contiguous(), sb[:, 1:4].contiguous()
        want = _check_matmul(a, s, b, t, torch.bfloat16)
        m = len(want)
        for pad in (0, 3, 6, 38):
            room = torch.full((m + 2, 90 + 2 * pad), 9.0, dtype=torch.bfloat16, device=DEV)
            got = api.gs_matmul_fp8(a, s, b, t, out=room[1:m + 1, pad:pad + 90])
            assert torch.equal(got, want)
            room[1:m + 1, pad:pad + 90] = 9
            assert (room == 9).all()
    # one scale for all
    one = torch.ones(1, 1, device=DEV)
    assert torch.equal(api.gs_matmul_fp8(qa, one.expand(150, 5), qb, one.expand(1, 5), dtype=torch.float32),
                       api.gs_matmul_fp8(qa, torch.ones(150, 5, device=DEV), qb, torch.ones(1, 5, device=DEV), dtype=torch.float32))


def test_matmul_of_nothing():
    q, s = api.gs_quantize_fp8(torch.ones(5, 0, device=DEV))
    assert (api.gs_matmul_fp8(q, s, *api.gs_quantize_fp8(torch.ones(7, 0, device=DEV), 128)) == torch.zeros(5, 7, device=DEV)).all()
    big = torch.ones(300, 0, device=DEV)
    assert (api.gs_matmul_fp8(*api.gs_quantize_fp8(big), *api.gs_quantize_fp8(big)) == torch.zeros(300, 300, device=DEV)).all()
    q, s = api.gs_quantize_fp8(torch.ones(0, 64, device=DEV))
    w = api.gs_quantize_fp8(torch.ones(7, 64, device=DEV), 128)
    assert api.gs_matmul_fp8(q, s, *w).shape == (0, 7)
    assert api.gs_matmul_fp8(*w[:1], torch.ones(7, 1, device=DEV), q, s).shape == (7, 0)


def test_matmul_of_values_that_are_not_finite():
    for m in (3, 200):
        x, w = torch.ones(m, 256, device=DEV), torch.ones(130, 256, device=DEV)
        x[1, 5] = float("nan")
        w[7, 200] = float("inf")
        out = api.gs_matmul_fp8(*api.gs_quantize_fp8(x), *api.gs_quantize_fp8(w))
        bad = out.isnan()
        assert bad[1].all() and bad[:, 7].all() and bad.sum() == 130 + m - 1
        assert (out[~bad] == 256).all()
    big = torch.full((4, 128), 3e4, device=DEV)
    assert api.gs_matmul_fp8(*api.gs_quantize_fp8(big), *api.gs_quantize_fp8(big), dtype=torch.float16).isinf().all()


def test_a_projection_and_its_gradients():
    # y = norm(x) w^T in 8 bits and its way back, as a training step runs them, against the same products of the values
    # that the 8-bit tensors stand for
    rows, c, n = 700, 320, 200
    x, w, dy = _rand((rows, c), torch.bfloat16, 1), _rand((n, c), torch.float32, 2, 0.1), _rand((rows, n), torch.bfloat16, 3)
    q, s, _, rstd = api.gs_rms_norm_fp8(x, torch.ones(c, device=DEV))
    _check_matmul(q, s, *api.gs_quantize_fp8(w, 128), torch.bfloat16)
    dt = _check_matmul(*api.gs_quantize_fp8(dy), *api.gs_quantize_fp8(w.t(), 128), torch.bfloat16)
    y = api.gs_rms_norm_fwd(x, torch.ones(c, device=DEV))[0]
    dw = _check_matmul(*api.gs_quantize_fp8(dy.t()), *api.gs_quantize_fp8(y.t()), torch.float32)
    dx, _ = api.gs_rms_norm_bwd(dt, x, rstd)
    # 8-bit roundings, 2^-4 of each factor at most, leave the directions of the gradients
    X, W, D = x.double(), w.double(), dy.double()
    X = X.requires_grad_()
    W = W.requires_grad_()
    ((X * (X.square().mean(1, keepdim=True) + 1e-6).rsqrt() @ W.t()) * D).sum().backward()
    for got, want in ((dx, X.grad), (dw, W.grad)):
        assert (got.double() - want).norm() <= 2 * 2.0 ** -4 * want.norm()


def test_weights_blocks_are_the_same_transposed():
    w = _rand((300, 450), torch.float32, 4)
    q, s = api.gs_quantize_fp8(w, 128)
    qt, st = api.gs_quantize_fp8(w.t(), 128)
    assert torch.equal(q.float().t(), qt.float()) and torch.equal(s.t(), st)


def test_streams_capture_and_the_same_bits_twice():
    qa, sa = api.gs_quantize_fp8(_rand((1000, 1024), torch.bfloat16, 1))
    qb, sb = api.gs_quantize_fp8(_rand((512, 1024), torch.bfloat16, 2), 128)
    x = _rand((1000, 1024), torch.bfloat16, 1)
    one, s1 = qa[:1], sa[:1]
    want = api.gs_matmul_fp8(qa, sa, qb, sb), api.gs_matmul_fp8(one, s1, qb, sb)
    side = [torch.cuda.Stream() for _ in range(3)]
    got = []
    torch.cuda.synchronize()
    for i in range(30):  # many at once
        st = side[i % 3]
        got.append((api.gs_matmul_fp8(qa, sa, qb, sb, stream=st), api.gs_matmul_fp8(one, s1, qb, sb, stream=st)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s = api.gs_quantize_fp8(x)
        out = api.gs_matmul_fp8(q, s, qb, sb), api.gs_matmul_fp8(q[:1], s[:1], qb, sb)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    x.mul_(2)  # new inputs of a replay
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0] * 2)
    assert api.gs_device_error() == _abi.GS_OK


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    q, s = api.gs_quantize_fp8(x)
    for bad in (lambda: api.gs_quantize_fp8(x.double()), lambda: api.gs_quantize_fp8(x, 64), lambda: api.gs_quantize_fp8(x[:, ::2]),
                lambda: api.gs_quantize_fp8(x, out=(x, s)), lambda: api.gs_quantize_fp8(x, out=(q[:2], s)), lambda: api.gs_quantize_fp8(x, out=(q, s[:2])),
                lambda: api.gs_matmul_fp8(x, s, q, s), lambda: api.gs_matmul_fp8(q, s[:2], q, s), lambda: api.gs_matmul_fp8(q, s, q, s.half()),
                lambda: api.gs_matmul_fp8(q, s, q[:, :48], s), lambda: api.gs_matmul_fp8(q, s, q, s.flatten()), lambda: api.gs_matmul_fp8(q, s, q, s[:3]),
                lambda: api.gs_matmul_fp8(q, s, q, s, out=torch.zeros(4, 5, device=DEV)),
                lambda: api.gs_matmul_fp8(q, s, q, s, dtype=torch.float16, out=torch.zeros(4, 4, device=DEV)),
                lambda: api.gs_matmul_fp8(q.cpu(), s, q, s), lambda: api.gs_matmul_fp8(q, s.cpu(), q, s), lambda: api.gs_matmul_fp8(q, s, q, s, dtype=torch.int8)):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(4, 200, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[:, :64]
    for bad in (lambda: api.gs_matmul_fp8(odd, s, q, s), lambda: api.gs_matmul_fp8(q, s, odd, s), lambda: api.gs_quantize_fp8(x, out=(odd, s)),
                lambda: api.gs_matmul_fp8(q[:, 8:], s, q[:, 8:], s)):
        with pytest.raises(_abi.GsError, match="16"):
            bad()
