"""The 8-bit decoder's operators where offsets pass 32 bits: the last rows as those rows alone give them, and calls on tensors of
more than two dimensions."""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _tail(rows, cols, n, dtype):
    """Rows of which only the last n are not zeros."""
    x = torch.zeros(rows, cols, dtype=dtype, device=DEV)
    x[-n:] = torch.randn(n, cols, device=DEV, generator=torch.Generator(device="cuda").manual_seed(rows)).to(dtype)
    return x


def _same(a, b):
    a, b = (t.contiguous().view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (a, b))
    return torch.equal(a, b)


@pytest.mark.parametrize("cols", [8192, 8191, 260, 20000])
def test_norm_of_many_rows(cols):
    rows, n = 2 ** 31 // cols + 300, 50
    x = _tail(rows, cols, n, torch.bfloat16)
    w = torch.rand(cols, device=DEV) + 0.5
    y, h, rstd = api.gs_rms_norm_fwd(x, w, x)
    few = api.gs_rms_norm_fwd(x[-n:].contiguous(), w, x[-n:].contiguous())
    assert torch.equal(y[-n:], few[0]) and torch.equal(h[-n:], few[1]) and torch.equal(rstd[-n:], few[2]) and not y[:-n].any()
    q, s, _, _ = api.gs_rms_norm_fp8(x, w, out=(torch.empty(rows, (cols + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device=DEV)[:, :cols],
                                                torch.empty(rows, -(-cols // 128), device=DEV), None, rstd))
    few = api.gs_rms_norm_fp8(x[-n:].contiguous(), w)
    assert _same(q[-n:], few[0]) and torch.equal(s[-n:], few[1]) and (s[:-n] == 1).all()
    del q, s, y
    rstd = api.gs_rms_norm_fwd(h, w, out=(h, None, rstd))[2].clamp(max=1e3)  # h is now the norm
    dx, dw = api.gs_rms_norm_bwd(x, h, rstd, w, x)
    few = api.gs_rms_norm_bwd(x[-n:].contiguous(), h[-n:].contiguous(), rstd[-n:].contiguous(), w, x[-n:].contiguous())
    assert torch.equal(dx[-n:], few[0]) and not dx[:-n].any()
    # sums of n terms that are not zeros, in another order
    size = (x[-n:].float() * h[-n:].float() * rstd[-n:, None]).abs().sum(0)
    assert ((dw - few[1]).abs() <= 2 * n * 2.0 ** -24 * size).all()
    assert api.gs_device_error() == _abi.GS_OK


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("cols", [16384, 16381])
def test_quantize_of_many_values(cols, transposed, block):
    rows = 2 ** 31 // cols // 128 * 128 + 256
    if transposed:  # the last columns, of all rows
        x = _tail(cols, rows, 130, torch.float16).t()
        q, s = api.gs_quantize_fp8(x, block)
        at = (cols - 130) // 128 * 128
        few = api.gs_quantize_fp8(x.t()[at:].contiguous().t(), block)
        assert _same(q[:, at:], few[0]) and torch.equal(s[:, at // 128:], few[1]) and (s[:, :at // 128] == 1).all()
        return
    x = _tail(rows, cols, 256, torch.float16)
    q, s = api.gs_quantize_fp8(x, block)
    few = api.gs_quantize_fp8(x[-256:].contiguous(), block)
    assert _same(q[-256:], few[0]) and torch.equal(s[-256 // block:], few[1]) and (s[:-256 // block] == 1).all()


@pytest.mark.parametrize("m,n,k,block", [(140000, 16384, 128, 128), (140001, 16381, 70, 1), (16384, 140000, 128, 128), (60, 2 ** 31 // 60 + 500, 16, 128),
                                         (17000, 400, 131072, 128)])
def test_products_of_many_elements(m, n, k, block):
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, w = (torch.randint(-4, 5, (r, k), device=DEV, generator=gen, dtype=torch.int8) for r in (m, n))
    pad = (k + 15) // 16 * 16
    ones = (torch.ones(m, -(-k // 128), device=DEV), torch.ones(-(-n // block), -(-k // 128), device=DEV))
    a, b = (torch.zeros(len(t), pad, dtype=torch.float8_e4m3fn, device=DEV)[:, :k].copy_(t) for t in (x, w))
    out = api.gs_matmul_fp8(a, ones[0], b, ones[1], dtype=torch.float32 if k < 1000 else torch.bfloat16)
    # whole numbers below 2^24, exact in float32
    for rows in (slice(0, 40), slice(m - 40, m)):
        for columns in (slice(0, 300), slice(n - 300, n)):
            want = x[rows].float() @ w[columns].float().t() if k < 1000 else (x[rows].double() @ w[columns].double().t())
            assert torch.equal(out[rows, columns], want.to(out.dtype))
    assert api.gs_device_error() == _abi.GS_OK


def test_clip_of_many_elements():
    n = 2 ** 31 + 4097
    g = torch.zeros(n, device=DEV)
    g[-5:] = 3.0
    h = torch.full((10,), 2.0, device=DEV, dtype=torch.float16)
    norm = api.gs_clip_grads([g, h], 1.0, eps=0.0)
    want = (5 * 9 + 10 * 4) ** 0.5
    assert abs(norm.item() - want) <= 2 ** -23 * want
    assert ((g[-5:] - 3 / want).abs() <= 2 ** -22 * 3 / want).all() and not g[:-5].any()


def test_more_than_two_dimensions():
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(3, 5, 7, 256, device=DEV, generator=gen, dtype=torch.bfloat16)
    flat = x.view(-1, 256)
    y, h, rstd = api.gs_rms_norm_fwd(x, None, x)
    assert y.shape == h.shape == x.shape and rstd.shape == (105,) and torch.equal(y.view(-1, 256), api.gs_rms_norm_fwd(flat, None, flat)[0])
    q, s = api.gs_quantize_fp8(x)
    assert q.shape == x.shape and _same(q.view(-1, 256), api.gs_quantize_fp8(flat)[0]) and s.shape == (105, 2)
    w, ws = api.gs_quantize_fp8(torch.randn(40, 256, device=DEV, generator=gen), 128)
    out = api.gs_matmul_fp8(q, s, w, ws)
    assert out.shape == (3, 5, 7, 40) and torch.equal(out.view(-1, 40), api.gs_matmul_fp8(q.view(-1, 256), s, w, ws))
    room = torch.zeros(3, 5, 7, 48, device=DEV, dtype=torch.bfloat16)
    assert torch.equal(api.gs_matmul_fp8(q, s, w, ws, out=room[..., :40]), out) and not room[..., 40:].any()
    dx, _ = api.gs_rms_norm_bwd(x, h, rstd, None, x)
    assert dx.shape == x.shape and torch.equal(dx.view(-1, 256), api.gs_rms_norm_bwd(flat, h.view(-1, 256), rstd, None, flat)[0])
    one = api.gs_matmul_fp8(q[0, 0, 0], s[:1], w, ws)  # a vector
    assert one.shape == (40,) and torch.equal(one, api.gs_matmul_fp8(q[0, 0, 0][None], s[:1], w, ws)[0])
