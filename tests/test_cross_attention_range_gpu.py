"""GPU cross attention, forward: probabilities far below the largest one.

A few keys take nearly all the weight and have values of zero, so that the output is what thousands of others contribute,
each 12 to 18 nats lower. float16's own range then decides how P is formed: with the largest key at 2^12, one 18 nats
(26 bits) lower is 2^-14, a normal number with its relative rounding of 2^-11.

Tolerance: a score and lse are off by at most 2^-20 of scale sum |q||k|, a probability by that, by 2^-20 for the
exponential and the sum, and by twice the type's unit roundoff; out is off by its probabilities' errors against sum P |v|
and rounded once (float16: to half the spacing of its subnormal numbers at least).
"""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
ACC = 2.0 ** -20


def _check(q, k, v):
    out, lse = api.gs_cross_attention_fwd(q, k, v)
    assert torch.isfinite(out).all()
    u, share = U[q.dtype], q.shape[2] // k.shape[2]
    for h in range(q.shape[2]):
        a, b, w = q[0, :, h].double(), k[0, :, h // share].double(), v[0, :, h // share].double()
        scale = a.shape[1] ** -0.5
        s = a @ b.t() * scale
        p = torch.softmax(s, 1)
        size = (a.abs() @ b.abs().t() * scale).amax(1)
        want, want_lse = p @ w, torch.logsumexp(s, 1)
        tol = (2 * u + ACC + 2 * ACC * size[:, None]) * (p @ w.abs()) + u * want.abs() + TINY[q.dtype]
        bad = (out[0, :, h].double() - want).abs() / tol
        assert (bad <= 1).all(), (h, bad.max().item())
        assert ((lse[0, h].double() - want_lse).abs() <= ACC * (1 + size + want_lse.abs())).all()
    assert api.gs_device_error() == _abi.GS_OK


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("len_q,heads,kv_heads,d", [(1, 2, 2, 64), (1, 4, 2, 64), (128, 2, 2, 64), (300, 2, 2, 40), (150, 2, 1, 128),
                                                    (140, 1, 1, 200)])
@pytest.mark.parametrize("others,below", [(399, 12.0), (399, 15.5), (2500, 16.0), (4346, 17.5), (4346, 18.0)])
@pytest.mark.parametrize("peaks", [(0,), (200,), (-1,), (3, 130, 131, -1)])
def test_values_that_only_low_probabilities_carry(dtype, len_q, heads, kv_heads, d, others, below, peaks):
    gen = torch.Generator(device="cuda").manual_seed(others + len_q)
    n = others + len(peaks)
    q = torch.zeros(1, len_q, heads, d, device=DEV)
    q[:, :, :, 1] = d ** 0.5
    k = torch.zeros(1, n, kv_heads, d, device=DEV)
    k[:, :, :, 1] = -below
    v = 0.5 + torch.rand(1, n, kv_heads, d, device=DEV, generator=gen)
    for at in peaks:
        k[:, at, :, 1] = 0.0
        v[:, at] = 0.0
    _check(*(t.to(dtype) for t in (q, k, v)))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("len_q,d", [(128, 64), (300, 64), (140, 128), (70, 256)])
@pytest.mark.parametrize("spread", [0.0, 1.5, 5.0, 12.0])
def test_scores_that_rise_from_tile_to_tile(dtype, len_q, d, spread):
    # every key tile's scores pass those before by up to 3.4, the last ones come back
    gen = torch.Generator(device="cuda").manual_seed(int(spread) + d)
    n = 128 * 14 + 60
    rand = lambda *s: torch.randn(1, *s, device=DEV, generator=gen)  # noqa: E731
    q, k, v = spread * rand(len_q, 2, d), rand(n, 2, d), rand(n, 2, d)
    q[:, :, :, 0] = d ** 0.5
    rise = torch.cumsum(torch.rand(15, device=DEV, generator=gen) * 3.4, 0)
    rise[11:] = rise[2:6]
    k[:, :, :, 0] = rise.repeat_interleave(128)[None, :n, None]
    _check(*(t.to(dtype) for t in (q, k, v)))
