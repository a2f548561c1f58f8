"""GPU cross attention, backward, 16-bit: sums over few rows in calls of many heads and batch entries.

Tolerance: with P in two parts (relative 2 u^2) dv = P^T dout is off by its own rounding and float32 accumulation alone;
without, by 1.4 times that rounding and more. 1.1 times it is allowed over all of dv, and 1.5 times over each key
head (1,000 elements and more, whose rounding errors' norm spreads by a few per cent).
"""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,h,hk,lq,lk,d", [(8, 16, 16, 5, 400, 64), (16, 48, 48, 1, 90, 32), (8, 16, 4, 5, 1000, 128), (4, 16, 16, 64, 300, 64),
                                            (8, 32, 2, 4, 260, 40)])
@pytest.mark.parametrize("spread", [1.0, 3.0])
def test_sums_of_few_rows_lose_no_more_than_the_results_rounding(dtype, b, h, hk, lq, lk, d, spread):
    gen = torch.Generator(device="cuda").manual_seed(lk + lq)
    rand = lambda n, heads: torch.randn(b, n, heads, d, device=DEV, generator=gen)  # noqa: E731
    q, k, v, dout = (t.to(dtype) for t in (spread * rand(lq, h), rand(lk, hk), rand(lk, hk), rand(lq, h)))
    out, lse = api.gs_cross_attention_fwd(q, k, v)
    dv = api.gs_cross_attention_bwd(dout, q, k, v, out, lse)[2].double()
    Q, K, G = (t.double().transpose(1, 2) for t in (q, k, dout))
    p = torch.softmax(Q @ K.repeat_interleave(h // hk, 1).transpose(2, 3) * d ** -0.5, 3)
    want = (p.transpose(2, 3) @ G).reshape(b, hk, h // hk, lk, d).sum(2).transpose(1, 2)
    least, off = want.to(dtype).double() - want, dv - want
    assert off.norm() <= 1.1 * least.norm()
    per = off.norm(dim=(1, 3)) / least.norm(dim=(1, 3))
    assert per.max() <= 1.5, per.max().item()
    assert api.gs_device_error() == _abi.GS_OK
