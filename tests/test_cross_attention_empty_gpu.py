"""GPU cross attention without queries or without keys: zeros and an lse of -inf in every element of the outputs, nothing
beside them, for every type, width and layout."""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _inside(shape, dtype, at):
    """A tensor inside a buffer of ones, its rows apart and off by `at` elements; and the buffer."""
    big = torch.ones(shape[0] + 1, shape[1] + 2, shape[2] + 1, shape[3] + 5, dtype=dtype, device=DEV)
    return big[1:, 1:1 + shape[1], :shape[2], at:at + shape[3]], big


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [1, 64, 100, 256])
@pytest.mark.parametrize("lq,lk", [(1, 0), (300, 0), (0, 300), (0, 0)])
@pytest.mark.parametrize("masked", [False, True])
def test_no_queries_or_no_keys(dtype, d, lq, lk, masked):
    b, h, hk = 3, 4, 2
    q, k = torch.randn(b, lq, h, d, device=DEV).to(dtype), torch.randn(b, lk, hk, d, device=DEV).to(dtype)
    args = {"key_mask": torch.ones(b, lk, dtype=torch.bool, device=DEV), "k_len": torch.full((b,), lk, dtype=torch.int32, device=DEV)} if masked else {}
    (out, ob), lse = _inside(q.shape, dtype, 3), torch.ones(b, h, lq, device=DEV)
    api.gs_cross_attention_fwd(q, k, k.clone(), out=(out, lse), **args)
    assert (out == 0).all() and (lse == -float("inf")).all()
    (dq, qb), (dk, kb), (dv, vb) = (_inside(s, dtype, a) for s, a in ((q.shape, 1), (k.shape, 2), (k.shape, 5)))
    api.gs_cross_attention_bwd(q.clone(), q, k, k.clone(), out, lse, grads=(dq, dk, dv), **args)
    for t, big in ((out, ob), (dq, qb), (dk, kb), (dv, vb)):
        assert (t == 0).all()
        t.fill_(1.0)
        assert (big == 1).all()
    assert api.gs_device_error() == _abi.GS_OK
