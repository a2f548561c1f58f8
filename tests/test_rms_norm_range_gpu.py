"""The root-mean-square norm at the ends of its squares' float32 range, as the header states them."""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("cols", [64, 1000, 4096, 10000])
def test_sums_of_squares_at_the_ends(cols):
    most = (2.0 ** 128 / cols) ** 0.5  # of equal elements whose squares' sum is 2^128
    x = torch.ones(6, cols, device=DEV)
    x[0] *= 0.99 * most
    x[1] *= 1.01 * most
    x[2] *= 2.0 ** -62
    x[3] *= 2.0 ** -80
    x[4] = 0
    y, _, rstd = api.gs_rms_norm_fwd(x, eps=0.0)
    assert ((y[0] - 1).abs() <= 2.0 ** -18).all() and ((y[2] - 1).abs() <= 2.0 ** -18).all()
    assert rstd[1] == 0 and (y[1] == 0).all()
    assert rstd[3].isinf() and y[3].isinf().all()  # squares of 2^-160
    assert rstd[4].isinf() and y[4].isnan().all()
    y, _, _ = api.gs_rms_norm_fwd(x[4:], eps=1e-6)
    assert (y[0] == 0).all()
