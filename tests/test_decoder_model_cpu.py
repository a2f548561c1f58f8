"""GaussianDecoder's checks of its tokens (CPU: before any kernel)."""
import pytest
import torch

from differentiable_gaussian_splatting_gs_gb300 import decoder


def _decoder(n=6):
    base = {"mean3d": torch.zeros(n, 3), "log_scale": torch.zeros(n, 3), "quat": torch.zeros(n, 4), "opacity_logit": torch.zeros(n),
            "sh": torch.zeros(n, 1, 3)}
    return decoder.GaussianDecoder(base, 24, channels=16, heads=2, head_dim=8)


@pytest.mark.parametrize("shape", [(2, 10, 24), (0, 10, 24), (10, 24), (1, 10, 25), (1, 1, 10, 24)])
def test_tokens_of_anything_but_one_scene_are_refused(shape):
    with pytest.raises(ValueError, match="one scene"):
        _decoder().forward(torch.zeros(shape))


def test_tokens_of_one_scene_reach_the_kernels():
    with pytest.raises(ValueError, match="CUDA"):  # which refuse host tensors
        _decoder().forward(torch.zeros(1, 10, 24))
