"""The gradient norm where its bound is met from the other side: tensors off 16 bytes, whose sums go as those of aligned ones
do, outputs off 16 bytes, and norms of more and larger gradients than float32 sums hold."""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_equal_elements_off_16_bytes(offset):
    # 64 equal squares v^2 to a thread, in four chains: the k-th partial sum's rounding is at most 2^-24 k v^2, a chain's 2^-24 x 17 / 2 of
    # its sum; two more additions join the chains. The root halves that, its own rounding and that of the pairs' sums add 1 unit.
    # (One chain of 64 may be off by 16 units, and is by 8.2 for this v.)
    v, n = 1.96956944465637207, 20_000_000
    g = torch.full((n + offset,), v, device=DEV)[offset:]
    want = (n * float(g[0]) ** 2) ** 0.5
    assert abs(api.gs_grad_norm([g]).item() / want - 1) <= ((17 / 2 + 2) / 2 + 1) * 2.0 ** -24
    assert abs(api.gs_clip_grads([g], 1e9).item() / want - 1) <= ((17 / 2 + 2) / 2 + 1) * 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("offset", [1, 3])
def test_chunks_off_16_bytes_end_anywhere(offset, dtype):
    gen = torch.Generator(device="cuda").manual_seed(offset)
    for n in (1, 255, 257, 767, 1025, 2047, 2049, 4096 + 300, 100_003):
        room = torch.randn(n + offset + 8, device=DEV, generator=gen).to(dtype)
        g, before = room[offset:offset + n], room.clone()
        want = g.double().square().sum().sqrt()
        norm = api.gs_clip_grads([g], 0.25)
        assert (norm.double() - want).abs() <= 11 * 2.0 ** -24 * want
        u = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]
        expected = before[offset:offset + n].double() * min(1.0, 0.25 / (float(want) + 1e-6))
        assert ((g.double() - expected).abs() <= expected.abs() * (u + 2.0 ** -20) + 2.0 ** -25).all()
        assert torch.equal(room[:offset], before[:offset]) and torch.equal(room[offset + n:], before[offset + n:])
    assert api.gs_device_error() == _abi.GS_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_the_norm_goes_by_the_gradients_whatever_the_outputs_alignment(offset, dtype):
    gen = torch.Generator(device="cuda").manual_seed(9)
    for n in (5, 2050, 300_001):
        g = torch.randn(n + offset, device=DEV, generator=gen).to(dtype)[offset:]
        want = api.gs_grad_norm([g])
        for to in (0, 1, 2, 3, offset):
            room = torch.full((n + to + 9,), 7.0, device=DEV, dtype=dtype)
            out = room[to:to + n]
            assert torch.equal(api.gs_clip_grads([g], 0.5, out=[out]), want)
            factor = torch.tensor(0.5, device=DEV) / (want + 1e-6)
            assert torch.equal(out, g if factor >= 1 else (g.float() * factor).to(dtype))
            assert (room[:to] == 7).all() and (room[to + n:] == 7).all()


def test_more_large_gradients_than_a_float32_sum_holds():
    # 4e10 squares of 1.1e28: every thread's 64 fit float32, their sum does not (one tensor many times: nothing is written)
    v, n, times = 1.5 * 2.0 ** 46, 100_000_000, 400
    g = torch.full((n,), v, device=DEV, dtype=torch.bfloat16)
    want = (n * times) ** 0.5 * v
    assert abs(api.gs_grad_norm([g] * times).item() / want - 1) <= 2.0 ** -23
