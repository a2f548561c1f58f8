"""The decoder operators' workspaces: what is refused, and one that is kept over calls of different sizes (same bits)."""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _rand(shape, dtype, seed):
    return torch.randn(shape, device=DEV, generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)


def _unsuitable(size):
    """Tensors of at least `size` elements that are not one piece of the device's memory."""
    yield torch.empty(size, dtype=torch.uint8)
    yield torch.empty(size, dtype=torch.uint8).pin_memory()
    yield torch.empty(1, dtype=torch.uint8, device=DEV).expand(size)
    yield torch.empty(2 * size, dtype=torch.uint8, device=DEV)[::2]
    yield torch.empty(1, dtype=torch.uint8)


def test_unsuitable_workspaces_are_refused():
    q, k = _rand((2, 40, 4, 64), torch.float32, 1), _rand((2, 90, 2, 64), torch.float32, 2)
    out, lse = api.gs_cross_attention_fwd(q, k, k)
    x, w = _rand((50, 64), torch.float32, 3), _rand((64,), torch.float32, 4)
    _, mean, rstd = api.gs_layer_norm_fwd(x, w)
    for ws in _unsuitable(1 << 22):
        for call in (lambda: api.gs_cross_attention_fwd(q, k, k, workspace=ws),
                     lambda: api.gs_cross_attention_bwd(q, q, k, k, out, lse, workspace=ws),
                     lambda: api.gs_layer_norm_bwd(x, x, mean, rstd, w, workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
    off = torch.empty((1 << 22) + 1, dtype=torch.uint8, device=DEV)[1:]
    for call in (lambda: api.gs_cross_attention_fwd(q, k, k, workspace=off),
                 lambda: api.gs_cross_attention_bwd(q, q, k, k, out, lse, workspace=off),
                 lambda: api.gs_layer_norm_bwd(x, x, mean, rstd, w, workspace=off)):
        with pytest.raises(_abi.GsError, match="aligned"):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_one_workspace_kept_over_calls_of_different_sizes(dtype):
    kept = torch.full((96 << 20,), 255, dtype=torch.uint8, device=DEV)  # every value in it is NaN
    small = torch.full((64,), 255, dtype=torch.uint8, device=DEV)
    for n, (lq, lk, h, hk, d, mask) in enumerate([
            (300, 700, 4, 2, 64, True), (1, 3000, 4, 4, 64, False), (1, 900, 4, 4, 40, True), (20, 90, 2, 2, 128, False),
            (260, 2000, 2, 1, 64, False), (70, 65, 2, 2, 200, True), (5, 4000, 8, 2, 33, True)]):
        q, k, v, dout = (_rand(s, dtype, 9 * n + i) for i, s in enumerate([(2, lq, h, d), (2, lk, hk, d), (2, lk, hk, d), (2, lq, h, d)]))
        m = _rand((2, lk), torch.float32, n) < 0.3 if mask else None
        want = api.gs_cross_attention_fwd(q, k, v, key_mask=m)
        grads = api.gs_cross_attention_bwd(dout, q, k, v, *want, key_mask=m)
        assert api.gs_cross_attention_workspace_bytes(q, k, v, key_mask=m, backward=True) <= kept.numel()
        for ws in (kept, small):
            got = api.gs_cross_attention_fwd(q, k, v, key_mask=m, workspace=ws)
            back = api.gs_cross_attention_bwd(dout, q, k, v, *got, key_mask=m, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(got + back, want + grads)), (n, ws.numel())
    for n, (rows, cols) in enumerate([(3000, 256), (7, 333), (2000, 1024), (5, 9000)]):
        x, dy, w = _rand((rows, cols), dtype, n), _rand((rows, cols), dtype, n + 20), _rand((cols,), dtype, n + 40)
        _, mean, rstd = api.gs_layer_norm_fwd(x, w)
        want = api.gs_layer_norm_bwd(dy, x, mean, rstd, w)
        for ws in (kept, small):
            assert all(torch.equal(a, b) for a, b in zip(api.gs_layer_norm_bwd(dy, x, mean, rstd, w, workspace=ws), want))
    assert (small == 255).all()
    assert api.gs_device_error() == _abi.GS_OK
