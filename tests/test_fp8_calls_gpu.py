"""The 8-bit decoder operators' calls: arguments that end in an exception, kept workspaces, several calls at once, tiles that
stand out of the result on every side."""
import subprocess
import sys

import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

WITHOUT_MEMORY = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from differentiable_gaussian_splatting_gs_gb300 import _abi, api
x = torch.randn(4, 128, device="cuda")
q, s = api.gs_quantize_fp8(x)
y, h, rstd = api.gs_rms_norm_fwd(x)
with FakeTensorMode():
    fx, fr = torch.empty(4, 128, device="cuda"), torch.empty(4, device="cuda")
    fq, fs = torch.empty(4, 128, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(4, 1, device="cuda")
raised = 0
for call in (lambda: api.gs_rms_norm_fwd(fx), lambda: api.gs_rms_norm_fp8(x, None, fx), lambda: api.gs_rms_norm_bwd(x, fx, rstd),
             lambda: api.gs_rms_norm_bwd(x, x, fr), lambda: api.gs_quantize_fp8(fx), lambda: api.gs_quantize_fp8(x, out=(fq, s)),
             lambda: api.gs_matmul_fp8(fq, s, q, s), lambda: api.gs_matmul_fp8(q, s, q, fs), lambda: api.gs_matmul_fp8(q, s, q, s, out=fx[:, :4]),
             lambda: api.gs_clip_grads([x, fx], 1.0), lambda: api.gs_clip_grads([x], 1.0, out=[fx]), lambda: api.gs_grad_norm([fx])):
    try:
        call()
    except (RuntimeError, ValueError, TypeError):
        raised += 1
assert raised == 12, raised
assert torch.equal(api.gs_rms_norm_fwd(x)[0], y) and torch.equal(api.gs_quantize_fp8(x)[0].float(), q.float())
assert api.gs_device_error() == _abi.GS_OK
print("usable")
"""


def test_tensors_without_memory_raise():
    # in a process of its own: an exception that leaves the interpreter without its lock ends it
    r = subprocess.run([sys.executable, "-c", WITHOUT_MEMORY], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("usable"), (r.returncode, r.stderr[-2000:])


def test_unsuitable_workspaces_are_refused():
    x, w = torch.randn(50, 64, device=DEV), torch.randn(64, device=DEV)
    _, h, rstd = api.gs_rms_norm_fwd(x, w)
    n = 1 << 20
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device=DEV).expand(n),
               torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]):
        for call in (lambda: api.gs_rms_norm_bwd(x, h, rstd, w, workspace=ws), lambda: api.gs_clip_grads([x], 1.0, workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
    off = torch.empty(n + 1, dtype=torch.uint8, device=DEV)[1:]
    for call in (lambda: api.gs_rms_norm_bwd(x, h, rstd, w, workspace=off), lambda: api.gs_clip_grads([x], 1.0, workspace=off)):
        with pytest.raises(_abi.GsError, match="aligned"):
            call()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_workspace_kept_over_calls_of_different_sizes(dtype):
    kept = torch.full((32 << 20,), 255, dtype=torch.uint8, device=DEV)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for rows, cols in ((3000, 256), (7, 333), (2000, 1024), (5, 9000), (1, 40)):
        x, dy, w = (torch.randn(s, device=DEV, generator=gen).to(dtype) for s in ((rows, cols), (rows, cols), (cols,)))
        rstd = api.gs_rms_norm_fwd(x, w)[2]
        want = api.gs_rms_norm_bwd(dy, x, rstd, w, dy)
        assert all(torch.equal(a, b) for a, b in zip(api.gs_rms_norm_bwd(dy, x, rstd, w, dy, workspace=kept), want))
        grads = [x, dy, w]
        assert torch.equal(api.gs_grad_norm(grads, workspace=kept), api.gs_grad_norm(grads))


def test_gradients_from_a_generator_and_on_a_stream():
    g = [torch.randn(n, device=DEV) for n in (10, 1000, 70000)]
    want = api.gs_grad_norm(g)
    assert torch.equal(api.gs_grad_norm(t for t in g), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.gs_grad_norm((t for t in g), stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    for stream in (None, side):
        with pytest.raises(ValueError):
            api.gs_clip_grads([], 1.0, stream=stream)


def _values(q, s):
    block = 1 if s.shape[0] == q.shape[0] else 128
    return q.double() * s.double().repeat_interleave(block, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k", [(100, 10000, 200), (128, 9730, 130), (130, 20000, 128), (257, 10240, 129), (70, 2500, 1000), (66, 128, 4096),
                                   (64, 5000, 640), (40, 17, 3000), (2500, 1025, 900), (12800, 256, 1), (9729, 8, 300)])
def test_tiles_out_of_the_result(m, n, k, block, dtype):
    # tolerance: as in test_fp8_gpu.py, of the sum of the magnitudes of the products
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    qa, sa = api.gs_quantize_fp8(torch.randn(m, k, device=DEV, generator=gen))
    qb, sb = api.gs_quantize_fp8(torch.randn(n, k, device=DEV, generator=gen), block)
    a, b = _values(qa, sa), _values(qb, sb)
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    for pad in (0, 8, 3):  # rows beside which nothing may be written, on 16 bytes or not
        room = torch.full((m + 1, n + pad), 5.0, device=DEV, dtype=dtype)
        got = api.gs_matmul_fp8(qa, sa, qb, sb, out=room[:m, :n])
        u = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
        assert ((got.double() - want).abs() <= size * (2.0 ** -15 + (2 + sa.shape[1]) * 2.0 ** -24) + u * want.abs()).all()
        assert (room[m:] == 5).all() and (room[:, n:] == 5).all()
    assert api.gs_device_error() == _abi.GS_OK


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,n,k", [(3, 40, 1), (70, 300, 129), (5, 1000, 1001), (4000, 2000, 519), (300, 200, 15), (200, 5000, 130)])
def test_what_lies_behind_the_rows_takes_no_part(m, n, k, block):
    wide = (k + 15) // 16 * 16 + 16
    rooms = [torch.full((r, wide), 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for r in (m, n)]  # NaN
    a, b = torch.randn(m, k, device=DEV), torch.randn(n, k, device=DEV)
    qa, sa = api.gs_quantize_fp8(a)
    qb, sb = api.gs_quantize_fp8(b, block)
    pa, _ = api.gs_quantize_fp8(a, out=(rooms[0][:, :k], sa))
    pb, _ = api.gs_quantize_fp8(b, block, out=(rooms[1][:, :k], sb))
    want = _values(qa, sa) @ _values(qb, sb).t()
    got = api.gs_matmul_fp8(pa, sa, pb, sb, dtype=torch.float32)
    assert ((got.double() - want).abs() <= 2.0 ** -15 * (_values(qa, sa).abs() @ _values(qb, sb).abs().t()) + 2.0 ** -24 * want.abs()).all()
    assert (rooms[0].view(torch.uint8)[:, k:] == 0x7F).all() and (rooms[1].view(torch.uint8)[:, k:] == 0x7F).all()


def test_many_products_of_all_forms_at_once():
    gen = torch.Generator(device="cuda").manual_seed(5)
    forms = []
    for m, n, k, block in ((3000, 2048, 512, 128), (2500, 1280, 700, 1), (1, 4096, 1024, 128), (40, 1000, 2000, 128), (200, 512, 2048, 1), (1000, 600, 300, 128)):
        a = api.gs_quantize_fp8(torch.randn(m, k, device=DEV, generator=gen))
        b = api.gs_quantize_fp8(torch.randn(n, k, device=DEV, generator=gen), block)
        forms.append((a + b, api.gs_matmul_fp8(*a, *b, dtype=torch.float32)))
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for i in range(120):
        args, want = forms[i % len(forms)]
        got.append((api.gs_matmul_fp8(*args, dtype=torch.float32, stream=streams[i % 4]), want))
    q = torch.randn(2, 700, 8, 64, device=DEV, dtype=torch.bfloat16)  # with other kernels that use tensor memory
    for i in range(20):
        with torch.cuda.stream(streams[i % 4]):
            api.gs_cross_attention_fwd(q, q, q)
        args, want = forms[i % len(forms)]
        got.append((api.gs_matmul_fp8(*args, dtype=torch.float32, stream=streams[i % 4]), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got) and api.gs_device_error() == _abi.GS_OK


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_and_columns_that_repeat(dtype, block):
    room = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    for x in (torch.randn(1, 300, device=DEV), torch.randn(70, 1, device=DEV)):
        one = room[:x.numel() * dtype.itemsize].view(dtype).view(x.shape)
        one.copy_(x)
        many = one.expand(700, 300) if x.shape[0] == 1 else one.expand(70, 500)
        out = api.gs_quantize_fp8(many.contiguous(), block)
        # right behind the only row or column
        at = (one.numel() * dtype.itemsize + 15) // 16 * 16
        wide = (many.shape[1] + 15) // 16 * 16
        q = room[at:at + many.shape[0] * wide].view(torch.float8_e4m3fn).view(-1, wide)[:, :many.shape[1]]
        got = api.gs_quantize_fp8(many, block, out=(q, torch.empty_like(out[1])))
        assert torch.equal(got[0].view(torch.uint8), out[0].view(torch.uint8)) and torch.equal(got[1], out[1])
