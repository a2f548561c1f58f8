"""GPU cross attention against the float64 one.

Tolerances. u is the element type's unit roundoff. A score is off by at most 2^-20 of scale sum |q||k| (float32
accumulation of up to 256 products) and so is lse; a probability by that, by 2^-20 for the exponential and the
sum, and by u where it is rounded to feed a matrix product (twice at most: once more through the running
maximum). out is then off by its probabilities' errors against sum P |v|, and rounded once. The gradients' bounds are the
same terms carried through dS = scale P (dP - delta), with dP accumulated to 2^-20 of sum |dout||v| and delta
formed from the rounded out (oracle.decoder.attention_bwd).
"""
import numpy as np
import pytest
import torch

from oracle import decoder

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
ACC = 2.0 ** -20


def _np(t):
    return t.double().cpu().numpy()


def _rand(shape, dtype, seed, factor=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, device=DEV, generator=g) * factor).to(dtype)


def _valid(b, lk, k_len, key_mask):
    v = np.ones((b, lk), bool)
    if k_len is not None:
        v &= np.arange(lk)[None] < k_len.cpu().numpy()[:, None]
    if key_mask is not None:
        v &= key_mask.bool().cpu().numpy()
    return v


def _check(q, k, v, k_len=None, key_mask=None, scale=None, dout=None, backward=True, seed=0):
    u, tiny = U[q.dtype], TINY[q.dtype]
    b, lq, h, d = q.shape
    sc = d ** -0.5 if scale is None else scale
    valid = _valid(b, k.shape[1], k_len, key_mask)
    out, lse = api.gs_cross_attention_fwd(q, k, v, k_len=k_len, key_mask=key_mask, scale=scale)
    r = decoder.attention_fwd(_np(q), _np(k), _np(v), valid, sc)
    size = r["size"].transpose(0, 2, 1)[..., None]
    tol = (2 * u + ACC + 2 * ACC * size) * r["mag"] + u * np.abs(r["out"]) + tiny
    got = _np(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - r["out"]) <= tol).all(), np.max(np.abs(got - r["out"]) / (tol + 1e-300))
    empty = ~np.isfinite(r["lse"])
    assert (_np(lse)[empty] == -np.inf).all()
    fin = ~empty
    assert (np.abs(_np(lse)[fin] - r["lse"][fin]) <= ACC * (1 + r["size"][fin] + np.abs(r["lse"][fin]))).all()
    if backward:
        dout = _rand(q.shape, q.dtype, seed + 77) if dout is None else dout
        grads = api.gs_cross_attention_bwd(dout, q, k, v, out, lse, k_len=k_len, key_mask=key_mask, scale=scale)
        w = decoder.attention_bwd(_np(dout), _np(q), _np(k), _np(v), valid, sc, rounding=u, accumulate=ACC)
        for name, g in zip(("dq", "dk", "dv"), grads):
            tol = w[name + "_tol"] + tiny
            assert torch.isfinite(g).all(), name
            bad = np.abs(_np(g) - w[name]) / (tol + 1e-300)
            assert (bad <= 1).all(), (name, bad.max())
        keys = np.broadcast_to(valid[:, :, None, None], grads[1].shape)
        assert (_np(grads[1])[~keys] == 0).all() and (_np(grads[2])[~keys] == 0).all()
    assert api.gs_device_error() == _abi.GS_OK
    return out, lse


def _qkv(b, lq, lk, h, hk, d, dtype, seed=0):
    return _rand((b, lq, h, d), dtype, seed, 1.5), _rand((b, lk, hk, d), dtype, seed + 1), _rand((b, lk, hk, d), dtype, seed + 2)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("b,lq,lk,h,hk,d", [
    (1, 1, 1, 1, 1, 1), (1, 1, 300, 2, 2, 64), (2, 3, 5, 2, 1, 8), (1, 128, 128, 1, 1, 64), (1, 129, 127, 2, 2, 64),
    (2, 200, 333, 4, 2, 64), (1, 300, 65, 3, 3, 40), (1, 257, 400, 6, 1, 128), (1, 64, 64, 2, 2, 32), (1, 70, 90, 2, 2, 80),
    (1, 45, 70, 2, 1, 33), (1, 50, 130, 2, 2, 136), (1, 33, 65, 1, 1, 256), (1, 17, 100, 2, 2, 255), (1, 2, 2000, 4, 2, 64),
    (1, 500, 1, 2, 2, 64), (1, 9, 5000, 2, 1, 128), (3, 1, 700, 8, 2, 96), (1, 1000, 33, 2, 2, 16), (1, 700, 700, 2, 2, 128)])
def test_sizes(dtype, b, lq, lk, h, hk, d):
    _check(*_qkv(b, lq, lk, h, hk, d, dtype), seed=lq)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("lq", [1, 6, 150])
@pytest.mark.parametrize("d", [64, 128, 48, 200])
@pytest.mark.parametrize("kind", ["len", "keys", "both"])
def test_masks_with_empty_rows_and_non_finite_masked_keys(dtype, lq, d, kind):
    b, lk = 5, 270
    q, k, v = _qkv(b, lq, lk, 4, 2, d, dtype, 3)
    k_len = torch.tensor([270, 0, 1, 128, 129], dtype=torch.int32, device=DEV) if kind != "keys" else None
    key_mask = None
    if kind != "len":
        g = torch.Generator(device="cuda").manual_seed(5)
        key_mask = torch.rand(b, lk, device=DEV, generator=g) < 0.5
        key_mask[3] = False
        key_mask[4, :200] = False
    bad = torch.from_numpy(~_valid(b, lk, k_len, key_mask)).to(DEV)
    k[bad] = float("nan")
    v[bad] = float("inf")
    v[:, ::2][bad[:, ::2]] = float("nan")
    _check(q, k, v, k_len=k_len, key_mask=key_mask, seed=d)


def test_lengths_outside_the_range_are_clamped():
    q, k, v = _qkv(3, 20, 50, 2, 2, 64, torch.bfloat16)
    far = torch.tensor([-7, 51, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    near = torch.tensor([0, 50, 50], dtype=torch.int32, device=DEV)
    a, b = (api.gs_cross_attention_fwd(q, k, v, k_len=n) for n in (far, near))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", list(U))
def test_large_scores_and_values_of_the_types_range(dtype):
    # scores of several hundred: one key takes all the weight; later keys raise the maximum again and again
    q, k, v = _qkv(1, 140, 500, 2, 2, 64, dtype)
    k = (k * torch.linspace(0.1, 12, 500, device=DEV)[None, :, None, None]).to(dtype)
    _check(q, k, v, seed=1)
    low = torch.full_like(k, -30.0)  # all scores equal and far below zero
    _check(torch.ones_like(q), low, v, seed=2)
    _check(q, k, v, scale=1e-3, seed=3)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("lq,lk,d", [(150, 260, 64), (1, 260, 64), (150, 260, 40)])
def test_strides_orders_and_misalignment(dtype, lq, lk, d):
    b, h = 2, 4
    q, k, v = _qkv(b, lq, lk, h, h, d, dtype, 9)
    want, wl = api.gs_cross_attention_fwd(q, k, v)
    dout = _rand(q.shape, dtype, 10)
    grads = api.gs_cross_attention_bwd(dout, q, k, v, want, wl)

    def head_first(t):  # [b, h, l, d] in memory
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    def packed(t, pad, at):  # rows inside a wider buffer, off by `at` elements
        big = torch.full((t.shape[0], t.shape[1], t.shape[2] * d + pad), 7.0, dtype=dtype, device=DEV)
        view = big[:, :, at:at + t.shape[2] * d].unflatten(2, (t.shape[2], d))
        view.copy_(t)
        return view

    def flipped(t):  # batch entries in reverse, one buffer
        return t.flip(0).contiguous().as_strided(t.shape, t.stride(), 0) if t.shape[0] == 1 else t

    for change in (head_first, lambda t: packed(t, 8, 0), lambda t: packed(t, 5, 3), lambda t: packed(t, 8, 1), flipped):
        got, gl = api.gs_cross_attention_fwd(change(q), change(k), change(v),
                                             out=(change(torch.zeros_like(q)), torch.empty_like(wl)))
        assert torch.equal(got, want) and torch.equal(gl, wl)
        into = tuple(change(torch.zeros_like(t)) for t in (q, k, v))
        gg = api.gs_cross_attention_bwd(change(dout), change(q), change(k), change(v), change(want), wl, grads=into)
        assert all(torch.equal(x, y) for x, y in zip(gg, grads))
    # one batch entry, head or token broadcast to all (stride 0)
    kb = k[:1].expand(b, -1, -1, -1)
    _check(q, kb, v[:, :, :1].expand(-1, -1, h, -1), backward=False)


def test_one_buffer_for_q_k_and_v_of_a_projection():
    qkv = _rand((2, 200, 3 * 4, 64), torch.bfloat16, 1)
    q, k, v = qkv[:, :, :4], qkv[:, :, 4:8], qkv[:, :, 8:]
    _check(q, k, v)


def test_writes_stay_inside_the_outputs():
    b, lq, lk, h, d = 1, 130, 140, 2, 72
    q, k, v = _qkv(b, lq, lk, h, h, d, torch.float16)
    ob = torch.full((b, lq + 20, h, d + 16), 5.0, dtype=torch.float16, device=DEV)
    out, lse = api.gs_cross_attention_fwd(q, k, v, out=(ob[:, 10:10 + lq, :, 8:8 + d], torch.empty(b, h, lq, device=DEV)))
    assert torch.equal(out, api.gs_cross_attention_fwd(q, k, v)[0])
    kb = torch.full((b, lk + 20, h, d + 16), 5.0, dtype=torch.float16, device=DEV)
    vb, qb = kb.clone(), ob.clone()
    inner = lambda t, n: t[:, 10:10 + n, :, 8:8 + d]  # noqa: E731
    api.gs_cross_attention_bwd(_rand(q.shape, q.dtype, 3), q, k, v, out, lse, grads=(inner(qb, lq), inner(kb, lk), inner(vb, lk)))
    for big, n in ((ob, lq), (kb, lk), (vb, lk)):
        inner(big, n).fill_(5.0)
        assert (big == 5.0).all()


@pytest.mark.parametrize("dtype", list(U))
def test_empty_lengths(dtype):
    q, k, v = _qkv(2, 5, 0, 2, 2, 64, dtype)
    out, lse = api.gs_cross_attention_fwd(q, k, v)
    assert (out == 0).all() and (lse == -float("inf")).all()
    dq, dk, dv = api.gs_cross_attention_bwd(q, q, k, v, out, lse)
    assert (dq == 0).all() and dk.shape == k.shape
    q, k, v = _qkv(2, 0, 5, 2, 2, 64, dtype)
    out, lse = api.gs_cross_attention_fwd(q, k, v)
    dq, dk, dv = api.gs_cross_attention_bwd(q, q, k, v, out, lse, grads=(q, torch.ones_like(k), torch.ones_like(v)))
    assert out.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    e = torch.empty(0, 4, 2, 64, dtype=dtype, device=DEV)
    assert api.gs_cross_attention_fwd(e, e, e)[0].shape == e.shape


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("lq,mask", [(3, False), (260, False), (260, True)])
def test_same_bits_twice_another_stream_and_graph(dtype, lq, mask):
    q, k, v = _qkv(2, lq, 1500, 4, 2, 64, dtype)
    m = torch.rand(2, 1500, device=DEV, generator=torch.Generator(device="cuda").manual_seed(1)) < 0.7 if mask else None
    dout = _rand(q.shape, dtype, 4)

    def both(stream=None):
        o = api.gs_cross_attention_fwd(q, k, v, key_mask=m, stream=stream)
        return o + api.gs_cross_attention_bwd(dout, q, k, v, *o, key_mask=m, stream=stream)

    a = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = both(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c = both()
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("h,hk", [(4, 4), (6, 2)])
def test_gradients_against_differences(h, hk):
    q, k, v = _qkv(1, 9, 14, h, hk, 32, torch.float32)
    dout = _rand(q.shape, torch.float32, 5)
    valid = np.ones((1, 14), bool)
    valid[0, 10:] = False
    n = torch.tensor([10], dtype=torch.int32, device=DEV)
    out, lse = api.gs_cross_attention_fwd(q, k, v, k_len=n)
    grads = api.gs_cross_attention_bwd(dout, q, k, v, out, lse, k_len=n)
    g = np.random.default_rng(1)
    args = [_np(t) for t in (q, k, v)]
    for at, got in enumerate(grads):
        u = g.standard_normal(args[at].shape)

        def loss(t):
            a = list(args)
            a[at] = a[at] + t * u
            return (decoder.attention_fwd(*a, valid, 32 ** -0.5)["out"] * _np(dout)).sum()

        want, terms = (loss(1e-5) - loss(-1e-5)) / 2e-5, np.abs(_np(got) * u).sum()
        assert abs((_np(got) * u).sum() - want) <= 1e-5 * terms


def test_refusals():
    q, k, v = _qkv(2, 5, 7, 4, 2, 64, torch.float16)
    fwd = api.gs_cross_attention_fwd
    i = torch.ones(2, dtype=torch.int32, device=DEV)
    for bad in (lambda: fwd(q.double(), k, v), lambda: fwd(q, k.float(), v), lambda: fwd(q, k, v[:, :6]),
                lambda: fwd(q[0], k, v), lambda: fwd(q[:, :, :3], k, v), lambda: fwd(q, k, v, k_len=i.long()),
                lambda: fwd(q, k, v, k_len=i[:1]), lambda: fwd(q, k, v, key_mask=i), lambda: fwd(q, k, v, scale=0.0),
                lambda: fwd(q, k, v, scale=-1.0), lambda: fwd(q, k.transpose(2, 3), v),
                lambda: fwd(q.transpose(1, 3), k, v), lambda: fwd(q, k, v, key_mask=torch.ones(2, 7, device=DEV)),
                lambda: fwd(q, k, v, out=(q[:, :4], torch.empty(2, 4, 5, device=DEV))),
                lambda: fwd(q, k, v, out=(q.clone(), torch.empty(2, 5, 4, device=DEV)))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_abi.GsError, match="head_dim"):
        t = torch.zeros(1, 2, 2, 300, device=DEV)
        fwd(t, t, t)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lq", [1, 200])
def test_scores_of_minus_infinity_before_very_low_ones(dtype, lq):
    # the first keys' scores are -inf, the others' around -500: these alone make the result
    q, k, v = _qkv(1, lq, 400, 2, 2, 64, dtype, 7)
    q, k = q.abs() + 0.25, torch.zeros_like(k)
    k[:, :150, :, 3] = -float("inf")
    k[:, 150:, :, 5] = torch.linspace(-4000, -4100, 250, device=DEV).to(dtype)[None, :, None]
    out, lse = api.gs_cross_attention_fwd(q, k, v)
    r = decoder.attention_fwd(_np(q), _np(k[:, 150:]), _np(v[:, 150:]), np.ones((1, 250), bool), 0.125)
    size = r["size"].transpose(0, 2, 1)[..., None]
    tol = (2 * U[dtype] + ACC + 2 * ACC * size) * r["mag"] + U[dtype] * np.abs(r["out"]) + TINY[dtype]
    assert (np.abs(_np(out) - r["out"]) <= tol).all()
    assert (np.abs(_np(lse) - r["lse"]) <= ACC * (1 + r["size"] + np.abs(r["lse"]))).all()


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float16, 128), (torch.float32, 64)])
def test_waits_that_give_up_are_reported_and_leave_the_context_usable(dtype, d):
    import ctypes as C

    q, k, v = _qkv(1, 400, 2000, 2, 2, d, dtype)
    dout = _rand(q.shape, dtype, 5)
    want = api.gs_cross_attention_fwd(q, k, v)
    grads = api.gs_cross_attention_bwd(dout, q, k, v, *want)
    (b, lq, h, _), (_, lk, hk, _) = q.shape, k.shape
    code = {torch.float32: _abi.GS_DTYPE_F32, torch.float16: _abi.GS_DTYPE_F16, torch.bfloat16: _abi.GS_DTYPE_BF16}[dtype]
    a = _abi.gs_attention(code, b, h, hk, d, lq, lk)
    a.spin_limit = 1  # every wait gives up at its first poll
    lib, stream = _abi.load(), torch.cuda.current_stream().cuda_stream
    out, lse = torch.empty_like(q), torch.empty_like(want[1])
    spare = [torch.empty_like(t) for t in (q, k, v)]

    def heads(*ts):
        return [C.byref(_abi.gs_heads(t.data_ptr(), *t.stride()[:3])) for t in ts]

    for backward in (0, 1):
        need = lib.gs_cross_attention_workspace_bytes(C.byref(a), backward)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
        if backward:
            st = lib.gs_cross_attention_bwd(C.byref(a), *heads(dout, q, k, v, want[0]), want[1].data_ptr(), *heads(*spare),
                                            ws.data_ptr(), need, stream)
        else:
            st = lib.gs_cross_attention_fwd(C.byref(a), *heads(q, k, v, out), lse.data_ptr(), ws.data_ptr(), need, stream)
        assert st == _abi.GS_OK  # enqueued
        assert api.gs_device_error() == _abi.GS_ERR_TIMEOUT
        assert api.gs_device_error() == _abi.GS_OK
    again = api.gs_cross_attention_fwd(q, k, v)
    assert all(torch.equal(x, y) for x, y in zip(again, want))
    assert all(torch.equal(x, y) for x, y in zip(api.gs_cross_attention_bwd(dout, q, k, v, *again), grads))
    assert api.gs_device_error() == _abi.GS_OK


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("b,lq,lk,h,hk,d,masked", [
    (1, 1, 3000, 8, 2, 64, False), (2, 1, 1500, 12, 4, 128, True), (1, 7, 900, 10, 2, 64, False), (1, 33, 700, 16, 1, 40, True),
    (2, 5, 600, 32, 2, 128, False), (1, 26, 400, 5, 1, 64, False), (1, 1, 500, 136, 1, 64, False), (1, 2, 640, 100, 1, 64, True),
    (1, 90, 300, 6, 2, 128, False), (3, 1, 9000, 4, 1, 80, True)])
def test_shared_heads_of_few_queries(dtype, b, lq, lk, h, hk, d, masked):
    q, k, v = _qkv(b, lq, lk, h, hk, d, dtype, lq)
    q = torch.randn(b, h, lq, d, device=DEV, generator=torch.Generator(device="cuda").manual_seed(lk)).to(dtype).transpose(1, 2)
    k_len = torch.tensor([lk, 0, lk // 2][:b], dtype=torch.int32, device=DEV) if masked else None
    _check(q, k, v, k_len=k_len, seed=lk)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,lq,lk,h,hk,d,masked", [
    (1, 300, 700, 2, 2, 256, False), (2, 129, 1000, 4, 2, 192, True), (1, 1, 3000, 8, 2, 256, False), (1, 3, 900, 3, 3, 160, True),
    (1, 2000, 130, 1, 1, 144, False), (1, 260, 64, 2, 1, 250, False)])
def test_wide_heads(dtype, b, lq, lk, h, hk, d, masked):
    q, k, v = _qkv(b, lq, lk, h, hk, d, dtype, lq)
    k_len = torch.tensor([lk - 70, 0][:b], dtype=torch.int32, device=DEV) if masked else None
    _check(q, k, v, k_len=k_len, seed=lk, backward=False)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lq,lk,h,hk,d", [(1, 3000, 8, 8, 40), (5, 390, 16, 16, 32), (2, 700, 8, 2, 128), (60, 100, 4, 4, 64)])
def test_few_queries_lose_no_more_than_the_results_rounding(dtype, lq, lk, h, hk, d):
    # dv = P^T dout: with P in two parts (relative 2 u^2) the result's own rounding is all that counts
    q, k, v = _qkv(1, lq, lk, h, hk, d, dtype, 11)
    q = q * 2
    dout = _rand(q.shape, dtype, 5)
    out, lse = api.gs_cross_attention_fwd(q, k, v)
    _, _, dv = api.gs_cross_attention_bwd(dout, q, k, v, out, lse)
    want = decoder.attention_bwd(_np(dout), _np(q), _np(k), _np(v), np.ones((1, lk), bool), d ** -0.5)["dv"]
    least = np.linalg.norm(_np(torch.from_numpy(want).to(dtype)) - want)
    assert np.linalg.norm(_np(dv) - want) <= 1.1 * least
