"""Refusals of the layer norm and cross attention entry points: host checks before any device work (CPU)."""
import ctypes as C

import pytest
import torch

import __graft_entry__
from differentiable_gaussian_splatting_gs_gb300 import _abi, api

ARG = _abi.GS_ERR_ARG


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _abi.load()


def test_layer_norm_refusals(lib):
    def fwd(x=256, xs=64, rows=4, cols=64, dt=0, w=256, b=256, wdt=0, eps=1e-5, y=256, ys=64, mean=256, rstd=256):
        return lib.gs_layer_norm_fwd(x, xs, rows, cols, dt, w, b, wdt, eps, y, ys, mean, rstd, None)

    assert fwd(rows=0) == _abi.GS_OK  # nothing to do
    for bad in (dict(x=None), dict(x=258), dict(xs=63), dict(rows=-1), dict(cols=0), dict(cols=1 << 30), dict(dt=3),
                dict(dt=-1), dict(wdt=1), dict(dt=1, wdt=2), dict(w=257), dict(b=258), dict(eps=-1.0),
                dict(eps=float("nan")), dict(y=None), dict(ys=10), dict(mean=None), dict(rstd=None), dict(rstd=2)):
        assert fwd(**bad) == ARG, bad
        assert lib.gs_last_error_message()

    def bwd(dy=256, x=256, rows=4, cols=64, dt=0, mean=256, w=256, wdt=0, dx=256, dw=256, db=256, ws=256, n=1 << 20):
        return lib.gs_layer_norm_bwd(dy, cols, x, cols, rows, cols, dt, mean, 256, w, wdt, dx, cols, dw, db, ws, n, None)

    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(dx=None), dict(ws=None), dict(ws=264), dict(n=16),
                dict(dw=257), dict(db=257), dict(wdt=2)):
        assert bwd(**bad) == ARG, bad
    assert lib.gs_layer_norm_workspace_bytes(4, 64) == 4 * 2 * 64 * 4
    assert lib.gs_layer_norm_workspace_bytes(-1, 64) == 0


def test_attention_refusals(lib):
    def fwd(q=256, k=256, v=256, out=256, lse=256, **kw):
        a = _abi.gs_attention(**{**dict(dtype=2, batch=1, heads=4, kv_heads=2, head_dim=64, len_q=8, len_k=8), **kw})
        hs = [_abi.gs_heads(data=p, batch_stride=1, len_stride=1, head_stride=1) for p in (q, k, v, out)]
        return lib.gs_cross_attention_fwd(C.byref(a), *(C.byref(h) for h in hs), lse, None, 0, None)

    assert fwd(batch=0) == _abi.GS_OK and fwd(len_q=0) == _abi.GS_OK
    for bad in (dict(dtype=5), dict(batch=-1), dict(heads=3), dict(heads=0), dict(kv_heads=0), dict(head_dim=0),
                dict(head_dim=257), dict(len_q=-1), dict(len_k=-1), dict(scale=-1.0), dict(scale=float("inf")),
                dict(q=None), dict(k=None), dict(v=257), dict(out=None), dict(lse=None), dict(lse=258), dict(k_len=2),
                dict(batch=1 << 20, len_q=1 << 20)):
        assert fwd(**bad) == ARG, bad
        assert lib.gs_last_error_message()
    assert lib.gs_cross_attention_fwd(None, None, None, None, None, None, None, 0, None) == ARG
    a = _abi.gs_attention(dtype=0, batch=2, heads=4, kv_heads=2, head_dim=16, len_q=9, len_k=8)
    assert lib.gs_cross_attention_workspace_bytes(C.byref(a), 1) >= 2 * 4 * 9 * 4
    h = _abi.gs_heads(data=256, batch_stride=1, len_stride=1, head_stride=1)
    args = [C.byref(h)] * 5
    assert lib.gs_cross_attention_bwd(C.byref(a), *args, 256, *[C.byref(h)] * 3, None, 0, None) == ARG
    assert b"workspace" in lib.gs_last_error_message()
    a.heads = 5
    assert lib.gs_cross_attention_workspace_bytes(C.byref(a), 1) == 0


def test_bindings_refuse_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        api.gs_layer_norm_fwd(x)
    q = torch.zeros(1, 2, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        api.gs_cross_attention_fwd(q, q, q)
