"""Outputs of layer norm and cross attention that lie on inputs, on one another or on themselves are refused (CPU: host
checks before any device work, addresses that are never read)."""
import ctypes as C

import pytest
import torch

import __graft_entry__
from differentiable_gaussian_splatting_gs_gb300 import _abi

if torch.cuda.is_available():
    pytest.skip("made-up addresses: only where no device could follow them", allow_module_level=True)

KEYS = ("dout", "q", "k", "v", "out")
ROOM = 1 << 40  # the addresses below are apart by more than the tensors' sizes


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return _abi.load()


def _heads(data, len_, heads, d=64, **strides):
    s = {"batch_stride": len_ * heads * d, "len_stride": heads * d, "head_stride": d, **strides}
    return _abi.gs_heads(data=data, **s)


def _attention(**kw):
    return _abi.gs_attention(**{**dict(dtype=2, batch=2, heads=4, kv_heads=2, head_dim=64, len_q=8, len_k=9), **kw})


def _call(lib, backward, at, a=None, strides=None):
    """The call with tensors at the addresses `at`, the others apart."""
    a = a or _attention()
    at = {**{n: ROOM * (i + 1) for i, n in enumerate(KEYS + ("dq", "dk", "dv"))}, **at}
    of = {n: _heads(at[n], *((a.len_k, a.kv_heads) if n in ("k", "v", "dk", "dv") else (a.len_q, a.heads)), **(strides or {}).get(n, {}))
          for n in at}
    ref = lambda *names: [C.byref(of[n]) for n in names]  # noqa: E731
    ws, n = 1 << 50, 1 << 40
    if backward:
        st = lib.gs_cross_attention_bwd(C.byref(a), *ref(*KEYS), 256, *ref("dq", "dk", "dv"), ws, n, None)
    else:
        st = lib.gs_cross_attention_fwd(C.byref(a), *ref("q", "k", "v", "out"), 256, ws, n, None)
    return st, lib.gs_last_error_message()


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_attention_output_on_an_input(lib, name):
    st, msg = _call(lib, False, {"out": 77 * ROOM, name: 77 * ROOM})
    assert st == _abi.GS_ERR_ARG and b"out lies on" in msg


@pytest.mark.parametrize("grad", ["dq", "dk", "dv"])
@pytest.mark.parametrize("name", KEYS)
def test_attention_gradient_on_an_input(lib, grad, name):
    st, msg = _call(lib, True, {grad: 77 * ROOM, name: 77 * ROOM})
    assert st == _abi.GS_ERR_ARG and grad.encode() + b" lies on" in msg


@pytest.mark.parametrize("one,other", [("dq", "dk"), ("dq", "dv"), ("dk", "dv")])
def test_attention_gradients_on_one_another(lib, one, other):
    st, msg = _call(lib, True, {one: 77 * ROOM, other: 77 * ROOM})
    assert st == _abi.GS_ERR_ARG and other.encode() + b" lies on" in msg


@pytest.mark.parametrize("stride", ["batch_stride", "len_stride", "head_stride"])
def test_attention_outputs_of_shared_elements(lib, stride):
    for name in ("out", "dq", "dk", "dv"):
        st, msg = _call(lib, name != "out", {}, strides={name: {stride: 0}})
        assert st == _abi.GS_ERR_ARG and name.encode() + b" share memory" in msg, name


def test_layer_norm_rows_over_rows_of_another_stride(lib):
    def fwd(y_stride, y=256, rows=4):
        return lib.gs_layer_norm_fwd(256, 64, rows, 64, 0, None, None, 0, 1e-5, y, y_stride, None, None, None)

    assert fwd(72) == _abi.GS_ERR_ARG and b"another row stride" in lib.gs_last_error_message()
    for ok in (dict(y_stride=64), dict(y_stride=72, y=ROOM), dict(y_stride=72, rows=1)):  # refused for the missing statistics
        assert fwd(**ok) == _abi.GS_ERR_ARG and b"mean or rstd" in lib.gs_last_error_message()

    def bwd(dx, dx_stride, dy=ROOM, x=2 * ROOM):
        return lib.gs_layer_norm_bwd(dy, 64, x, 72, 4, 64, 0, None, None, None, 0, dx, dx_stride, None, None, None, 0, None)

    for bad in (dict(dx=ROOM, dx_stride=72), dict(dx=2 * ROOM, dx_stride=64)):
        assert bwd(**bad) == _abi.GS_ERR_ARG and b"another row stride" in lib.gs_last_error_message()
    for ok in (dict(dx=ROOM, dx_stride=64), dict(dx=2 * ROOM, dx_stride=72), dict(dx=3 * ROOM, dx_stride=80)):
        assert bwd(**ok) == _abi.GS_ERR_ARG and b"mean or rstd" in lib.gs_last_error_message()
