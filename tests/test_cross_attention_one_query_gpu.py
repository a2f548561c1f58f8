"""GPU cross attention of one query whose heads share no keys (a kernel of its own): masks, lengths that leave whole shares
of the keys without any, what masked keys hold, and layouts.

Tolerance: a score and lse are off by at most 2^-20 of scale sum |q||k|, a probability by that and by 2^-20 for the
exponential and the sum; out is off by its probabilities' errors against sum P |v| and rounded once. (P is not rounded
here; the bound of the other forms, twice the type's unit roundoff, is not needed.)
"""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
ACC = 2.0 ** -20


def _rand(shape, dtype, seed, factor=1.0):
    return (factor * torch.randn(shape, device=DEV, generator=torch.Generator(device="cuda").manual_seed(seed))).to(dtype)


def _check(q, k, v, valid, **kw):
    out, lse = api.gs_cross_attention_fwd(q, k, v, **kw)
    assert torch.isfinite(out).all()
    scale = q.shape[3] ** -0.5
    for i in range(q.shape[0]):
        at = valid[i].nonzero()[:, 0]
        if at.numel() == 0:
            assert (out[i] == 0).all() and (lse[i] == -float("inf")).all()
            continue
        a, b, w = q[i, 0].double(), k[i, at].double(), v[i, at].double()  # [h, d], [n, h, d]
        s = torch.einsum("hd,nhd->hn", a, b) * scale
        p = torch.softmax(s, 1)
        size = (torch.einsum("hd,nhd->hn", a.abs(), b.abs()) * scale).amax(1)
        want, mag, want_lse = torch.einsum("hn,nhd->hd", p, w), torch.einsum("hn,nhd->hd", p, w.abs()), torch.logsumexp(s, 1)
        tol = (ACC + 2 * ACC * size[:, None]) * mag + U[q.dtype] * want.abs() + TINY[q.dtype]
        bad = (out[i, 0].double() - want).abs() / tol
        assert (bad <= 1).all(), (i, bad.max().item())
        assert ((lse[i, :, 0].double() - want_lse).abs() <= ACC * (1 + size + want_lse.abs())).all()
    assert api.gs_device_error() == _abi.GS_OK
    return out, lse


def _masks(b, lk, kind):
    """k_len, key_mask and their keys: none, one, half, a length inside and one at the end of a block's turn, all but one."""
    lens = [0, 1, lk // 2, min(lk, 513), max(0, lk - 1), lk]
    k_len = torch.tensor([lens[i % 6] for i in range(b)], dtype=torch.int32, device=DEV) if kind != "keys" else None
    key_mask = None
    if kind != "len":
        key_mask = torch.rand(b, lk, device=DEV, generator=torch.Generator(device="cuda").manual_seed(lk)) < 0.4
        key_mask[0] = False
        key_mask[1, : lk - lk // 5] = False  # only the last share has any
        if b > 2:
            key_mask[2, lk // 5:] = False    # only the first
    valid = torch.ones(b, lk, dtype=torch.bool, device=DEV)
    if k_len is not None:
        valid &= torch.arange(lk, device=DEV)[None] < k_len[:, None]
    if key_mask is not None:
        valid &= key_mask
    return k_len, key_mask, valid


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("b,h,lk,d", [(6, 2, 5000, 64), (6, 1, 4346, 128), (6, 16, 700, 40), (2, 1, 64, 8), (6, 2, 3001, 33), (6, 2, 900, 200),
                                      (6, 60, 333, 64), (6, 1, 1, 64), (6, 3, 130, 256)])
@pytest.mark.parametrize("kind", ["len", "keys", "both"])
def test_masked_keys_take_no_part_whatever_they_hold(dtype, b, h, lk, d, kind):
    q, k, v = _rand((b, 1, h, d), dtype, 1, 1.5), _rand((b, lk, h, d), dtype, 2), _rand((b, lk, h, d), dtype, 3)
    k_len, key_mask, valid = _masks(b, lk, kind)
    kw = dict(k_len=k_len, key_mask=key_mask)
    want = _check(q, k, v, valid, **kw)
    for held in (float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max, torch.finfo(dtype).min):
        k[~valid] = held
        v[~valid] = held
        got = api.gs_cross_attention_fwd(q, k, v, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), held
    # each side alone
    k[~valid] = float("nan")
    v[~valid] = 0
    assert torch.equal(api.gs_cross_attention_fwd(q, k, v, **kw)[0], want[0])
    k[~valid] = 0
    v[~valid] = float("nan")
    assert torch.equal(api.gs_cross_attention_fwd(q, k, v, **kw)[0], want[0])


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("d", [64, 40, 33])
def test_layouts(dtype, d):
    b, h, lk = 3, 4, 700
    q, k, v = _rand((b, 1, h, d), dtype, 1, 1.5), _rand((b, lk, h, d), dtype, 2), _rand((b, lk, h, d), dtype, 3)
    k_len, key_mask, valid = _masks(b, lk, "both")
    want = _check(q, k, v, valid, k_len=k_len, key_mask=key_mask)

    def inside(t, before, at):  # rows and batch entries of a larger buffer, from its middle on
        big = torch.full((t.shape[0] + 2, t.shape[1] + 3, t.shape[2] + 1, d + before), 9.0, dtype=dtype, device=DEV)
        view = big[1:-1, 2:-1, :-1, at:at + d]
        return view.copy_(t)

    def head_first(t):
        return t.transpose(1, 2).contiguous().transpose(1, 2)

    def batch_inside(t):  # batch entries nearest to one another
        return t.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)

    wide = torch.zeros(b, lk + 37, dtype=torch.bool, device=DEV)  # a mask whose rows are apart
    wide[:, 5:5 + lk] = key_mask
    for change in (lambda t: inside(t, 8, 0), lambda t: inside(t, 5, 3), lambda t: inside(t, 16, 8), head_first, batch_inside):
        lse = torch.empty_like(want[1])
        got = api.gs_cross_attention_fwd(change(q), change(k), change(v), k_len=k_len, key_mask=wide[:, 5:5 + lk],
                                         out=(change(torch.zeros_like(q)), lse))
        assert torch.equal(got[0], want[0]) and torch.equal(lse, want[1])
    got = api.gs_cross_attention_fwd(q, k, v, k_len=k_len, key_mask=key_mask.to(torch.uint8) * 7)
    assert torch.equal(got[0], want[0])
    # one mask, or one batch entry's keys, for all
    one = key_mask[1:2].expand(b, -1)
    _check(q, k[:1].expand(b, -1, -1, -1), v[:1].expand(b, -1, -1, -1), one, key_mask=one)


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("lq,h,hk", [(1, 4, 4), (7, 4, 2), (200, 2, 2)])
@pytest.mark.parametrize("d", [64, 40, 128])
def test_layouts_of_the_other_forms(dtype, lq, h, hk, d):
    # the forward and the backward of a call whose tensors lie between others of a larger buffer, against whole tensors
    b, lk = 3, 333
    q, k, v, dout = (_rand(s, dtype, i) for i, s in enumerate([(b, lq, h, d), (b, lk, hk, d), (b, lk, hk, d), (b, lq, h, d)]))
    k_len, key_mask, _ = _masks(b, lk, "both")
    kw = dict(k_len=k_len, key_mask=key_mask)
    want = api.gs_cross_attention_fwd(q, k, v, **kw)
    grads = api.gs_cross_attention_bwd(dout, q, k, v, *want, **kw)

    def inside(t, at):
        big = torch.full((t.shape[0] + 2, t.shape[1] + 3, t.shape[2] + 1, d + 16), 9.0, dtype=dtype, device=DEV)
        return big[1:-1, 2:-1, :-1, at:at + d].copy_(t)

    def batch_inside(t, at):
        return t.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)

    for change, at in ((inside, 0), (inside, 8), (inside, 3), (batch_inside, 0)):
        c = [change(t, at) for t in (dout, q, k, v)]
        got = api.gs_cross_attention_fwd(*c[1:], out=(change(torch.zeros_like(q), at), torch.empty_like(want[1])), **kw)
        back = api.gs_cross_attention_bwd(*c, *got, grads=tuple(change(torch.zeros_like(t), at) for t in (q, k, v)), **kw)
        assert all(torch.equal(x, y) for x, y in zip(got + back, want + grads)), (at, change)
