"""GPU cross attention, forward: the order of the softmax warps and of the products.

A warp of 32 queries takes about twice as long over a key tile in which one of its rows' maximum is raised, so here the
rows of a single warp raise theirs, in chosen key tiles, and the others never do.

Tolerance: a score and lse are off by at most 2^-20 of scale sum |q||k|, a probability by that, by 2^-20 for the
exponential and the sum, and by twice the type's unit roundoff; out is off by its probabilities' errors against sum P |v|
and rounded once.
"""
import pytest
import torch

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from differentiable_gaussian_splatting_gs_gb300 import _abi, api  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
ACC = 2.0 ** -20
TILE = 128


def _check(q, k, v, out, lse):
    """Against the definition in 64 bits; heads of q and k are the same ones."""
    for h in range(q.shape[2]):
        a, b, w = (t[0, :, h].double() for t in (q, k, v))
        scale = a.shape[1] ** -0.5
        s = a @ b.t() * scale
        p = torch.softmax(s, 1)
        size = (a.abs() @ b.abs().t() * scale).amax(1)
        want, want_lse = p @ w, torch.logsumexp(s, 1)
        u = U[q.dtype]
        tol = (2 * u + ACC + 2 * ACC * size[:, None]) * (p @ w.abs()) + u * want.abs() + TINY[q.dtype]
        bad = (out[0, :, h].double() - want).abs() / tol
        assert (bad <= 1).all(), (h, bad.max().item(), (bad > 1).any(1).nonzero()[:, 0].tolist()[:8])
        assert ((lse[0, h].double() - want_lse).abs() <= ACC * (1 + size + want_lse.abs())).all()


# 128 queries: a query tile per block. Five key tiles are walked whole; 48 key tiles of 16 heads are split into shares of
# several tiles. 120 heads of 256 queries: two query tiles per block.
@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("d", [64, 40, 128])
@pytest.mark.parametrize("heads,len_q,tiles,raises", [
    (2, 128, 5, (1, 3)), (2, 128, 5, (3,)), (2, 128, 7, (2, 5)), (3, 128, 2, (1,)), (16, 128, 48, tuple(range(1, 48))),
    (120, 256, 5, (1, 3))])
@pytest.mark.parametrize("warp", [0, 1, 2, 3])
def test_rows_of_one_warp_raise_their_maximum(dtype, d, heads, len_q, tiles, raises, warp):
    gen = torch.Generator(device="cuda").manual_seed(100 * warp + tiles)
    rand = lambda n: torch.randn(1, n, heads, d, device=DEV, generator=gen)  # noqa: E731
    q, k, v = rand(len_q), rand(tiles * TILE), rand(tiles * TILE)
    mine = torch.zeros(len_q, dtype=torch.bool, device=DEV)
    mine[32 * warp:32 * warp + 32] = True  # of the block's first query tile
    q[:, :, :, 0] = torch.where(mine, d ** 0.5, 0.0)[None, :, None]
    k[:, :, :, 0] = 0.0
    for at, tile in enumerate(raises):  # one key of the tile: 16 more than any score before it, in this warp's rows
        k[:, tile * TILE + 17, :, 0] = 24.0 + 16 * at
    q, k, v = (t.to(dtype) for t in (q, k, v))
    first = None
    for _ in range(5):
        got = api.gs_cross_attention_fwd(q, k, v)
        if first is None:
            first = got
            _check(q, k, v, *got)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert api.gs_device_error() == _abi.GS_OK
